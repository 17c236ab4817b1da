"""rf_norm_rope and its gradient against their definitions in 64 bits.

Bounds. Forward: a head's squares are summed in fp32 over at most 256 channels, some 16 of them one after another and
the rest pairwise, so the mean is off by less than 24 2^-24 relatively and its inverse root by half of that, plus an
SFU's 2^-22 or two roundings; gain and inverse root are two more products: a normalised channel is off by
22 2^-24 < 1.4e-6 of itself. The rotation adds what it adds in rf_rope: (2^-19.5 or 1e-6) (|x1| + |x2|). bf16 rows are
rounded once, by at most half a step, 2^-8 of the value.
Backward: u, w as above; dx = r (w - x r^2 mean(w x)), whose mean is off by less than 24 2^-24 of mean(|w x|)."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu

EPS = 1e-5
CASES = [
    # rows, query heads, key heads, hd, rot, layout, dtype, scaling, positions
    (1, 1, 0, 8, 2, 0, 0, 0, False),
    (1, 40, 8, 128, 128, 0, 0, 0, True),
    (5, 3, 1, 128, 128, 0, 0, 2, False),
    (257, 5, 2, 64, 64, 0, 1, 1, True),
    (1000, 32, 8, 128, 64, 0, 0, 2, True),
    (33, 5, 5, 128, 96, 1, 0, 3, True),
    (33, 0, 5, 96, 32, 1, 1, 4, True),
    (70, 9, 3, 64, 20, 0, 0, 4, False),      # halves that do not divide into 16-byte pieces
    (70, 9, 3, 64, 20, 1, 1, 3, True),
    (70, 9, 3, 64, 22, 0, 1, 0, True),
    (19, 2, 2, 256, 256, 0, 1, 0, True),
    (19, 2, 2, 256, 256, 1, 1, 0, True),
    (19, 2, 2, 256, 100, 0, 0, 0, False),
    (19, 2, 2, 40, 40, 1, 0, 1, True),
    (19, 2, 1, 40, 40, 0, 0, 1, True),
    (4099, 28, 5, 128, 128, 0, 0, 0, False),
]


def _desc(rows, q, k, hd, rot, layout, dtype, scaling, ld_in, ld_out, off=0, amp=1.0, theta=1e4, eps=EPS):
    rope = rf.rf_rope_desc(n_rows=rows, n_heads=q + k, head_dim=hd, rot_dim=rot, ld_in=ld_in, ld_out=ld_out,
                           pos_offset=off, theta=theta, factor=4.0, original_rows=4096.0, low_turns=1.0, high_turns=8.0,
                           amplitude=amp, layout=layout, dtype=dtype, transpose=0, scaling=scaling)
    return rf.rf_norm_rope_desc(rope=rope, n_q_heads=q, eps=eps)


def _setup(rows, q, k, hd, rot, layout, dtype, scaling, given, pad_in=24, pad_out=8):
    t = torch.float32 if dtype else torch.bfloat16
    heads = q + k
    s = dict(x=R.randn((rows, heads * hd + pad_in), rows + hd, t), theta=1e4 if scaling != 4 else 5e5,
             amp=1.25 if scaling == 4 else 1.0, off=12345)
    s["x"] *= torch.linspace(0.01, 3.0, rows, device="cuda")[:, None].to(t)
    s["gq"], s["gk"] = (R.randn((hd,), i, torch.float32, 0.3).add_(1.0).to(t) for i in (1, 2))
    s["given"] = (torch.randperm(max(rows, 5000), generator=torch.Generator().manual_seed(rows))[:rows] * 7 - 300).int().cuda()
    s["pos"] = s["given"] if given else torch.arange(rows, device="cuda") + s["off"]
    s["freqs"] = R.frequencies(rot, s["theta"], scaling, 4.0, 4096.0, 1.0, 8.0)
    s["given"] = s["given"] if given else None
    s["desc"] = _desc(rows, q, k, hd, rot, layout, dtype, scaling, heads * hd + pad_in, heads * hd + pad_out, s["off"],
                      s["amp"], s["theta"])
    return s


def _normalised(x, gain):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r * gain, r


def _gains(s, q, k, hd):
    return torch.cat([s["gq"].double().expand(q, hd), s["gk"].double().expand(k, hd)])


@pytest.mark.parametrize("rows,q,k,hd,rot,layout,dtype,scaling,given", CASES)
def test_norm_rope_matches_its_definition(rows, q, k, hd, rot, layout, dtype, scaling, given):
    s = _setup(rows, q, k, hd, rot, layout, dtype, scaling, given)
    x, w = s["x"], (q + k) * hd
    y = torch.full((rows, w + 8), math.nan, dtype=x.dtype, device="cuda")
    rf.rf_norm_rope(s["desc"], x, s["gq"], s["gk"], y, s["given"])
    torch.cuda.synchronize()
    n, _ = _normalised(x[:, :w].reshape(rows, q + k, hd).double(), _gains(s, q, k, hd))
    want, mag = R.rope(n, s["pos"], s["freqs"], layout == 1, False, s["amp"])
    turned = mag != 0
    mag = torch.where(turned, mag, n.abs())
    bound = (1e-6 if dtype else 2.0 ** -19.5) * mag * turned + 1.4e-6 * mag + (R.U24 if dtype else R.U8) * want.abs() + 1e-30
    assert R.within(y[:, :w].reshape(rows, q + k, hd), want, bound) <= 1.0
    assert bool(torch.isnan(y[:, w:]).all())                      # nothing beyond the heads is written
    d = s["desc"]
    d.rope.ld_out = d.rope.ld_in
    rf.rf_norm_rope(d, x, s["gq"], s["gk"], x, s["given"])        # in place: the same bits
    torch.cuda.synchronize()
    bits = torch.int32 if dtype else torch.int16
    assert torch.equal(x[:, :w].contiguous().view(bits), y[:, :w].contiguous().view(bits))


def _exact_gradient(s, rows, q, k, hd, layout, dy):
    """float64 dx, dq_gain, dk_gain and their bounds, from the formula."""
    heads, w = q + k, (q + k) * hd
    x = s["x"][:, :w].reshape(rows, heads, hd).double()
    gain = _gains(s, q, k, hd)
    u, mag = R.rope(dy[:, :w].reshape(rows, heads, hd).double(), s["pos"], s["freqs"], layout == 1, True, s["amp"])
    mag = torch.where(mag != 0, mag, u.abs())
    unit, r = _normalised(x, 1.0)
    wu = gain * u
    dot = (wu * unit).mean(-1, keepdim=True)
    dx = r * (wu - unit * dot)
    dg = (u * unit).sum(0)
    tiny = 2.0 ** -19 if dy.dtype == torch.bfloat16 else 2.5e-6
    size = r * ((gain.abs() * mag) + unit.abs() * (gain.abs() * mag * unit.abs()).mean(-1, keepdim=True))
    b_dx = 2 * tiny * size + (R.U8 if dy.dtype == torch.bfloat16 else R.U24) * dx.abs() + 1e-30
    # sums over rows and heads: at most 60 additions one after another in any way to the result
    b_dg = ((tiny + 60 * R.U24) * mag * unit.abs()).sum(0)
    # (without heads of a kind its sum and its bound are both 0: the 1e-30 keeps 0 / 0 out of the comparison)
    return (dx, dg[:q].sum(0), dg[q:].sum(0)), (b_dx, b_dg[:q].sum(0) + 1e-30, b_dg[q:].sum(0) + 1e-30)


def _backward(s, dy, sums=True):
    d = s["desc"]
    hd = d.rope.head_dim
    dx = torch.full_like(s["x"], math.nan)
    dq, dk = (torch.full((hd,), math.nan, device="cuda") for _ in range(2))
    ws = torch.empty(rf.rf_norm_rope_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    rf.rf_norm_rope_backward(d, s["x"], s["gq"], s["gk"], dy, s["given"], dx, dq if sums else None, dk if sums else None,
                             ws, ws.numel())
    torch.cuda.synchronize()
    return dx, dq, dk


@pytest.mark.parametrize("rows,q,k,hd,rot,layout,dtype,scaling,given", CASES)
def test_norm_rope_gradient_matches_its_formula(rows, q, k, hd, rot, layout, dtype, scaling, given):
    s = _setup(rows, q, k, hd, rot, layout, dtype, scaling, given)
    w = (q + k) * hd
    dy = R.randn((rows, w + 8), 3, s["x"].dtype)
    dx, dq, dk = _backward(s, dy)
    want, bound = _exact_gradient(s, rows, q, k, hd, layout, dy)
    assert R.within(dx[:, :w].reshape(rows, q + k, hd), want[0], bound[0]) <= 1.0
    assert R.within(dq, want[1], bound[1]) <= 1.0 and R.within(dk, want[2], bound[2]) <= 1.0
    assert bool(torch.isnan(dx[:, w:]).all())
    again = _backward(s, dy)                                      # the same bits, with the gains' gradients or without
    alone = _backward(s, dy, sums=False)
    for a, b in zip((dx, dq, dk), again):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    assert torch.equal(alone[0].nan_to_num(7.0), dx.nan_to_num(7.0)) and bool(torch.isnan(alone[1]).all())


@pytest.mark.parametrize("layout,hd,rot", [(0, 64, 64), (1, 64, 48), (0, 64, 20)])
def test_norm_rope_gradient_against_differences(layout, hd, rot):
    """Central differences of L = <dy, y> along random directions, fp32 rows. A step of h = 2^-8 leaves the third
    derivative's h^2/6 (1.5e-5 of a curve of unit scale, taken eight times for the norm's) and the rounding of y,
    2 2^-24 sum|dy y| / 2h."""
    rows, q, k = 13, 3, 2
    s = _setup(rows, q, k, hd, rot, layout, 1, 0, False, 0, 0)
    s["x"] = R.randn((rows, (q + k) * hd), 5, torch.float32)
    dy = R.randn((rows, (q + k) * hd), 6, torch.float32)
    dx, dq, dk = _backward(s, dy)
    h = 2.0 ** -8

    def value(x, gq, gk):
        y = torch.empty_like(x)
        rf.rf_norm_rope(s["desc"], x, gq, gk, y)
        return (y.double() * dy.double()).sum(), (y * dy).double().abs().sum()

    for seed in range(3):
        e = R.randn(s["x"].shape, 20 + seed, torch.float32)
        eq, ek = R.randn((hd,), 30 + seed, torch.float32), R.randn((hd,), 40 + seed, torch.float32)
        up, size = value(s["x"] + h * e, s["gq"] + h * eq, s["gk"] + h * ek)
        down, _ = value(s["x"] - h * e, s["gq"] - h * eq, s["gk"] - h * ek)
        got = float((dx.double() * e.double()).sum() + (dq.double() * eq.double()).sum() + (dk.double() * ek.double()).sum())
        rounding = 40 * R.U24 * float(size) / h
        assert abs(float(up - down) / (2 * h) - got) <= rounding + 8 * h * h / 6 * float(size)


def test_norm_rope_without_gains_rows_or_key_heads():
    rows, hd = 6, 64
    s = _setup(rows, 2, 1, hd, hd, 0, 1, 0, False, 0, 0)
    y, z = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    one = torch.ones(hd, device="cuda")
    rf.rf_norm_rope(s["desc"], s["x"], None, None, y)
    rf.rf_norm_rope(s["desc"], s["x"], one, one, z)
    assert torch.equal(y, z)
    d = _desc(0, 2, 1, hd, hd, 0, 1, 0, 3 * hd, 3 * hd)           # no rows: gradients of nothing are zero
    dq, dk = torch.ones(hd, device="cuda"), torch.ones(hd, device="cuda")
    ws = torch.empty(rf.rf_norm_rope_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    rf.rf_norm_rope_backward(d, None, None, None, None, None, None, dq, dk, ws, ws.numel())
    assert not bool(dq.any()) and not bool(dk.any())
    d = _desc(rows, 3, 0, hd, hd, 0, 1, 0, 3 * hd, 3 * hd)        # no key heads
    dk.fill_(1.0)
    dx = torch.empty_like(s["x"])
    rf.rf_norm_rope_backward(d, s["x"], None, None, y, None, dx, dq, dk, ws, ws.numel())
    assert bool(dq.any()) and not bool(dk.any())


def test_norm_rope_heads_of_zeros_and_of_what_is_not_finite():
    """A head of zeros gives zeros and a finite gradient; a NaN or infinity stays within its head."""
    rows, hd = 9, 128
    s = _setup(rows, 2, 2, hd, hd, 0, 0, 0, False, 0, 0)
    x = s["x"].view(rows, 4, hd)
    clean, dy = torch.empty_like(s["x"]), R.randn(s["x"].shape, 8)
    rf.rf_norm_rope(s["desc"], s["x"], s["gq"], s["gk"], clean)
    clean_dx = _backward(s, dy)[0].view(rows, 4, hd)
    x[2, 1], x[4, 3, 5], x[5, 0, 7] = 0.0, math.nan, math.inf
    y = torch.empty_like(s["x"])
    rf.rf_norm_rope(s["desc"], s["x"], s["gq"], s["gk"], y)
    dx = _backward(s, dy, sums=False)[0].view(rows, 4, hd)
    y, clean = y.view(rows, 4, hd), clean.view(rows, 4, hd)
    assert not bool(y[2, 1].any()) and bool(torch.isfinite(dx[2, 1]).all())
    assert bool(torch.isnan(y[4, 3]).all()) and bool(torch.isnan(y[5, 0]).any())
    other = torch.ones((rows, 4), dtype=torch.bool, device="cuda")
    other[2, 1] = other[4, 3] = other[5, 0] = False
    assert torch.equal(y[other], clean[other]) and torch.equal(dx[other], clean_dx[other])


def test_norm_rope_gradient_in_place_of_its_inputs():
    rows, hd = 50, 128
    s = _setup(rows, 4, 2, hd, hd, 0, 0, 0, True, 0, 0)
    dy = R.randn(s["x"].shape, 9)
    dx, dq, _ = _backward(s, dy)
    for over in ("in", "d_out"):
        x, g = s["x"].clone(), dy.clone()
        to = x if over == "in" else g
        rf.rf_norm_rope_backward(s["desc"], x, s["gq"], s["gk"], g, s["given"], to)
        torch.cuda.synchronize()
        assert torch.equal(to, dx)


def test_norm_rope_and_gradient_in_one_graph():
    """Captured, replayed on new values, on a stream of its own, while an eager call runs on another."""
    rows, hd = 300, 128
    s = _setup(rows, 4, 2, hd, hd, 0, 0, 0, True, 0, 0)
    dy = R.randn(s["x"].shape, 9)
    y, dx, dq, dk = torch.empty_like(s["x"]), torch.empty_like(s["x"]), *(torch.empty(hd, device="cuda") for _ in range(2))
    ws = torch.empty(rf.rf_norm_rope_backward_workspace_bytes(s["desc"]), dtype=torch.uint8, device="cuda")

    def step():
        rf.rf_norm_rope(s["desc"], s["x"], s["gq"], s["gk"], y, s["given"])
        rf.rf_norm_rope_backward(s["desc"], s["x"], s["gq"], s["gk"], dy, s["given"], dx, dq, dk, ws, ws.numel())

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    s["x"].copy_(R.randn(s["x"].shape, 77))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(s["x"])
    g.replay()
    with torch.cuda.stream(side):
        rf.rf_norm_rope(s["desc"], s["x"], s["gq"], s["gk"], other, s["given"])
    torch.cuda.synchronize()
    got = (y.clone(), dx.clone(), dq.clone(), dk.clone())
    step()
    torch.cuda.synchronize()
    assert torch.equal(other, y) and all(torch.equal(a, b) for a, b in zip(got, (y, dx, dq, dk)))
