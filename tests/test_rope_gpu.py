"""rf_rope and rf_tree_build against their definitions in 64 bits.

Bounds: the fixed-point angle is off by less than 2e-7 rad (fp32 rounding of the reduced
angle) plus the table's rounding, a few 2^-52 of the unreduced angle; sine and cosine by
2^-20.4 (bf16 rows) or two fp32 ulps (fp32 rows); two products and a sum follow in fp32,
and bf16 rows are rounded once. An element is therefore within
(2^-19.5 or 1e-6) (|x1| + |x2|) amplitude, plus half an ulp of bf16."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu

CASES = [
    # rows, heads, hd, rot, layout, dtype, transpose, scaling, positions
    (1, 1, 8, 2, 0, 0, 0, 0, False),
    (5, 3, 128, 128, 0, 0, 0, 0, False),
    (257, 7, 64, 64, 0, 1, 1, 1, True),
    (1000, 40, 128, 64, 0, 0, 1, 2, True),
    (33, 5, 128, 96, 1, 0, 0, 3, True),
    (33, 5, 96, 32, 1, 1, 0, 4, True),
    (70, 9, 64, 20, 0, 0, 0, 4, False),
    (70, 9, 64, 20, 1, 1, 1, 3, True),
    (19, 2, 256, 256, 0, 1, 0, 0, True),
    (19, 2, 40, 40, 1, 0, 0, 1, True),
    (4099, 33, 128, 128, 0, 0, 0, 0, False),
]


def _desc(rows, heads, hd, rot, layout, dtype, transpose, scaling, ld_in, ld_out, off=0, amp=1.0, theta=1e4):
    return rf.rf_rope_desc(n_rows=rows, n_heads=heads, head_dim=hd, rot_dim=rot, ld_in=ld_in, ld_out=ld_out,
                           pos_offset=off, theta=theta, factor=4.0, original_rows=4096.0, low_turns=1.0, high_turns=8.0,
                           amplitude=amp, layout=layout, dtype=dtype, transpose=transpose, scaling=scaling)


def _check(got, x, pos, freqs, interleaved, transpose, amp, dtype):
    want, mag = R.rope(x.double(), pos, freqs, interleaved, transpose, amp)
    bound = (1e-6 if dtype else 2.0 ** -19.5) * mag + (0.0 if dtype else R.U8) * want.abs() + 1e-30
    rot = 2 * len(freqs)
    assert torch.equal(got[..., rot:], x[..., rot:])
    assert R.within(got[..., :rot], want[..., :rot], bound[..., :rot]) <= 1.0


@pytest.mark.parametrize("rows,heads,hd,rot,layout,dtype,transpose,scaling,given", CASES)
def test_rope_matches_its_definition(rows, heads, hd, rot, layout, dtype, transpose, scaling, given):
    t = torch.float32 if dtype else torch.bfloat16
    ld_in, ld_out = heads * hd + 24, heads * hd + 8
    x = R.randn((rows, ld_in), rows + hd, t)
    y = torch.full((rows, ld_out), math.nan, dtype=t, device="cuda")
    theta = 1e4 if scaling != 4 else 5e5
    amp = 1.25 if scaling == 4 else 1.0
    pos = (torch.randperm(max(rows, 5000), generator=torch.Generator().manual_seed(rows))[:rows] * 7 - 300).int().cuda()
    off = 12345
    d = _desc(rows, heads, hd, rot, layout, dtype, transpose, scaling, ld_in, ld_out, off, amp, theta)
    rf.rf_rope(d, x, y, pos if given else None)
    torch.cuda.synchronize()
    p = pos if given else torch.arange(rows, device="cuda") + off
    fr = R.frequencies(rot, theta, scaling, 4.0, 4096.0, 1.0, 8.0)
    w = heads * hd
    _check(y[:, :w].reshape(rows, heads, hd), x[:, :w].reshape(rows, heads, hd), p, fr, layout == 1, bool(transpose),
           amp, dtype)
    assert bool(torch.isnan(y[:, w:]).all())                      # nothing beyond the heads is written
    rf.rf_rope(_desc(rows, heads, hd, rot, layout, dtype, transpose, scaling, ld_in, ld_in, off, amp, theta), x, x,
               pos if given else None)                            # in place: the same bits
    torch.cuda.synchronize()
    assert torch.equal(x[:, :w].view(torch.int16 if not dtype else torch.int32),
                       y[:, :w].contiguous().view(torch.int16 if not dtype else torch.int32))


@pytest.mark.parametrize("off", [0, -4096, (1 << 27) + 12345])
def test_rope_far_positions_and_agreement_with_rope_rows(off):
    rows, heads, hd = 130, 3, 128
    x = R.randn((rows, heads * hd), 3)
    y, z = torch.empty_like(x), torch.empty_like(x)
    rf.rf_rope(_desc(rows, heads, hd, hd, 0, 0, 0, 0, heads * hd, heads * hd, off, theta=1e6), x, y)
    rf.rf_rope_rows(x, z, rows, heads * hd, heads, hd, 1e6, off, False)
    torch.cuda.synchronize()
    fr = R.frequencies(hd, 1e6)
    _check(y.view(rows, heads, hd), x.view(rows, heads, hd), torch.arange(rows, device="cuda") + off, fr, False, False,
           1.0, 0)
    # the same angles to the table's last bits: at most an ulp of bf16 apart, almost never that
    differ = (y.view(torch.int16) != z.view(torch.int16)).float().mean()
    assert float(differ) < 2e-3


@pytest.mark.parametrize("layout", [0, 1])
def test_rope_gradient_is_the_transposed_rotation(layout):
    """<g, J dx> = <Jᵀ g, dx>: the transposed call is the gradient of the forward one, against the formula (inner
    products of random vectors, fp32 rows) and against differences of the forward call."""
    rows, heads, hd, rot = 37, 4, 64, 48
    x, g = R.randn((rows, heads * hd), 5, torch.float32), R.randn((rows, heads * hd), 6, torch.float32)
    f = _desc(rows, heads, hd, rot, layout, 1, 0, 0, heads * hd, heads * hd, 1000, 1.5)
    b = _desc(rows, heads, hd, rot, layout, 1, 1, 0, heads * hd, heads * hd, 1000, 1.5)
    jx, jtg = torch.empty_like(x), torch.empty_like(x)
    rf.rf_rope(f, x, jx)
    rf.rf_rope(b, g, jtg)
    lhs, rhs = (g.double() * jx.double()).sum(), (jtg.double() * x.double()).sum()
    size = (g.double() * jx.double()).abs().sum()
    assert abs(float(lhs - rhs)) <= 4e-6 * float(size)
    # central differences of L = <g, R(x)> in one direction (the map is linear: only rounding remains)
    dx = R.randn((rows, heads * hd), 7, torch.float32)
    up, dn = torch.empty_like(x), torch.empty_like(x)
    rf.rf_rope(f, x + 0.5 * dx, up)
    rf.rf_rope(f, x - 0.5 * dx, dn)
    diff = (g.double() * (up.double() - dn.double())).sum()
    want = (jtg.double() * dx.double()).sum()
    assert abs(float(diff - want)) <= 1e-5 * float((g.double() * jx.double()).abs().sum() + (g * dx).double().abs().sum())


@pytest.mark.parametrize("B,n", [(1, 1), (3, 7), (2, 64), (2, 65), (5, 200), (1, 1024)])
def test_tree_build_masks_and_positions(B, n):
    par = [R.random_parents(n, 10 * b + n, reach=1 if b == 1 else 5) for b in range(B)]
    p = torch.tensor(par, dtype=torch.int32).cuda()
    nxt = (torch.arange(B, dtype=torch.int32) * 1000 + 5).cuda()
    mask = torch.full((B, n, (n + 63) // 64), -1, dtype=torch.int64, device="cuda")
    pos = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rf.rf_tree_build(B, n, p, nxt, mask, pos, st)
    only = torch.empty_like(mask)
    rf.rf_tree_build(B, n, p, None, only, None, st)
    torch.cuda.synchronize()
    seen = torch.stack([R.ancestors(x) for x in par])
    assert torch.equal(mask.cpu(), R.words(seen)) and torch.equal(only, mask) and int(st.item()) == 0
    assert torch.equal(pos.cpu(), (nxt.cpu()[:, None] + seen.sum(-1) - 1).int())


@pytest.mark.parametrize("bad", [[0, 0, 1], [-1, 1, 0], [-1, 0, 2], [-1, -1, 0], [-1, 0, -7], [-1, 5, 0]])
def test_tree_build_reports_wrong_parents_and_leaves_their_outputs(bad):
    p = torch.tensor([[-1, 0, 0], bad, [-1, 0, 1]], dtype=torch.int32).cuda()
    nxt = torch.tensor([0, 10, 20], dtype=torch.int32).cuda()
    mask = torch.full((3, 3, 1), -1, dtype=torch.int64, device="cuda")
    pos = torch.full((3, 3), -1, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rf.rf_tree_build(3, 3, p, nxt, mask, pos, st)
    torch.cuda.synchronize()
    assert int(st.item()) == rf.RF_ERR_INVALID_ARG
    assert mask.cpu()[:, :, 0].tolist() == [[1, 3, 5], [-1, -1, -1], [1, 3, 7]]
    assert pos.cpu().tolist() == [[0, 1, 1], [-1, -1, -1], [20, 21, 22]]
