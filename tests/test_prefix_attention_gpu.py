"""rf_prefix_attention against its definition in 64 bits: the sequences' keys are the prefix's rows followed by
their own, within the bounds that decoderef.attention derives for one sequence's attention (joining parts adds a
few 2^-24 to its 2^-19). What must have no influence is filled with NaN."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _seen(kind, B, n, seed):
    if kind == "order":
        return None
    if kind == "tree":
        return torch.stack([R.ancestors(R.random_parents(n, seed + b)) for b in range(B)])
    if kind == "none":
        return torch.zeros((B, n, n), dtype=torch.bool)
    g = torch.Generator().manual_seed(seed)
    s = torch.rand((B, n, n), generator=g) < 0.3
    s[:, ::3] = False                      # rows that see no drafted row
    return s


def _desc(q, kp, k, kd, out, H, scale):
    B, n, Hq, hd = q.shape
    return rf.rf_prefix_attn_desc(
        attn=rf.rf_attn_desc(n_seqs=B, n_q_heads=Hq, n_kv_heads=H, head_dim=hd, n_nodes=n, capacity=k.shape[1],
                             q_row_stride=q.stride(1), q_seq_stride=q.stride(0), draft_row_stride=kd.stride(1),
                             draft_seq_stride=kd.stride(0), cache_row_stride=k.stride(1), cache_seq_stride=k.stride(0),
                             out_row_stride=out.stride(1), out_seq_stride=out.stride(0), scale=scale),
        prefix_capacity=kp.shape[0], prefix_row_stride=kp.stride(0))


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _call(q, kp, vp, plen, k, v, kd, vd, lens, mask, scale, H, out=None, lse=True, status=None, ws=None):
    B, n, Hq, hd = q.shape
    out = torch.full((B, n, Hq, hd), math.nan, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse_t = torch.full((B, n, Hq), math.nan, device=DEV) if lse else None
    d = _desc(q, kp, k, kd, out, H, scale)
    wsb = rf.rf_prefix_attn_workspace_bytes(d)
    ws = torch.full((wsb,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws   # NaN everywhere
    st = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
    rf.rf_prefix_attention(d, q, kp, vp, plen, k, v, lens, kd, vd, mask, out, lse_t, st, ws, wsb)
    return out, lse_t, st


def _data(B, n, H, G, hd, P, lens, seed, sharp=2.0):
    cap = max(max(lens), 1) + 3
    q = R.randn((B, n, H * G, hd), seed, std=sharp)
    kp, vp = R.randn((P + 5, H, hd), seed + 5), R.randn((P + 5, H, hd), seed + 6)
    k, v = R.randn((B, cap, H, hd), seed + 1), R.randn((B, cap, H, hd), seed + 2)
    kd, vd = R.randn((B, n, H, hd), seed + 3), R.randn((B, n, H, hd), seed + 4)
    for b in range(B):                       # rows not in use hold anything
        k[b, lens[b]:] = math.nan
        v[b, lens[b]:] = math.nan
    kp[P:], vp[P:] = math.nan, math.nan
    return q, kp, vp, k, v, kd, vd


def _want(q, kp, vp, P, k, v, kd, vd, lens, seen, scale):
    """Every sequence's keys in one row of rows."""
    B, cap = k.shape[:2]
    long = torch.zeros((B, P + cap) + k.shape[2:], dtype=k.dtype, device=DEV), torch.zeros((B, P + cap) + k.shape[2:], dtype=k.dtype, device=DEV)
    for x, p, own in zip(long, (kp, vp), (k, v)):
        x[:, :P] = p[:P]
        for b in range(B):
            x[b, P:P + lens[b]] = own[b, :lens[b]]
    return R.attention(q, *long, kd, vd, [P + m for m in lens], seen, scale)


CASES = [
    # B, n, H, G, hd, prefix, lens, kind
    (1, 1, 1, 1, 128, 0, [0], "order"),
    (1, 1, 1, 1, 64, 0, [0], "none"),                          # a row that sees nothing
    (1, 1, 1, 1, 64, 1, [0], "none"),
    (2, 1, 2, 5, 128, 1, [1, 0], "order"),
    (3, 1, 2, 4, 64, 127, [127, 128, 129], "order"),
    (3, 1, 2, 4, 64, 128, [0, 5, 0], "order"),
    (3, 1, 2, 4, 128, 129, [300, 1, 17], "order"),
    (4, 1, 8, 5, 128, 5001, [200, 0, 77, 130], "order"),       # one row tile, parts of many CTAs
    (32, 1, 1, 4, 128, 3000, [10 * b for b in range(32)], "order"),    # 128 rows exactly
    (33, 1, 1, 4, 128, 3000, [10 * b for b in range(33)], "order"),    # two row tiles, four rows in the second
    (64, 1, 2, 4, 128, 1000, [(37 * b) % 500 for b in range(64)], "order"),
    (100, 3, 2, 10, 64, 777, [(131 * b) % 300 for b in range(100)], "order"),   # tiles of 4 sequences, 120 rows
    (40, 3, 2, 2, 64, 0, [(37 * b) % 400 for b in range(40)], "tree"),  # two row tiles without a prefix
    (9, 7, 2, 3, 128, 640, [0, 300, 5, 128, 127, 1, 2, 3, 4], "tree"),
    (6, 16, 2, 8, 64, 2000, [1000, 1, 0, 513, 128, 7], "random"),      # a sequence's rows are a whole tile
    (2, 13, 1, 10, 128, 300, [700, 255], "tree"),              # a sequence's rows take two tiles
    (3, 64, 2, 4, 128, 1500, [900, 40, 0], "tree"),
    (2, 65, 1, 7, 64, 640, [100, 333], "random"),
    (2, 200, 2, 5, 128, 333, [50, 129], "order"),
    (1, 129, 1, 1, 64, 129, [0], "order"),
    (2, 300, 1, 2, 128, 100, [100, 3], "random"),              # five mask words, three draft tiles
    (3, 2, 1, 128, 128, 900, [9, 0, 130], "order"),            # every row of a tile is one node
    (300, 1, 1, 1, 64, 20000, [b % 3 for b in range(300)], "order"),   # three row tiles, many short items
    (5, 1, 3, 1, 128, 20000, [0] * 5, "order"),
    (20, 13, 8, 4, 128, 8500, [(29 * b) % 90 for b in range(20)], "tree"),      # five items a head over more than 32 MB: in step
    (33, 7, 7, 3, 128, 9500, [(29 * b) % 300 for b in range(33)], "random"),
]


@pytest.mark.parametrize("B,n,H,G,hd,P,lens,kind", CASES)
def test_prefix_attention_matches_its_definition(B, n, H, G, hd, P, lens, kind):
    q, kp, vp, k, v, kd, vd = _data(B, n, H, G, hd, P, lens, 7 * n + H)
    seen = _seen(kind, B, n, n)
    mask = None if seen is None else R.words(seen).cuda()
    scale = hd ** -0.5
    args = (q, kp, vp, _ints([P]), k, v, kd, vd, _ints(lens), mask, scale, H)
    out, lse, st = _call(*args)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want, wl, bo, bl = _want(q, kp, vp, P, k, v, kd, vd, lens, seen, scale)
    assert R.within(out, want, bo) <= 1.0
    assert R.within(lse, wl, bl) <= 1.0
    again, lse2, _ = _call(*args)                              # the same bits every time
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G", [4, 8])
def test_prefix_attention_strides_views_and_a_null_lse(G):
    """The prefix as one layer and sequence of a filled cache; queries, keys and values as parts of one projection's
    rows; an output with room between rows. What lies between is not written."""
    B, n, H, hd, P, cap = 5, 4, 2, 128, 400, 70
    W = G * H + 2 * H + 1
    fused = R.randn((B, n + 2, W, hd), 11)
    q, kd, vd = fused[:, 1:n + 1, :G * H], fused[:, 1:n + 1, G * H:G * H + H], fused[:, 1:n + 1, G * H + H:G * H + 2 * H]
    filled = R.randn((3, 2, P, H + 1, hd), 13)
    kp, vp = filled[1, 0, :, 1:], filled[2, 1, :, 1:]
    caches = R.randn((3, 2, B, cap, H, hd), 12)
    k, v = caches[1, 0], caches[1, 1]
    big = torch.full((B, n, G * H + 3, hd), 5.0, dtype=torch.bfloat16, device=DEV)
    lens = [59, 17, 0, 70, 1]
    seen = _seen("tree", B, n, 3)
    _call(q, kp, vp, _ints([P - 3]), k, v, kd, vd, _ints(lens), R.words(seen).cuda(), 0.1, H, out=big[:, :, 1:G * H + 1], lse=False)
    torch.cuda.synchronize()
    want, _, bo, _ = _want(q, kp, vp, P - 3, k, v, kd, vd, lens, seen, 0.1)
    assert R.within(big[:, :, 1:G * H + 1], want, bo) <= 1.0
    assert bool((big[:, :, 0] == 5.0).all()) and bool((big[:, :, G * H + 1:] == 5.0).all())


@pytest.mark.parametrize("B,n,G", [(2, 3, 4), (70, 2, 4), (3, 64, 4)])
def test_prefix_attention_without_a_prefix_and_as_one_sequence(B, n, G):
    """An empty prefix gives what rf_tree_attention gives; a prefix that is all of the cache, too."""
    H, hd = 2, 64
    lens = [(61 * b) % 200 for b in range(B)]
    q, kp, vp, k, v, kd, vd = _data(B, n, H, G, hd, 50, lens, 5)
    out, lse, st = _call(q, kp, vp, _ints([0]), k, v, kd, vd, _ints(lens), None, 0.125, H)
    want, wl, bo, bl = R.attention(q, k, v, kd, vd, lens, None, 0.125)
    assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0
    plain, plain_lse = torch.empty_like(out), torch.empty_like(lse)
    d = _desc(q, kp, k, kd, out, H, 0.125).attn
    ws = torch.empty(rf.rf_attn_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    rf.rf_tree_attention(d, q, k, v, _ints(lens), kd, vd, None, plain, plain_lse, None, ws, ws.numel())
    torch.cuda.synchronize()
    assert R.within(out, plain.double(), 2 * bo + 1e-30) <= 1.0 and R.within(lse, plain_lse.double(), 2 * bl) <= 1.0


@pytest.mark.parametrize("B,n,G", [(3, 6, 4), (40, 6, 4), (2, 64, 4)])
def test_prefix_attention_values_that_are_not_finite(B, n, G):
    """Drafted rows that a node does not see may hold NaN and infinities; those that are seen, and prefix rows, decide."""
    H, hd, P = 2, 128, 333
    lens = [(37 * b) % 150 for b in range(B)]
    q, kp, vp, k, v, kd, vd = _data(B, n, H, G, hd, P, lens, 3)
    seen = torch.stack([R.ancestors([-1] + [0] * (n - 1))] * B)       # a star: node i sees 0 and itself
    mask = R.words(seen).cuda()
    base = (k, v)
    clean, lse0, _ = _call(q, kp, vp, _ints([P]), *base, kd, vd, _ints(lens), mask, 0.09, H)
    kd2, vd2 = kd.clone(), vd.clone()
    vd2[1, 1] = math.nan
    vd2[0, 2, 0, 5], vd2[0, 2, 1, 70] = math.inf, -math.inf
    kd2[0, 3] = math.nan
    out, lse, st = _call(q, kp, vp, _ints([P]), *base, kd2, vd2, _ints(lens), mask, 0.09, H)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    same = torch.ones((B, n), dtype=torch.bool, device=DEV)
    same[1, 1] = same[0, 2] = same[0, 3] = False
    assert torch.equal(out[same], clean[same]) and torch.equal(lse[same], lse0[same])
    want, wl, bo, bl = _want(q, kp, vp, P, *base, kd2, vd2, lens, seen, 0.09)
    assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0
    kp[7, 1] = math.nan                                               # a prefix row that all see: one KV head is lost
    out, lse, _ = _call(q, kp, vp, _ints([P]), *base, kd, vd, _ints(lens), mask, 0.09, H)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[:, :, G:]).all()) and torch.equal(out[:, :, :G], clean[:, :, :G])


@pytest.mark.parametrize("B,n", [(4, 1), (80, 1), (3, 40)])
def test_prefix_attention_lengths_out_of_range(B, n):
    H, G, hd, P = 2, 4, 64, 200
    lens = [20] * B
    q, kp, vp, k, v, kd, vd = _data(B, n, H, G, hd, P, lens, 9)
    good, lse_good, _ = _call(q, kp, vp, _ints([P]), k, v, kd, vd, _ints(lens), None, 0.1, H)
    bad = list(lens)
    bad[1], bad[2] = -1, k.shape[1] + 1
    out, lse, st = _call(q, kp, vp, _ints([P]), k, v, kd, vd, _ints(bad), None, 0.1, H)
    torch.cuda.synchronize()
    assert int(st.item()) == rf.RF_ERR_INVALID_ARG
    rest = [b for b in range(B) if b not in (1, 2)]
    want, wl, bo, bl = _want(q, kp, vp, P, k, v, kd, vd, lens, None, 0.1)
    assert R.within(out[rest], want[rest], bo[rest]) <= 1.0
    assert bool(torch.isnan(out[1:3].float()).all()) and bool(torch.isnan(lse[1:3]).all())
    for wrong in (-1, kp.shape[0] + 1):
        out, lse, st = _call(q, kp, vp, _ints([wrong]), k, v, kd, vd, _ints(lens), None, 0.1, H)
        torch.cuda.synchronize()
        assert int(st.item()) == rf.RF_ERR_INVALID_ARG
        assert bool(torch.isnan(out.float()).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("B,n", [(6, 1), (60, 2), (4, 50)])
def test_prefix_attention_in_a_graph_whose_lengths_change(B, n):
    H, G, hd, P = 2, 4, 128, 700
    lens = [(17 * b) % 90 for b in range(B)]
    q, kp, vp, k, v, kd, vd = _data(B, n, H, G, hd, P, lens, 21)
    ln, pl = _ints(lens), _ints([P])
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    d = _desc(q, kp, k, kd, out, H, 0.1)
    ws = torch.empty(rf.rf_prefix_attn_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    _call(q, kp, vp, pl, k, v, kd, vd, ln, None, 0.1, H, out=out, lse=False, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _ = rf.rf_prefix_attention(d, q, kp, vp, pl, k, v, ln, kd, vd, None, out, None, None, ws, ws.numel())
    for p, step in ((P, 0), (5, 1), (0, 2), (699, 3)):
        now = [max(0, m - 3 * step) for m in lens]
        ln.copy_(_ints(now))
        pl.fill_(p)
        g.replay()
        torch.cuda.synchronize()
        want, _, bo, _ = _want(q, kp, vp, p, k, v, kd, vd, now, None, 0.1)
        assert R.within(out, want, bo) <= 1.0
        eager, _, _ = _call(q, kp, vp, pl, k, v, kd, vd, ln, None, 0.1, H)
        torch.cuda.synchronize()
        assert torch.equal(eager.view(torch.int16), out.view(torch.int16))


def test_prefix_attention_on_two_streams_with_workspaces_of_their_own():
    B, n, H, G, hd, P = 20, 1, 2, 4, 64, 900
    lens = [5 * b for b in range(B)]
    q, kp, vp, k, v, kd, vd = _data(B, n, H, G, hd, P, lens, 2)
    pl, ln = _ints([P]), _ints(lens)
    want, _, _ = _call(q, kp, vp, pl, k, v, kd, vd, ln, None, 0.1, H)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([_call(q, kp, vp, pl, k, v, kd, vd, ln, None, 0.1, H)[0] for _ in range(5)])
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, want) for x in o)
