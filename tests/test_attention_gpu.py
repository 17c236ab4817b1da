"""rf_tree_attention against its definition in 64 bits, within the bounds that
decoderef.attention derives; what must have no influence is filled with NaN."""
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


def _call(q, k, v, kd, vd, lens, mask, scale, H, out=None, lse=True, status=None, stream=None, ws=None):
    B, n, Hq, hd = q.shape
    cap = k.shape[1]
    out = torch.full((B, n, Hq, hd), math.nan, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse_t = torch.full((B, n, Hq), math.nan, device=DEV) if lse else None
    d = rf.rf_attn_desc(n_seqs=B, n_q_heads=Hq, n_kv_heads=H, head_dim=hd, n_nodes=n, capacity=cap,
                        q_row_stride=q.stride(1), q_seq_stride=q.stride(0), draft_row_stride=kd.stride(1),
                        draft_seq_stride=kd.stride(0), cache_row_stride=k.stride(1), cache_seq_stride=k.stride(0),
                        out_row_stride=out.stride(1), out_seq_stride=out.stride(0), scale=scale)
    wsb = rf.rf_attn_workspace_bytes(d)
    ws = torch.full((wsb,), 0xFF, dtype=torch.uint8, device=DEV) if ws is None else ws   # NaN everywhere
    st = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
    rf.rf_tree_attention(d, q, k, v, lens, kd, vd, mask, out, lse_t, st, ws, wsb, stream=stream)
    return out, lse_t, st


def _data(B, n, H, G, hd, cap, lens, seed, sharp=2.0):
    q = R.randn((B, n, H * G, hd), seed, std=sharp)
    k, v = R.randn((B, cap, H, hd), seed + 1), R.randn((B, cap, H, hd), seed + 2)
    kd, vd = R.randn((B, n, H, hd), seed + 3), R.randn((B, n, H, hd), seed + 4)
    for b in range(B):                       # rows not in use hold anything
        k[b, lens[b]:] = math.nan
        v[b, lens[b]:] = math.nan
    return q, k, v, kd, vd


CASES = [
    # B, n, H, G, hd, lens, kind
    (1, 1, 1, 1, 128, [0], "order"),
    (1, 1, 1, 1, 64, [0], "none"),                         # a row that sees nothing
    (1, 1, 2, 5, 128, [1], "order"),
    (3, 1, 2, 4, 64, [127, 128, 129], "order"),
    (1, 1, 8, 5, 128, [5001], "order"),
    (2, 7, 2, 3, 128, [0, 300], "tree"),
    (4, 16, 2, 8, 64, [1000, 1, 0, 513], "random"),        # 128 rows exactly
    (2, 13, 1, 10, 128, [700, 255], "tree"),               # two row tiles, 120 rows in a full one
    (2, 64, 2, 4, 128, [1500, 40], "tree"),
    (1, 65, 1, 7, 64, [640], "random"),
    (1, 200, 2, 5, 128, [333], "order"),
    (1, 129, 1, 1, 64, [0], "order"),
    (1, 300, 1, 2, 128, [100], "random"),                  # five mask words, three draft tiles
    (1, 1024, 1, 1, 64, [77], "tree"),
    (40, 3, 2, 2, 64, [(37 * b) % 400 for b in range(40)], "tree"),
    (1, 2, 1, 128, 128, [900], "order"),                   # every row of a tile is one node
    (2, 1, 1, 128, 64, [256, 3], "order"),
    (1, 5, 3, 1, 128, [20000], "order"),                   # one head's keys over many shares
]


@pytest.mark.parametrize("B,n,H,G,hd,lens,kind", CASES)
def test_attention_matches_its_definition(B, n, H, G, hd, lens, kind):
    cap = max(max(lens), 1) + 3
    q, k, v, kd, vd = _data(B, n, H, G, hd, cap, lens, 7 * n + H)
    seen = _seen(kind, B, n, n)
    mask = None if seen is None else R.words(seen).cuda()
    scale = hd ** -0.5
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse, st = _call(q, k, v, kd, vd, ln, mask, scale, H)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want, wl, bo, bl = R.attention(q, k, v, kd, vd, lens, seen, scale)
    assert R.within(out, want, bo) <= 1.0
    assert R.within(lse, wl, bl) <= 1.0
    again, lse2, _ = _call(q, k, v, kd, vd, ln, mask, scale, H)       # the same bits every time
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_attention_strides_views_and_a_null_lse():
    """Queries, keys and values as parts of one projection's rows; a layer of a [layers][rows][heads] cache; an
    output with room between rows. What lies between is not written."""
    B, n, H, G, hd, cap = 2, 9, 2, 4, 128, 260
    W = G * H + 2 * H + 1
    fused = R.randn((B, n + 2, W, hd), 11)
    q, kd, vd = fused[:, 1:n + 1, :G * H], fused[:, 1:n + 1, G * H:G * H + H], fused[:, 1:n + 1, G * H + H:G * H + 2 * H]
    caches = R.randn((3, 2, B, cap, H, hd), 12)
    k, v = caches[1, 0], caches[1, 1]
    big = torch.full((B, n, G * H + 3, hd), 5.0, dtype=torch.bfloat16, device=DEV)
    lens = [259, 17]
    seen = _seen("tree", B, n, 3)
    _call(q, k, v, kd, vd, torch.tensor(lens, dtype=torch.int32, device=DEV), R.words(seen).cuda(), 0.1, H,
          out=big[:, :, 1:G * H + 1], lse=False)
    torch.cuda.synchronize()
    want, _, bo, _ = R.attention(q, k, v, kd, vd, lens, seen, 0.1)
    assert R.within(big[:, :, 1:G * H + 1], want, bo) <= 1.0
    assert bool((big[:, :, 0] == 5.0).all()) and bool((big[:, :, G * H + 1:] == 5.0).all())


@pytest.mark.parametrize("n,G", [(6, 4), (64, 4)])
def test_attention_unseen_drafted_rows_have_no_influence(n, G):
    """Drafted rows that a node does not see may hold NaN and infinities in K and V: nodes that do not see them are
    unchanged; nodes that do get what the sum gives."""
    H, hd, lens = 2, 128, [333]
    q, k, v, kd, vd = _data(1, n, H, G, hd, 340, lens, 3)
    seen = torch.stack([R.ancestors([-1] + [0] * (n - 1))])       # a star: node i sees 0 and itself
    mask = R.words(seen).cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    clean, lse0, _ = _call(q, k, v, kd, vd, ln, mask, 0.09, H)
    kd2, vd2 = kd.clone(), vd.clone()
    vd2[0, 1] = math.nan
    vd2[0, 2, 0, 5], vd2[0, 2, 1, 70] = math.inf, -math.inf
    kd2[0, 3] = math.nan
    out, lse, st = _call(q, k, v, kd2, vd2, ln, mask, 0.09, H)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    others = [i for i in range(n) if i not in (1, 2, 3)]
    assert torch.equal(out[:, others], clean[:, others]) and torch.equal(lse[:, others], lse0[:, others])
    want, wl, bo, bl = R.attention(q, k, v, kd2, vd2, lens, seen, 0.09)
    assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0


def test_attention_in_order_ignores_later_rows_that_are_not_finite():
    n, H, G, hd, lens = 150, 1, 2, 64, [50]
    q, k, v, kd, vd = _data(1, n, H, G, hd, 64, lens, 4)
    vd[0, 140:] = math.nan
    kd[0, 145:] = math.inf
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse, _ = _call(q, k, v, kd, vd, ln, None, 0.1, H)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[0, :140]).all()) and bool(torch.isnan(out[0, 140:]).all())
    want, wl, bo, bl = R.attention(q[:, :140], k, v, kd[:, :140], vd[:, :140], lens, None, 0.1)
    assert R.within(out[:, :140], want, bo) <= 1.0 and R.within(lse[:, :140], wl, bl) <= 1.0


def test_attention_growing_scores_rescale_the_accumulator():
    """Scores that grow along the keys by far more than the deferred rescaling lets pass, up to weights that vanish."""
    H, G, hd, m = 1, 4, 64, 2000
    q = torch.ones((1, 2, G, hd), dtype=torch.bfloat16, device=DEV)
    k = (torch.arange(m, device=DEV, dtype=torch.float32) / 16).to(torch.bfloat16)[None, :, None, None].expand(1, m, 1, hd).contiguous()
    v = R.randn((1, m, 1, hd), 5)
    kd, vd = torch.zeros((1, 2, 1, hd), dtype=torch.bfloat16, device=DEV), R.randn((1, 2, 1, hd), 6)
    for scale in (1.0 / 64, 0.25, 4.0):
        out, lse, _ = _call(q, k, v, kd, vd, torch.tensor([m], dtype=torch.int32, device=DEV), None, scale, H)
        flip = k.flip(1).contiguous()
        out2, lse2, _ = _call(q, flip, v.flip(1).contiguous(), kd, vd, torch.tensor([m], dtype=torch.int32, device=DEV),
                              None, scale, H)
        torch.cuda.synchronize()
        want, wl, bo, bl = R.attention(q, k, v, kd, vd, [m], None, scale)
        assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0
        assert R.within(out2, want, bo) <= 1.0 and R.within(lse2, wl, bl) <= 1.0


@pytest.mark.parametrize("bad", [-1, 1 << 30, 301])
def test_attention_reports_a_wrong_length_and_goes_on_with_the_rest(bad):
    B, n, H, G, hd = 3, 4, 2, 4, 128
    lens = [300, 300, 150]
    q, k, v, kd, vd = _data(B, n, H, G, hd, 300, lens, 8)
    good, _, _ = _call(q, k, v, kd, vd, torch.tensor(lens, dtype=torch.int32, device=DEV), None, 0.09, H)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse, _ = _call(q, k, v, kd, vd, torch.tensor([300, bad, 150], dtype=torch.int32, device=DEV), None, 0.09, H,
                        status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == rf.RF_ERR_INVALID_ARG
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
    want, _, bo, _ = R.attention(q[[0, 2]], k[[0, 2]], v[[0, 2]], kd[[0, 2]], vd[[0, 2]], [300, 150], None, 0.09)
    assert R.within(out[[0, 2]], want, bo) <= 1.0


def test_attention_on_another_stream_and_offsets_beyond_32_bits():
    """The second sequence lies 2^31 elements behind the first."""
    B, n, H, G, hd, cap = 2, 3, 1, 2, 128, 500
    stride = (1 << 31) + 64 * hd
    buf = torch.empty(stride + cap * hd, dtype=torch.bfloat16, device=DEV)
    k = buf.as_strided((B, cap, H, hd), (stride, hd, hd, 1))
    q, ks, vs, kd, vd = _data(B, n, H, G, hd, cap, [500, 500], 9)
    k.copy_(ks)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse, st = _call(q, k, k, kd, vd, torch.tensor([500, 129], dtype=torch.int32, device=DEV), None, 0.09, H,
                             stream=s)
    s.synchronize()
    want, wl, bo, bl = R.attention(q, k, k, kd, vd, [500, 129], None, 0.09)
    assert int(st.item()) == 0
    assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0


def test_attention_in_a_cuda_graph_follows_new_lengths():
    B, n, H, G, hd, cap = 2, 4, 2, 4, 64, 700
    q, k, v, kd, vd = _data(B, n, H, G, hd, cap, [700, 700], 10)
    ln = torch.tensor([10, 20], dtype=torch.int32, device=DEV)
    out = torch.zeros((B, n, H * G, hd), dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    _call(q, k, v, kd, vd, ln, None, 0.125, H, out=out, lse=False, status=st, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(q, k, v, kd, vd, ln, None, 0.125, H, out=out, lse=False, status=st, ws=ws)
    for lens in ([700, 1], [0, 333]):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, _, bo, _ = R.attention(q, k, v, kd, vd, lens, None, 0.125)
        assert R.within(out, want, bo) <= 1.0


@pytest.mark.parametrize("B,n,H,G,hd,lens", [
    (200, 1, 1, 4, 64, [(13 * b) % 260 for b in range(200)]),      # more items than shares, some of one tile
    (7, 2, 1, 2, 128, [0, 1, 0, 0, 129, 0, 2]),                    # shares that hold no tile
    (1, 4, 2, 8, 128, [12000]),                                    # 32 rows in many parts
    (1, 3, 1, 3, 64, [30000]),                                     # 9 rows, more parts than a round of loads joins
    (2, 33, 1, 4, 128, [3000, 1]),                                 # two row tiles, the second of one node
])
def test_attention_however_the_work_is_shared(B, n, H, G, hd, lens):
    cap = max(lens) + 1
    q, k, v, kd, vd = _data(B, n, H, G, hd, cap, lens, 11 * n + B)
    scale = hd ** -0.5
    out, lse, st = _call(q, k, v, kd, vd, torch.tensor(lens, dtype=torch.int32, device=DEV), None, scale, H)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want, wl, bo, bl = R.attention(q, k, v, kd, vd, lens, None, scale)
    assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0


def test_attention_many_drafted_tiles_in_a_row_for_two_row_tiles():
    """Every drafted tile is looked through for what is not finite, by one of the two issuing warps for both: a dozen
    of them one after another, many times over, with the same bits every time."""
    n, H, G, hd, lens = 1500, 2, 2, 128, [130, 0]
    q, k, v, kd, vd = _data(2, n, H, G, hd, 140, lens, 12)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse, st = _call(q, k, v, kd, vd, ln, None, 0.09, H)
    for _ in range(30):
        again, lse2, _ = _call(q, k, v, kd, vd, ln, None, 0.09, H, status=st)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    assert int(st.item()) == 0
    want, wl, bo, bl = R.attention(q, k, v, kd, vd, lens, None, 0.09)
    assert R.within(out, want, bo) <= 1.0 and R.within(lse, wl, bl) <= 1.0
