"""rf_attn_weights against its definition in 64 bits (bounds: decoderef.weights), and the
whole decoding step: attention's statistics give weights that add up to one per query."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _desc(q, k, n, H, scale):
    B, _, Hq, hd = q.shape
    return rf.rf_attn_desc(n_seqs=B, n_q_heads=Hq, n_kv_heads=H, head_dim=hd, n_nodes=n, capacity=k.shape[1],
                           q_row_stride=q.stride(1), q_seq_stride=q.stride(0), draft_row_stride=H * hd,
                           draft_seq_stride=n * H * hd, cache_row_stride=k.stride(1), cache_seq_stride=k.stride(0),
                           out_row_stride=Hq * hd, out_seq_stride=n * Hq * hd, scale=scale)


def _call(q, lse, path, cnt, k, lens, decay, score, out, scale):
    B, n, Hq, hd = q.shape
    d = _desc(q, k, n, k.shape[2], scale)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(rf.rf_attn_weights_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    rf.rf_attn_weights(d, q, lse, path, cnt, k, lens, decay, score, out, st, ws, ws.numel())
    torch.cuda.synchronize()
    return int(st.item())


def _stats(q, k, lens, paths, scale, H):
    """lse of each path node over the rows it sees (others arbitrary)."""
    B, n, Hq, hd = q.shape
    G = Hq // H
    lse = R.randn((B, n, Hq), 99, torch.float32)
    for b in range(B):
        for j, node in enumerate(paths[b]):
            last = lens[b] - len(paths[b]) + j
            for a in range(Hq):
                s = k[b, :last + 1, a // G].double() @ q[b, node, a].double() * scale
                lse[b, node, a] = torch.logsumexp(s, 0).float()
    return lse


@pytest.mark.parametrize("B,n,H,G,hd,lens,take,decay", [
    (1, 1, 1, 1, 64, [1], [1], 1.0),
    (1, 1, 2, 5, 128, [129], [1], 0.5),
    (3, 9, 2, 4, 128, [300, 1, 128], [4, 1, 9], 0.9),
    (2, 16, 2, 8, 64, [700, 255], None, 1.0),
    (2, 64, 1, 10, 128, [1000, 64], None, 0.0),          # 640 queries: three steps
    (1, 70, 1, 10, 128, [513], None, 0.7),               # more than one launch
    (1, 100, 2, 16, 64, [260], None, 1.0),               # 1,600 queries of 64 channels
    (5, 6, 3, 3, 64, [0, 17, 640, 2, 129], [0, 3, 6, 2, 1], 1.0),
    (1, 3, 1, 128, 128, [400], [2], 1.0),
    (1, 2, 1, 1, 128, [20000], [2], 1.0),                # many shares of one head
    (33, 4, 1, 2, 64, [(29 * b) % 300 + 4 for b in range(33)], [b % 5 for b in range(33)], 0.25),
])
def test_weights_match_their_definition(B, n, H, G, hd, lens, take, decay):
    take = take or [n] * B
    lens = [max(a, c) for a, c in zip(lens, take)]
    cap = max(lens) + 5
    scale = hd ** -0.5
    q, k = R.randn((B, n, H * G, hd), 1, std=2.0), R.randn((B, cap, H, hd), 2)
    g = torch.Generator().manual_seed(n)
    paths = [sorted(torch.randperm(n, generator=g)[:c].tolist()) for c in take]
    given = [c for c in take] != [n] * B
    path = torch.full((B, n), -1, dtype=torch.int32)
    for b in range(B):
        path[b, :take[b]] = torch.tensor(paths[b], dtype=torch.int32)
    lse = _stats(q, k, lens, paths, scale, H)
    for b in range(B):
        k[b, lens[b]:] = math.nan
        for i in set(range(n)) - set(paths[b]):
            q[b, i], lse[b, i] = math.nan, math.nan
    score = torch.rand((B, H, cap), device=DEV)
    out = torch.full_like(score, math.nan)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    args = (path.cuda(), torch.tensor(take, dtype=torch.int32, device=DEV)) if given else (None, None)
    assert _call(q, lse, *args, k, ln, decay, score if decay else None, out, scale) == 0
    want, bound = R.weights(q, lse, k, lens, paths, decay, score, scale)
    assert R.within(out, want, bound) <= 1.0                       # NaN beyond a length: not written
    same = score.clone()
    assert _call(q, lse, *args, k, ln, decay, same, same, scale) == 0   # in place, the same bits
    for b in range(B):
        assert torch.equal(same[b, :, :lens[b]], out[b, :, :lens[b]])
        assert torch.equal(same[b, :, lens[b]:], score[b, :, lens[b]:])


def test_weights_leave_out_queries_that_see_nothing():
    q, k = R.randn((1, 4, 2, 64), 1), R.randn((1, 50, 1, 64), 2)
    lse = _stats(q, k, [50], [[0, 1, 2, 3]], 0.1, 1)
    lse[0, 2], q[0, 2] = -math.inf, math.nan
    score, out = torch.zeros((1, 1, 50), device=DEV), torch.zeros((1, 1, 50), device=DEV)
    ln = torch.tensor([50], dtype=torch.int32, device=DEV)
    assert _call(q, lse, None, None, k, ln, 1.0, score, out, 0.1) == 0
    want, bound = R.weights(q, lse, k, [50], [[0, 1, 2, 3]], 1.0, score, 0.1)
    assert R.within(out, want, bound) <= 1.0


@pytest.mark.parametrize("what", ["length", "count", "path-low", "path-high", "more-than-rows"])
def test_weights_report_what_is_out_of_range_and_go_on_with_the_rest(what):
    B, n, H, hd = 3, 4, 2, 64
    q, k = R.randn((B, n, 4, hd), 1), R.randn((B, 100, H, hd), 2)
    lens, cnt = [100, 90, 50], [2, 2, 2]
    path = torch.tensor([[0, 2, -1, -1]] * B, dtype=torch.int32)
    lse = _stats(q, k, lens, [[0, 2]] * B, 0.1, H)
    if what == "length":
        lens[1] = 101
    elif what == "count":
        cnt[1] = 5
    elif what == "path-low":
        path[1, 1] = -1
    elif what == "path-high":
        path[1, 0] = 4
    else:
        lens[1] = 1
    score, out = torch.ones((B, H, 100), device=DEV), torch.full((B, H, 100), math.nan, device=DEV)
    st = _call(q, lse, path.cuda(), torch.tensor(cnt, dtype=torch.int32, device=DEV), k,
               torch.tensor(lens, dtype=torch.int32, device=DEV), 1.0, score, out, 0.1)
    assert st == rf.RF_ERR_INVALID_ARG and bool(torch.isnan(out[1]).all())
    for b in (0, 2):
        want, bound = R.weights(q[b:b + 1], lse[b:b + 1], k[b:b + 1], [lens[b]], [[0, 2]], 1.0, score[b:b + 1], 0.1)
        assert R.within(out[b:b + 1], want, bound) <= 1.0


@pytest.mark.parametrize("hd,G,n,m", [(128, 4, 5, 777), (64, 3, 70, 300)])
def test_attention_then_weights_add_up_to_one_a_query(hd, G, n, m):
    """Rows in order behind m cached ones: attention's lse, then the rows join the cache, then their weights: a KV
    head's weights add up to its number of queries."""
    B, H, cap, scale = 2, 2, m + n + 3, 0.09
    q, k, v = R.randn((B, n, H * G, hd), 1, std=2.0), R.randn((B, cap, H, hd), 2), R.randn((B, cap, H, hd), 3)
    kd, vd = R.randn((B, n, H, hd), 4), R.randn((B, n, H, hd), 5)
    lens = torch.tensor([m, m // 2], dtype=torch.int32, device=DEV)
    d = _desc(q, k, n, H, scale)
    out = torch.empty((B, n, H * G, hd), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((B, n, H * G), device=DEV)
    ws = torch.empty(rf.rf_attn_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    rf.rf_tree_attention(d, q, k, v, lens, kd, vd, None, out, lse, None, ws, ws.numel())
    for b in range(B):
        x = int(lens[b])
        k[b, x:x + n] = kd[b]
    score = torch.zeros((B, H, cap), device=DEV)
    assert _call(q, lse, None, None, k, lens + n, 0.0, None, score, scale) == 0
    total = score.double().sum(-1)
    # each weight is off by 2 eps (both scores) relatively, eps = hd 2^-22 scale sum |q||k| < hd^2 2^-22 x 0.09 x 40
    assert float((total / (n * G) - 1).abs().max()) <= 2 * hd * hd * 2.0 ** -22 * 0.09 * 40


@pytest.mark.parametrize("n,G,hd,m", [(64, 10, 128, 700), (70, 10, 128, 300), (257, 1, 64, 600), (256, 2, 64, 257), (3, 128, 64, 40)])
def test_weights_of_all_nodes_equal_those_along_the_path_of_all_nodes(n, G, hd, m):
    """All nodes in order, given as such or as a path: the same bits. Queries are part of wider rows, the first
    sequence shorter than the other; one query sees nothing and holds NaN."""
    B, H, scale = 2, 2, hd ** -0.5
    lens = [n, max(m, n)]
    wide = R.randn((B, n, H * G + 3, hd), 1, std=2.0)
    q, k = wide[:, :, 1:1 + H * G], R.randn((B, max(lens) + 2, H, hd), 2)
    paths = [list(range(n))] * B
    lse = _stats(q, k, lens, paths, scale, H)
    q[1, n // 2, G - 1], lse[1, n // 2, G - 1] = math.nan, -math.inf
    for b in range(B):
        k[b, lens[b]:] = math.nan
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    path = torch.arange(n, dtype=torch.int32, device=DEV).expand(B, n).contiguous()
    cnt = torch.full((B,), n, dtype=torch.int32, device=DEV)
    score = torch.rand((B, H, k.shape[1]), device=DEV)
    out, along = torch.full_like(score, math.nan), torch.full_like(score, math.nan)
    assert _call(q, lse, None, None, k, ln, 0.5, score, out, scale) == 0
    assert _call(q, lse, path, cnt, k, ln, 0.5, score, along, scale) == 0
    assert torch.equal(out.view(torch.int32), along.view(torch.int32))
    want, bound = R.weights(q, lse, k, lens, paths, 0.5, score, scale)
    assert R.within(out, want, bound) <= 1.0


@pytest.mark.parametrize("B,n,H,G,hd,m,take", [
    (1, 7, 2, 4, 128, 400, 7),         # 28 queries in 32 columns
    (2, 9, 1, 3, 64, 300, 5),          # 15 in 16, two sequences
    (1, 64, 1, 10, 128, 300, 64),      # 640 in 672, three steps
    (1, 16, 1, 16, 64, 500, 16),       # 256: no column is spare but that of a query that sees nothing
])
def test_weights_of_keys_with_infinities_are_those_of_the_queries_alone(B, n, H, G, hd, m, take):
    """A key with an infinity whose product with every query is -inf receives nothing: spare columns, and the query that
    sees nothing, do not make it NaN. A key that is NaN makes its own sum NaN and no other."""
    q = R.randn((B, n, H * G, hd), 1)
    q[..., 3] = -q[..., 3].abs() - 0.125
    k = R.randn((B, m, H, hd), 2)
    paths = [list(range(n - take, n)) for _ in range(B)]
    path = torch.full((B, n), -1, dtype=torch.int32)
    path[:, :take] = torch.arange(n - take, n)
    args = (None, None) if take == n else (path.cuda(), torch.full((B,), take, dtype=torch.int32, device=DEV))
    lse = _stats(q, k, [m] * B, paths, 0.1, H)
    lse[:, n - 2, 0] = -math.inf
    score = torch.rand((B, H, m), device=DEV)
    ln = torch.full((B,), m, dtype=torch.int32, device=DEV)
    plain, out = torch.full_like(score, -3.0), torch.full_like(score, -3.0)
    assert _call(q, lse, *args, k, ln, 0.5, score, plain, 0.1) == 0
    assert bool(torch.isfinite(plain).all())
    odd, bad = [0, 50, 127, 130, m - take, m - 1], 77
    k[:, odd, :, 3] = math.inf
    k[:, bad] = math.nan
    assert _call(q, lse, *args, k, ln, 0.5, score, out, 0.1) == 0
    assert torch.equal(out[..., odd], score[..., odd] * 0.5)
    assert bool(torch.isnan(out[..., bad]).all())
    rest = [t for t in range(m) if t not in odd + [bad]]
    assert R.within(out[..., rest], plain[..., rest].double(), 8 * take * G * R.U24 * plain[..., rest].double() + 1e-30) <= 1.0
