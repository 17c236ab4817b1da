"""rf_evict: which rows stay, which move, and that nothing else changes. All of it is
whole numbers and moved bits, so results are compared exactly."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _scores(shape, kind, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = torch.empty(shape, device=DEV).exponential_(1.0, generator=g)
    if kind == "ties":
        s = (s * 3).floor()
    elif kind == "equal":
        s = torch.zeros(shape, device=DEV)
    elif kind == "odd":                       # negative, both zeros, infinities, NaN, denormals
        s = s - 1.0
        pick = torch.randint(0, 9, shape, generator=g, device=DEV)
        for i, x in enumerate((0.0, -0.0, math.inf, -math.inf, math.nan, 1e-42)):
            s = torch.where(pick == i, x, s)
    return s


def _run(L, B, H, hd, cap, keep, sink, recent, lens, kind, inplace, seed=0, pos_kind="perm"):
    W = H * hd
    k0, v0 = R.randn((L, B, cap, W + 8), seed + 1), R.randn((L, B, cap, W + 8), seed + 2)
    score0 = _scores((L, B, H, cap), kind, seed + 3)
    g = torch.Generator(device=DEV).manual_seed(seed + 4)
    pos0 = (torch.rand((L, B, H, cap), generator=g, device=DEV).argsort(-1) if pos_kind == "perm"
            else torch.arange(cap, device=DEV).expand(L, B, H, cap)).int().contiguous()
    k, v = k0.clone(), v0.clone()
    score, pos = score0.clone(), pos0.clone()
    so = score if inplace else torch.full_like(score, -3.0)
    po = pos if inplace else torch.full_like(pos, -3)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    nx = ln + 2
    nl = ln.clone() if inplace else torch.zeros_like(ln)
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=W + 8,
                         seq_stride=cap * (W + 8), layer_stride=B * cap * (W + 8))
    wsb = rf.rf_evict_workspace_bytes(d, keep)
    ws = torch.full((wsb,), 0xA5, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    rf.rf_evict(d, keep, sink, recent, nl if inplace else ln, nx, k, v, score, pos, so, po, nl, st, ws, wsb)
    torch.cuda.synchronize()
    return dict(k0=k0, v0=v0, score0=score0, pos0=pos0, k=k, v=v, so=so, po=po, nl=nl, st=int(st.item()), nx=nx, ws=ws)


def _expect(r, L, B, H, hd, cap, keep, sink, recent, lens, inplace):
    wk, wv = r["k0"].clone(), r["v0"].clone()
    ws = r["score0"].clone() if inplace else torch.full_like(r["score0"], -3.0)
    wp = r["pos0"].clone() if inplace else torch.full_like(r["pos0"], -3)
    sc, ps = r["score0"].cpu().tolist(), r["pos0"].cpu().tolist()
    for l in range(L):
        for b in range(B):
            n = lens[b]
            for h in range(H):
                stay = R.evict_order(sc[l][b][h], ps[l][b][h], n, keep, sink, n + 2 - recent)
                holes, movers = R.evict_moves(stay, n, keep)
                low = torch.tensor([t for t in stay if t < keep], dtype=torch.long, device=DEV)
                ws[l, b, h, low], wp[l, b, h, low] = r["score0"][l, b, h, low], r["pos0"][l, b, h, low]
                if holes:
                    ho, mo = torch.tensor(holes, device=DEV), torch.tensor(movers, device=DEV)
                    c = slice(h * hd, (h + 1) * hd)
                    wk[l, b, ho, c], wv[l, b, ho, c] = r["k0"][l, b, mo, c], r["v0"][l, b, mo, c]
                    ws[l, b, h, ho], wp[l, b, h, ho] = r["score0"][l, b, h, mo], r["pos0"][l, b, h, mo]
    return wk, wv, ws, wp


def _same(a, b):
    t = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(t), b.contiguous().view(t))


@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "in-place"])
@pytest.mark.parametrize("L,B,H,hd,cap,keep,sink,recent,lens,kind", [
    (1, 1, 1, 8, 1, 1, 0, 0, [1], "plain"),
    (1, 2, 2, 64, 40, 1, 0, 0, [40, 0], "plain"),
    (2, 3, 2, 128, 300, 256, 4, 32, [300, 256, 257], "plain"),
    (2, 3, 2, 128, 300, 100, 4, 32, [299, 33, 150], "ties"),
    (1, 2, 3, 64, 1500, 700, 0, 0, [1500, 1033], "equal"),
    (1, 2, 3, 64, 1500, 700, 3, 100, [1499, 1025], "odd"),
    (1, 2, 2, 40, 2100, 33, 50, 10, [2100, 2047], "plain"),     # more sure rows than stay
    (1, 1, 2, 16, 200, 500, 0, 0, [200], "plain"),              # nothing to evict
    (3, 1, 2, 128, 5000, 4990, 4, 256, [5000], "plain"),
])
def test_evict_keeps_moves_and_leaves_alone(L, B, H, hd, cap, keep, sink, recent, lens, kind, inplace):
    r = _run(L, B, H, hd, cap, keep, sink, recent, lens, kind, inplace, seed=cap + keep)
    assert r["st"] == 0 and r["nl"].tolist() == [min(n, keep) for n in lens]
    wk, wv, ws, wp = _expect(r, L, B, H, hd, cap, keep, sink, recent, lens, inplace)
    assert _same(r["k"], wk) and _same(r["v"], wv)
    # entries beyond the new length are not written
    assert _same(r["so"], ws) and torch.equal(r["po"], wp)


def test_evict_long_caches_beyond_shared_memory():
    """More rows than fit in shared memory: ranks are read again from memory."""
    L, B, H, hd, cap, keep = 1, 1, 2, 8, 60000, 20001
    r = _run(L, B, H, hd, cap, keep, 4, 500, [59999], "ties", False, seed=3)
    assert r["st"] == 0
    wk, wv, ws, wp = _expect(r, L, B, H, hd, cap, keep, 4, 500, [59999], False)
    assert _same(r["k"], wk) and _same(r["v"], wv) and _same(r["so"], ws) and torch.equal(r["po"], wp)


@pytest.mark.parametrize("bad", [-1, 101])
def test_evict_reports_a_wrong_length_and_goes_on_with_the_rest(bad):
    lens = [100, bad, 90]
    r = _run(1, 3, 2, 16, 100, 50, 0, 0, lens, "plain", False)
    assert r["st"] == rf.RF_ERR_INVALID_ARG
    assert r["nl"].tolist() == [50, bad, 50]
    assert _same(r["k"][:, 1], r["k0"][:, 1]) and bool((r["po"][:, 1] == -3).all())
    assert not _same(r["k"][:, 0], r["k0"][:, 0])


def test_evict_over_rounds_keeps_the_heavy_rows_and_their_positions():
    """Appending and evicting several times in place: the rows in the cache are always the sinks, the recent ones
    and the heaviest of the rest, each with its own position, whatever order they lie in."""
    L, B, H, hd, cap, keep, sink, recent = 1, 1, 2, 16, 96, 64, 2, 8
    W = H * hd
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=W, seq_stride=cap * W,
                         layer_stride=cap * W)
    wsb = rf.rf_evict_workspace_bytes(d, keep)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    k, v = torch.zeros((cap, W), dtype=torch.bfloat16, device=DEV), torch.zeros((cap, W), dtype=torch.bfloat16, device=DEV)
    score, pos = torch.zeros((H, cap), device=DEV), torch.zeros((H, cap), dtype=torch.int32, device=DEV)
    ln, nx = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(1)
    weight = torch.rand((H, 400), generator=g, device=DEV)
    held = [set() for _ in range(H)]
    p = 0
    for step in (96, 20, 32, 7, 32):
        n = int(ln.item())
        add = min(step, cap - n)
        for j in range(add):
            k[n + j], v[n + j] = float(p + j), -float(p + j)
            score[:, n + j], pos[:, n + j] = weight[:, p + j], p + j
            for h in range(H):
                held[h].add(p + j)
        p += add
        ln.fill_(n + add)
        nx.fill_(p)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        rf.rf_evict(d, keep, sink, recent, ln, nx, k, v, score, pos, score, pos, ln, st, ws, wsb)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(ln.item()) == min(keep, n + add)
        m = int(ln.item())
        for h in range(H):
            sure = {t for t in held[h] if t < sink or t >= p - recent}
            rest = sorted(held[h] - sure, key=lambda t: -float(weight[h, t]))
            held[h] = sure | set(rest[:m - len(sure)])
            assert set(pos[h, :m].tolist()) == held[h]
            assert torch.equal(k[:m, h * hd].float(), pos[h, :m].to(torch.bfloat16).float())
            assert torch.equal(v[:m, h * hd].float(), -pos[h, :m].to(torch.bfloat16).float())
            assert torch.equal(score[h, :m], weight[h][pos[h, :m].long()])


@pytest.mark.parametrize("kind", ["plain", "ties"])
@pytest.mark.parametrize("cap,keep", [(20, 19), (640, 513), (641, 513), (642, 513), (4224, 4096), (9000, 8901)])
def test_evict_gives_the_same_wherever_lengths_and_scores_go(cap, keep, kind):
    """New lengths over the old ones or apart, scores in place or apart: the same rows move, bit for bit."""
    L, B, H, hd, W = 2, 2, 2, 16, 32
    lens = [cap, (cap + keep) // 2]
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=W, seq_stride=cap * W,
                         layer_stride=B * cap * W)
    wsb = rf.rf_evict_workspace_bytes(d, keep)
    results = []
    for lens_apart in (False, True):
        for scores_apart in (False, True):
            k, v = R.randn((L, B, cap, W), 1), R.randn((L, B, cap, W), 2)
            score = _scores((L, B, H, cap), kind, 3)
            pos = torch.arange(cap, dtype=torch.int32, device=DEV).expand(L, B, H, cap).contiguous()
            so, po = (score.clone(), pos.clone()) if scores_apart else (score, pos)
            ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
            nx, nl = ln.clone(), torch.zeros_like(ln) if lens_apart else ln
            ws = torch.full((wsb,), 0xA5, dtype=torch.uint8, device=DEV)
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            rf.rf_evict(d, keep, 4, 8, ln, nx, k, v, score, pos, so, po, nl, st, ws, wsb)
            torch.cuda.synchronize()
            assert int(st.item()) == 0 and nl.tolist() == [min(n, keep) for n in lens]
            results.append((k, v, so[..., :keep], po[..., :keep]))
    for r in results[1:]:
        assert all(_same(x, y) for x, y in zip(r, results[0]))


@pytest.mark.parametrize("cap,keep", [(100, 64), (300, 100)])
def test_evict_writes_lengths_over_the_next_positions(cap, keep):
    """new_lens may be next_pos. Thousands of heads of one sequence, so that some are selected long after the first: all
    read the position that was there before the call. (36 rows can move, which takes one launch, and 100, which takes
    two.)"""
    L, B, H, hd = 500, 1, 8, 8
    W = H * hd
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=W, seq_stride=cap * W,
                         layer_stride=cap * W)
    wsb = rf.rf_evict_workspace_bytes(d, keep)
    results = []
    for over in (False, True):
        k, v = R.randn((L, B, cap, W), 1), R.randn((L, B, cap, W), 2)
        score = _scores((L, B, H, cap), "plain", 3)
        pos = torch.arange(cap, dtype=torch.int32, device=DEV).flip(0).expand(L, B, H, cap).contiguous()
        ln, nx = torch.full((B,), cap, dtype=torch.int32, device=DEV), torch.full((B,), cap, dtype=torch.int32, device=DEV)
        nl = nx if over else torch.zeros_like(ln)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = torch.full((wsb,), 0xA5, dtype=torch.uint8, device=DEV)
        rf.rf_evict(d, keep, 2, 20, ln, nx, k, v, score, pos, score, pos, nl, st, ws, wsb)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and nl.tolist() == [keep] and ln.tolist() == [cap]
        assert bool(((pos[..., :keep] >= cap - 20).sum(-1) == 20).all())      # the newest twenty of every head
        results.append((k, v, score[..., :keep], pos[..., :keep]))
    assert all(_same(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("inplace", [False, True], ids=["apart", "in-place"])
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("cap,keep", [(17408, 5000), (17409, 5000), (17409, 17300), (32768, 8192), (32768, 32700),
                                      (49152, 100), (49152, 49152), (49153, 20000), (49153, 49050)])
def test_evict_of_long_caches(cap, keep, kind, inplace):
    """Either side of the capacities at which ranks leave registers and shared memory, with more and with fewer moves
    than one launch makes (the latter where the new lengths lie apart), whole and ragged."""
    B, H, hd, sink, recent = 2, 1, 8, 4, 300
    lens = [cap, max(1, cap - 77)]
    r = _run(1, B, H, hd, cap, keep, sink, recent, lens, kind, inplace, seed=keep)
    assert r["st"] == 0 and r["nl"].tolist() == [min(n, keep) for n in lens]
    wk, wv, ws, wp = _expect(r, 1, B, H, hd, cap, keep, sink, recent, lens, inplace)
    assert _same(r["k"], wk) and _same(r["v"], wv)
    assert _same(r["so"], ws) and torch.equal(r["po"], wp)
