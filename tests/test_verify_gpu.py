"""rf_verify_draft and rf_commit_draft. The walk's decisions are whole numbers: they have
to equal those of the definition in 64 bits. Decisions that a rounding could turn are
counted by the reference: their margins are kept above 1e-4 (a chain of refusals rounds
each number a few times, 1e-6 at most, and its sums by 1e-5 at most)."""
import numpy as np
import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(B, n, V, seed, with_draft, sharp=3.0, agree=0.8, reach=4, ld=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ld = ld or V
    par = [R.random_parents(n, seed + 31 * b, reach) for b in range(B)]
    logits = torch.randn((B, n, V), generator=g, device=DEV) * sharp
    target = torch.zeros((B, n, ld), device=DEV)
    target[..., :V] = torch.softmax(logits, -1)
    draft = None
    if with_draft:
        draft = torch.zeros((B, n, ld), device=DEV)
        draft[..., :V] = torch.softmax(logits + agree * torch.randn((B, n, V), generator=g, device=DEV), -1)
    src = draft if with_draft else target
    tokens = torch.zeros((B, n), dtype=torch.int32, device=DEV)
    race = torch.empty((B, n, V), device=DEV).exponential_(1.0, generator=g)
    for b in range(B):
        for i in range(1, n):
            tokens[b, i] = (src[b, par[b][i], :V] / race[b, i]).argmax()
    u = torch.rand((B, n), generator=g, device=DEV)
    noise = torch.empty((B, ld), device=DEV).exponential_(1.0, generator=g)
    return par, target, draft, tokens, u, noise


def _run(par, target, draft, tokens, u, noise, V, stream=None):
    B, n = tokens.shape
    ld = target.shape[-1]
    d = rf.rf_verify_desc(n_seqs=B, n_nodes=n, vocab=V, ld_target=ld, ld_draft=ld, ld_noise=noise.shape[-1])
    path = torch.full((B, n), -7, dtype=torch.int32, device=DEV)
    cnt, tok = (torch.full((B,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    rf.rf_verify_draft(d, target, draft, tokens, torch.tensor(par, dtype=torch.int32).cuda(), u, noise, path, cnt, tok,
                       st, stream=stream)
    torch.cuda.synchronize()
    return path.cpu(), cnt.cpu(), tok.cpu(), int(st.item())


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft-probabilities", "outright"])
@pytest.mark.parametrize("B,n,V,reach,ld", [(1, 1, 5, 1, None), (4, 5, 1000, 1, None), (9, 17, 333, 5, 341),
                                           (3, 64, 50257, 8, None), (2, 64, 4096, 64, None), (2, 130, 64, 3, 72), (2, 6, 140001, 6, None)])
def test_verify_walks_like_the_definition(B, n, V, reach, ld, with_draft):
    checked = 0
    for seed in range(4):
        par, target, draft, tokens, u, noise = _inputs(B, n, V, 1000 * seed + n + V, with_draft, reach=reach, ld=ld)
        path, cnt, tok, st = _run(par, target, draft, tokens, u, noise, V)
        assert st == 0
        for b in range(B):
            want, token, near = R.verify(target[b, :, :V], None if draft is None else draft[b, :, :V], tokens[b], par[b],
                                         u[b], noise[b, :V])
            if near < 1e-4:
                continue
            checked += 1
            assert path[b].tolist() == want + [-1] * (n - len(want)) and int(cnt[b]) == len(want)
            assert int(tok[b]) == token
    assert checked >= 2 * B


def test_verify_accepts_all_refuses_all_and_takes_the_lowest_of_equals():
    n, V = 4, 11
    par = [[-1, 0, 1, 2]] * 3
    target = torch.full((3, n, V), 1.0 / 16, device=DEV)       # exact in fp32; argmax ties
    draft = target.clone()
    tokens = torch.tensor([[0, 3, 4, 5]] * 3, dtype=torch.int32, device=DEV)
    noise = torch.ones((3, V), device=DEV)
    u = torch.full((3, n), 0.5, device=DEV)
    target[1, 0, 3] = 0.0                                       # the first child cannot be accepted
    target[2, 2] = 0.0                                          # no mass after node 2: nothing left at all
    path, cnt, tok, st = _run(par, target, draft, tokens, u, noise, V)
    assert st == 0
    assert path.tolist() == [[0, 1, 2, 3], [0, -1, -1, -1], [0, 1, 2, -1]]
    # sequence 1's residual is empty (target <= draft everywhere), so the target row itself decides
    assert tok.tolist() == [0, 0, 0] and cnt.tolist() == [4, 1, 3]


def test_verify_siblings_with_an_empty_residual_keep_the_row():
    """Two refused siblings of which the second would leave nothing: r and Z stay as they were."""
    V = 8
    par = [[-1, 0, 0, 0]]
    target = torch.zeros((1, 4, V), device=DEV)
    draft = torch.zeros((1, 4, V), device=DEV)
    target[0, 0, 2] = 1.0
    draft[0, 0, 2] = 1.0
    target[0, 3, 5] = 1.0
    tokens = torch.tensor([[0, 1, 1, 2]], dtype=torch.int32, device=DEV)
    u = torch.full((1, 4), 0.25, device=DEV)
    noise = torch.ones((1, V), device=DEV)
    path, cnt, tok, st = _run(par, target, draft, tokens, u, noise, V)
    assert st == 0 and path.tolist() == [[0, 3, -1, -1]] and cnt.tolist() == [2] and tok.tolist() == [5]


def test_verify_keeps_the_targets_distribution():
    """Chains of one drafted token over 6 values: the kept first token is distributed as the target's, within five
    standard deviations for 20,000 sequences."""
    B, V = 20000, 6
    g = torch.Generator(device=DEV).manual_seed(5)
    p = torch.tensor([0.4, 0.05, 0.2, 0.0, 0.25, 0.1], device=DEV)
    q = torch.tensor([0.1, 0.3, 0.2, 0.2, 0.15, 0.05], device=DEV)
    target, draft = p.expand(B, 2, V).contiguous(), q.expand(B, 2, V).contiguous()
    tokens = torch.zeros((B, 2), dtype=torch.int32, device=DEV)
    tokens[:, 1] = torch.multinomial(q, B, replacement=True, generator=g).int()
    u = torch.rand((B, 2), generator=g, device=DEV)
    noise = torch.empty((B, V), device=DEV).exponential_(1.0, generator=g)
    path, cnt, tok, st = _run([[-1, 0]] * B, target, draft, tokens, u, noise, V)
    assert st == 0
    first = torch.where(cnt == 2, tokens[:, 1].cpu(), tok).long()
    freq = torch.bincount(first, minlength=V).double() / B
    dev = 5 * (p.cpu().double() * (1 - p.cpu().double()) / B).sqrt()
    assert bool(((freq - p.cpu().double()).abs() <= dev + 1e-12).all())


@pytest.mark.parametrize("what", ["parents", "token-low", "token-high"])
def test_verify_reports_wrong_trees_and_goes_on_with_the_rest(what):
    B, n, V = 3, 5, 40
    par, target, draft, tokens, u, noise = _inputs(B, n, V, 9, True)
    good = _run(par, target, draft, tokens, u, noise, V)
    if what == "parents":
        par[1] = [-1, 0, 3, 1, 2]
    else:
        tokens[1, 2] = -1 if what == "token-low" else V
    path, cnt, tok, st = _run(par, target, draft, tokens, u, noise, V)
    assert st == rf.RF_ERR_INVALID_ARG
    assert path[1].tolist() == [-1] * n and int(cnt[1]) == 0 and int(tok[1]) == -1
    for b in (0, 2):
        assert torch.equal(path[b], good[0][b]) and cnt[b] == good[1][b] and tok[b] == good[2][b]


@pytest.mark.parametrize("L,B,n,H,hd,cap,layout", [(1, 1, 1, 1, 8, 1, "lb"), (3, 4, 9, 2, 64, 30, "lb"),
                                                  (2, 3, 5, 3, 128, 17, "bl"), (2, 2, 6, 2, 40, 12, "rows")])
def test_commit_appends_the_accepted_rows(L, B, n, H, hd, cap, layout):
    """Layers first, sequences first, and rows of all sequences interleaved; the rest of the cache keeps its bits."""
    W = H * hd
    shape = {"lb": (L, B, cap, W + 8), "bl": (B, L, cap, W + 8), "rows": (L, cap, B, W + 8)}[layout]
    k0, v0 = R.randn(shape, 1), R.randn(shape, 2)
    st3 = k0.stride()
    ls, ss, rs = {"lb": (st3[0], st3[1], st3[2]), "bl": (st3[1], st3[0], st3[2]), "rows": (st3[0], st3[2], st3[1])}[layout]
    view = {"lb": lambda x: x, "bl": lambda x: x.transpose(0, 1), "rows": lambda x: x.transpose(1, 2)}[layout]
    kd, vd = R.randn((L, B, n, W), 3), R.randn((L, B, n, W), 4)
    cnt = [min(n, cap, b + 1) for b in range(B)]
    lens = [cap - c if b % 2 == 0 else 0 for b, c in enumerate(cnt)]
    g = torch.Generator().manual_seed(n)
    path = torch.full((B, n), -1, dtype=torch.int32)
    for b in range(B):
        path[b, :cnt[b]] = torch.randperm(n, generator=g)[:cnt[b]].sort().values.int()
    score0 = R.randn((L, B, H, cap), 5, torch.float32)
    pos0 = torch.full((L, B, H, cap), -5, dtype=torch.int32, device=DEV)
    k, v, score, pos = k0.clone(), v0.clone(), score0.clone(), pos0.clone()
    ln, nx = torch.tensor(lens, dtype=torch.int32, device=DEV), torch.arange(B, dtype=torch.int32, device=DEV) * 10 + 40
    nl, nn = ln.clone(), nx.clone()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=rs, seq_stride=ss,
                         layer_stride=ls)
    # lengths are updated in place
    rf.rf_commit_draft(d, n, kd.stride(2), kd.stride(1), kd.stride(0), path.cuda(), torch.tensor(cnt, dtype=torch.int32).cuda(),
                       nl, nn, kd, vd, k, v, score, pos, nl, nn, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    wk, wv, ws, wp = k0.clone(), v0.clone(), score0.clone(), pos0.clone()
    for b in range(B):
        for j in range(cnt[b]):
            view(wk)[:, b, lens[b] + j, :W] = kd[:, b, int(path[b, j])]
            view(wv)[:, b, lens[b] + j, :W] = vd[:, b, int(path[b, j])]
            ws[:, b, :, lens[b] + j] = 0.0
            wp[:, b, :, lens[b] + j] = int(nx[b]) + j
    assert torch.equal(k, wk) and torch.equal(v, wv) and torch.equal(score, ws) and torch.equal(pos, wp)
    assert nl.tolist() == [a + c for a, c in zip(lens, cnt)] and nn.tolist() == [int(x) + c for x, c in zip(nx, cnt)]


@pytest.mark.parametrize("what", ["full", "path", "count", "length"])
def test_commit_refuses_what_does_not_fit_and_goes_on_with_the_rest(what):
    L, B, n, H, hd, cap = 2, 3, 4, 2, 16, 10
    k0 = R.randn((L, B, cap, H * hd), 1)
    k, v = k0.clone(), k0.clone()
    kd = R.randn((L, B, n, H * hd), 3)
    path = torch.tensor([[0, 2, -1, -1]] * B, dtype=torch.int32)
    cnt = torch.full((B,), 2, dtype=torch.int32)
    lens = torch.full((B,), 3, dtype=torch.int32)
    if what == "full":
        lens[1] = 9
    elif what == "path":
        path[1, 1] = 4
    elif what == "count":
        cnt[1] = 5
    else:
        lens[1] = -2
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    nl = torch.zeros(B, dtype=torch.int32, device=DEV)
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=H * hd,
                         seq_stride=cap * H * hd, layer_stride=B * cap * H * hd)
    rf.rf_commit_draft(d, n, kd.stride(2), kd.stride(1), kd.stride(0), path.cuda(), cnt.cuda(), lens.cuda(), None, kd, kd,
                       k, v, None, None, nl, None, st)
    torch.cuda.synchronize()
    assert int(st.item()) == rf.RF_ERR_INVALID_ARG
    assert nl.tolist() == [5, int(lens[1]), 5]
    assert torch.equal(k[:, 1], k0[:, 1]) and torch.equal(v[:, 1], k0[:, 1])
    for b in (0, 2):
        assert torch.equal(k[:, b, 3:5], kd[:, b, [0, 2]])


@pytest.mark.parametrize("where", ["apart", "lens over next_pos", "one array for all", "over n_path", "next_pos over lens"])
def test_commit_reads_its_inputs_before_it_writes_over_them(where):
    """New lengths and positions over any input of their size: every layer still sees what was there before. More
    layers and sequences than the GPU takes at once."""
    L, B, n, H, hd, cap = 60, 100, 3, 1, 8, 40
    k, v = torch.zeros((L, B, cap, H * hd), dtype=torch.bfloat16, device=DEV), torch.zeros((L, B, cap, H * hd),
                                                                                      dtype=torch.bfloat16, device=DEV)
    kd, vd = R.randn((L, B, n, H * hd), 1), R.randn((L, B, n, H * hd), 2)
    pos = torch.full((L, B, H, cap), -5, dtype=torch.int32, device=DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lens, cnt = [b % 30 for b in range(B)], [b % (n + 1) for b in range(B)]
    nxt = lens if where == "one array for all" else [x + 7 for x in lens]
    path = ints([[0, 1, 2]] * B)
    a_len, a_cnt = ints(lens), ints(cnt)
    a_nxt = a_len if where == "one array for all" else ints(nxt)
    nl, nn = {"apart": (ints([0] * B), ints([0] * B)), "lens over next_pos": (a_nxt, None), "one array for all": (a_len, a_len),
              "over n_path": (a_cnt, ints([0] * B)), "next_pos over lens": (None, a_len)}[where]
    d = rf.rf_cache_desc(n_layers=L, n_seqs=B, n_kv_heads=H, head_dim=hd, capacity=cap, row_stride=H * hd,
                         seq_stride=cap * H * hd, layer_stride=B * cap * H * hd)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    rf.rf_commit_draft(d, n, kd.stride(2), kd.stride(1), kd.stride(0), path, a_cnt, a_len, a_nxt, kd, vd, k, v, None, pos,
                       nl, nn, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    wk, wp = torch.zeros_like(k), torch.full_like(pos, -5)
    for b in range(B):
        for j in range(cnt[b]):
            wk[:, b, lens[b] + j] = kd[:, b, j]
            wp[:, b, :, lens[b] + j] = nxt[b] + j
    assert torch.equal(k, wk) and torch.equal(pos, wp)
    if nl is not None:
        assert nl.tolist() == [x + c for x, c in zip(lens, cnt)]
    if nn is not None:
        assert nn.tolist() == [x + c for x, c in zip(nxt, cnt)]


@pytest.mark.parametrize("V", [8, 140001], ids=["registers", "memory"])
@pytest.mark.parametrize("with_draft", [False, True], ids=["outright", "draft-probabilities"])
def test_verify_goes_on_from_the_row_that_an_empty_residual_leaves(V, with_draft):
    """A refusal that would leave nothing is undone; the next refusal works on the row before it, not on nothing."""
    par = [[-1, 0, 0, 0, 3]]
    n = len(par[0])
    target = torch.zeros((1, n, V), device=DEV)
    target[0, 0, 2] = 0.5                       # half of a row: token 2 alone
    target[0, 3, 5] = target[0, 4, 6] = 1.0
    draft = None
    if with_draft:                              # r/Z - q is empty each time: r = 0.5 at token 2 stays, Z = 1
        draft = torch.zeros((1, n, V), device=DEV)
        draft[0, 0, 2] = 1.0
    tokens = torch.tensor([[0, 2, 1, 2, 5]], dtype=torch.int32, device=DEV)
    # outright: token 2 refused (0.9 >= 0.5, nothing is left), token 1 refused (leaves token 2, Z = 0.5), token 2
    # accepted (0.9 0.5 < 0.5); with draft probabilities: 0.9, then q(1) = 0 against r(1) = 0, then 0.4 < 0.5
    u = torch.tensor([[0.0, 0.9, 0.9, 0.4 if with_draft else 0.9, 0.5]], device=DEV)
    noise = torch.ones((1, V), device=DEV)
    want, token, near = R.verify(target[0], None if draft is None else draft[0], tokens[0], par[0], u[0], noise[0])
    assert want == [0, 3, 4] and token == 6
    path, cnt, tok, st = _run(par, target, draft, tokens, u, noise, V)
    assert st == 0 and path.tolist() == [[0, 3, 4, -1, -1]] and cnt.tolist() == [3] and tok.tolist() == [6]


def _quotient_rows(B, seed, orders):
    """float32 (r, c, Z, Q): Z = r + c and Q = r / Z as IEEE rounds them, r <= Z and Q <= r. orders: the powers of two
    below which r lies, in turns."""
    g = np.random.default_rng(seed)
    r = np.ldexp(g.uniform(0.5, 1.0, B).astype(np.float32), np.array(orders)[np.arange(B) % len(orders)]).astype(np.float32)
    r = np.maximum(r, np.float32(1e-44))
    c = np.exp2(g.uniform(0.5, 6.0, B)).astype(np.float32)
    if max(orders) > 20:
        c = c * r
    z = r + c
    return r, c, z, r / z


@pytest.mark.parametrize("orders", [(0, -1, -5), (-90, -99, -100, -101, -110), (-120, -125, -127, -135, -140, -146), (30, 60)],
                         ids=["usual", "small", "denormal", "large"])
@pytest.mark.parametrize("B,V", [(20000, 4), (120, 131080)], ids=["registers", "memory"])
def test_verify_rounds_quotients_as_ieee_does(B, V, orders):
    """Two refusals leave r/Z - q at token 1, where q is the quotient or the number below it: the token is drawn if and
    only if the kernel's quotient is larger than q, and token 2 otherwise."""
    r, c, z, quot = _quotient_rows(B, 7, orders)
    for below in (False, True):
        q = np.nextafter(quot, np.float32(0.0)) if below else quot
        p = q + r
        use = (p - q == r) & (quot > 0)         # what the first refusal leaves is r itself
        assert use.sum() >= B // 4
        target, draft = torch.zeros((B, 3, V)), torch.zeros((B, 3, V))
        target[:, 0, 0], draft[:, 0, 0] = 0.25, 0.5
        target[:, 0, 1], draft[:, 0, 1] = torch.from_numpy(p), torch.from_numpy(q)
        target[:, 0, 2] = torch.from_numpy(c)
        noise = torch.ones((B, V))
        noise[:, 1], noise[:, 2] = 1e-30, 1e30
        u = torch.full((B, 3), 0.99, device=DEV)
        tokens = torch.zeros((B, 3), dtype=torch.int32, device=DEV)
        path, cnt, tok, st = _run([[-1, 0, 0]] * B, target.cuda(), draft.cuda(), tokens, u, noise.cuda(), V)
        assert st == 0 and bool((cnt == 1).all())
        assert np.array_equal(tok.numpy()[use], np.full(use.sum(), 1 if below else 2))


@pytest.mark.parametrize("V", [40, 140001], ids=["registers", "memory"])
def test_verify_divides_by_sums_whose_reciprocal_is_infinite(V):
    """The first refusal leaves 8e-40 in all; the second one's residual is that over itself, less nothing."""
    target, draft = torch.zeros((1, 3, V), device=DEV), torch.zeros((1, 3, V), device=DEV)
    target[0, 0, 0], draft[0, 0, 0] = 0.9, 0.95
    target[0, 0, 20], target[0, 0, 30] = 3e-40, 5e-40
    noise = torch.full((1, V), 1e10, device=DEV)    # under which 5e-40 itself would vanish
    u = torch.full((1, 3), 0.99, device=DEV)
    path, cnt, tok, st = _run([[-1, 0, 0]], target, draft, torch.zeros((1, 3), dtype=torch.int32, device=DEV), u, noise, V)
    want, token, _ = R.verify(target[0], draft[0], [0, 0, 0], [-1, 0, 0], u[0], noise[0])
    assert (want, token) == ([0], 30)
    assert st == 0 and path.tolist() == [[0, -1, -1]] and tok.tolist() == [30]
