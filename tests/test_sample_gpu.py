"""rf_sample against its definition in 64 bits.

What stays (probabilities > 0, n_kept) has to be equal, the drawn token too unless the two best scores lie within
1e-5 of each other. Bound on a probability w/Z, relatively: w by the SFU, 2^-22, and its argument's last part, 2^-24; Z of
such weights, a sum of at most V/512 terms to a thread one after another and some 20 additions beside them, each
2^-24; a reciprocal and a product, 2^-23 together. A log-probability is off by that much and by 2^-23 of its terms."""
import math

import pytest
import torch

import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(kind, R, V, seed, dtype):
    g = _gen(seed)
    x = torch.empty((R, V), device="cuda").normal_(0.0, 3.0, generator=g)
    if kind == "ranked":                                # weights that fall as a power of their rank
        x = torch.empty((R, V), device="cuda").exponential_(1.0, generator=g).mul_(1.2).add_(x, alpha=0.15)
    elif kind == "flat":                                # all weights within an octave
        x.mul_(0.05)
    elif kind == "equal":
        x.fill_(-2.5)
    elif kind == "steps":                               # thousands of ties
        x = (x * 2).round_() / 2
    elif kind == "far":                                 # a few tokens, and the rest 40 octaves and more below
        x = x * 0.1 - 60.0
        x[:, ::97] += 60.0
    elif kind == "masked":
        x = x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") > 0.02, -math.inf)
    elif kind == "lowest":
        x = x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") > 0.3, torch.finfo(dtype).min)
    elif kind == "huge":                                # distances beyond fp32
        x *= 2e37
    return x.to(dtype)


def _keep(x, T, k, p, mp):
    """(tokens in order, their probabilities) of one row of float64 logits."""
    x = torch.where(torch.isnan(x), -math.inf, x)
    if bool((x == math.inf).any()):
        x = torch.where(x == math.inf, 0.0, -math.inf).double()
    order = torch.argsort(-x, stable=True)
    order = order[:int((x > -math.inf).sum())]
    if len(order) == 0:
        return order, order.double()
    if T == 0.0:
        return order[:1], torch.ones(1, dtype=torch.float64, device=x.device)
    if k > 0:
        order = order[:k]
    away = (x[order] - x[order[0]]) / T
    w = away.exp()
    if p < 1.0:
        before = torch.cat([torch.zeros(1, dtype=torch.float64, device=x.device), w.cumsum(0)[:-1]])
        stay = before < p * w.sum()
        stay[0] = True
        near = (before[1:] / w.sum() - p).abs().min() if len(w) > 1 else 1.0
        assert float(near) > 2.0 ** -36, "an input whose border 64 bits do not decide"
        order, away, w = order[stay], away[stay], w[stay]
    if mp > 0.0:
        stay = away >= math.log(mp)
        order, w = order[stay], w[stay]
    return order, w / w.sum()


def _run(x, T=None, k=None, p=None, mp=None, noise=None, probs=True, draw=True, ld_probs=None):
    R, V = x.shape
    f = lambda v, t: None if v is None else torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    ld_probs = ld_probs or V
    P = torch.full((R, ld_probs), math.nan, device="cuda") if probs else None
    tok, cnt = (torch.full((R,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    lp = torch.full((R,), math.nan, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if noise is None:
        noise = torch.empty((R, V), device="cuda").exponential_(1.0, generator=_gen(R * 31 + V)).clamp_(min=1e-30)
    d = rf.rf_sample_desc(n_rows=R, vocab=V, ld_logits=x.stride(0), ld_noise=V, ld_probs=ld_probs,
                          dtype=rf.RF_BF16 if x.dtype == torch.bfloat16 else rf.RF_F32)
    rf.rf_sample(d, x, f(T, torch.float32), f(k, torch.int32), f(p, torch.float32), f(mp, torch.float32),
                 noise if draw else None, P, tok if draw else None, lp if draw else None, cnt, st)
    torch.cuda.synchronize()
    return P, tok, lp, cnt, int(st.item()), noise


def _check_row(V, x, T, k, p, mp, P, tok, lp, cnt, noise, draw):
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    order, prob = _keep(x.double(), f32(T), k, f32(p), f32(mp))
    assert int(cnt) == len(order)
    if P is not None:
        want = torch.zeros(V, dtype=torch.float64, device="cuda")
        want[order] = prob
        big = want > 2.0 ** -100                        # (weights below 2^-126 are 0)
        assert torch.equal((P[:V] > 0) & big, big) and bool((P[:V][want == 0] == 0).all())
        bound = (2.0 ** -21 + (V / 512 + 32) * U24) * want
        if bool(big.any()):
            assert float(((P[:V].double() - want).abs()[big] / bound[big]).max()) <= 1.0
        assert bool(torch.isnan(P[V:]).all())
    if draw:
        if len(order) == 0:
            assert int(tok) == -1 and float(lp) == -math.inf
            return
        score = prob / noise[order].double()
        best = score.topk(min(2, len(score))).values
        if len(best) == 1 or float(best[0] - best[1]) > 1e-5 * float(best[0]):
            assert int(tok) == int(order[score.argmax()])
        at = (order == int(tok)).nonzero()
        assert len(at) == 1
        ln = float(prob[at[0, 0]].log())
        span = abs(float((x.double()[order[at[0, 0]]] - x.double()[order[0]]) / (T or 1.0)))
        span = (span if math.isfinite(span) else 0.0) + math.log(V + 1.0)
        assert abs(float(lp) - ln) <= 2.0 ** -21 + (V / 512 + 32) * U24 + 2.0 ** -22 * min(span, 200.0)


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (1.3, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.6, 40, 0.95, 0.02), (0.0, 5, 0.5, 0.1),
            (1.0, 1, 1.0, 0.0), (2.0, 1000, 0.99, 0.0), (1.0, 128, 0.5, 0.0), (1.0, 129, 1.0, 0.0), (0.05, 0, 0.999, 0.0),
            (30.0, 0, 0.3, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 20000, 0.9999, 1e-6), (1.0, 7, 1.0, 1.0), (1.0, 0, 1e-9, 0.0)]
KINDS = ["normal", "ranked", "flat", "equal", "steps", "far", "masked", "lowest", "huge"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4099, 32000, 131072])
@pytest.mark.parametrize("kind", KINDS)
def test_sample_matches_its_definition(kind, V, dtype):
    if kind == "huge" and V > 4099:
        pytest.skip("as at smaller vocabularies")
    R = len(SETTINGS)
    x = _logits(kind, R, V, V + len(kind), dtype)
    T, k, p, mp = map(list, zip(*SETTINGS))
    if kind in ("equal", "steps", "lowest", "flat", "huge"):     # borders that fall between equal masses are none of 64 bits'
        p = [min(1.0, q * 1.0000172) if 0.0 < q < 1.0 else q for q in p]
    P, tok, lp, cnt, st, noise = _run(x, T, k, p, mp)
    assert st == 0
    for r in range(R):
        _check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [257, 1030, 5001, 131072])
@pytest.mark.parametrize("kind", ["normal", "steps", "masked", "ranked"])
def test_sample_top_k_from_one_to_more_than_are_listed_at_once(kind, V, dtype):
    k = [1, 2, 16, 17, 64, 65, 127, 200, 255, 256, 257, 300]
    R = len(k)
    x = _logits(kind, R, V, 7 * V + len(kind), dtype)
    if kind == "masked":
        x[4:6, 5:] = -math.inf                          # fewer tokens than top_k
    T, p, mp = [0.9] * R, [1.0, 0.97] * (R // 2), [0.0, 0.0, 1e-3] * (R // 3)
    if kind == "steps":                                 # (as above)
        p = [min(1.0, q * 1.0000172) for q in p]
    P, tok, lp, cnt, st, noise = _run(x, T, k, p, mp)
    assert st == 0
    for r in range(R):
        _check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_borders_among_many_equal_tokens_where_the_last_bin_begins(dtype):
    """2,000 tokens 31.9725 octaves below the first, 3,000 twice as far: runs that end among them."""
    V = 8192
    x = torch.full((3, V), -math.inf, device="cuda", dtype=dtype)
    x[:, 17] = 0.0
    x[:, 100:2100] = -16.0
    x[:, 3000:6000] = -32.0
    T, k, p, mp = [16.0 * math.log2(math.e) / 31.9725] * 3, [1500, 2001, 4500], [1.0] * 3, [0.0] * 3
    P, tok, lp, cnt, st, noise = _run(x, T, k, p, mp)
    for r in range(3):
        _check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("R,V,pad,ldp", [(1, 1 << 20, 0, 0), (3, 100003, 5, 100010), (40, 5001, 1, 5001), (170, 3001, 0, 3004),
                                         (700, 257, 3, 257), (1, 2049, 7, 2050)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_rows_strides_and_clusters(R, V, pad, ldp, dtype):
    """Any stride (rows that start between 16-byte boundaries), one to eight CTAs a row, more rows than SMs."""
    x = _logits("ranked", R, V + pad, R, dtype)[:, :V]
    pick = [SETTINGS[i % len(SETTINGS)] for i in range(R)]
    T, k, p, mp = map(list, zip(*pick))
    P, tok, lp, cnt, st, noise = _run(x, T, k, p, mp, ld_probs=ldp or V)
    assert st == 0
    for r in range(0, R, max(1, R // 24)):
        _check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("V", [70, 32000])
def test_sample_rows_that_leave_nothing_and_values_that_are_not_finite(V):
    x = _logits("normal", 8, V, 3, torch.float32)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 3:60] = math.nan
    x[3, [5, 9, 60]] = math.inf
    x[4, [5, 9, 60]] = math.inf
    x[4, 11] = math.nan
    x[5, 1:] = -math.inf
    x[6, :5], x[6, 5:] = 0.0, -0.0                              # all equal
    x[7] = torch.finfo(torch.float32).min
    for setting in [(1.0, 0, 1.0, 0.0), (0.8, 40, 0.9, 0.01), (0.0, 0, 1.0, 0.0), (1.0, 0, 0.51234, 0.0), (1.0, 2, 1.0, 0.0)]:
        P, tok, lp, cnt, st, noise = _run(x, *([v] * 8 for v in setting))
        assert st == 0
        for r in range(8):
            _check_row(V, x[r], *setting, P[r], tok[r], lp[r], cnt[r], noise[r], True)


def test_sample_settings_out_of_range_are_reported_row_by_row():
    V = 5000
    x = _logits("normal", 9, V, 4, torch.bfloat16)
    T = [1.0, -1.0, math.nan, math.inf, 1e-38, 1.0, 1.0, 1.0, 1.0]
    k = [0, 0, 0, 0, 0, -1, 0, 0, 0]
    p = [1.0, 1.0, 1.0, 1.0, 1.0, 1.0, math.nan, -0.1, 7.0]
    mp = [0.0] * 9
    P, tok, lp, cnt, st, noise = _run(x, T, k, p, mp)
    assert st == rf.RF_ERR_INVALID_ARG
    for r in range(9):
        if r in (0, 8):
            _check_row(V, x[r], 1.0, 0, 1.0, 0.0, P[r], tok[r], lp[r], cnt[r], noise[r], True)
        else:
            assert int(tok[r]) == -1 and int(cnt[r]) == 0 and float(lp[r]) == -math.inf and not bool(P[r].any())
    for bad in (-0.1, 1.5, math.nan):
        _, tok, _, _, st, _ = _run(x[:1], mp=[bad])
        assert st == rf.RF_ERR_INVALID_ARG and int(tok[0]) == -1


def test_sample_without_settings_token_probabilities_or_place_of_their_own():
    R, V = 6, 40001
    x = _logits("ranked", R, V, 5, torch.float32)
    T, k, p, mp = map(list, zip(*(SETTINGS[i] for i in (0, 1, 2, 3, 4, 5))))
    P, tok, lp, cnt, _, noise = _run(x, T, k, p, mp)
    only, *_ = _run(x, T, k, p, mp, draw=False)                  # probabilities alone
    assert torch.equal(only, P)
    none, tok2, lp2, cnt2, _, _ = _run(x, T, k, p, mp, noise=noise, probs=False)
    assert none is None and torch.equal(tok2, tok) and torch.equal(lp2, lp) and torch.equal(cnt2, cnt)
    soft, *_ = _run(x, draw=False)                              # no settings: the softmax
    assert float((soft.double() / torch.softmax(x.double(), 1) - 1).abs().max()) < 2e-5
    y = x.clone()                                               # over the logits
    d = rf.rf_sample_desc(n_rows=R, vocab=V, ld_logits=V, ld_noise=V, ld_probs=V, dtype=rf.RF_F32)
    tok3, lp3 = torch.empty_like(tok), torch.empty_like(lp)
    f = lambda v, t=torch.float32: torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    rf.rf_sample(d, y, f(T), f(k, torch.int32), f(p), f(mp), noise, y, tok3, lp3)
    torch.cuda.synchronize()
    assert torch.equal(y, P) and torch.equal(tok3, tok) and torch.equal(lp3, lp)


def test_sample_reads_the_noise_of_tokens_that_stay_alone():
    V = 32000
    x = _logits("ranked", 3, V, 6, torch.float32)
    s = [(1.0, 20, 1.0, 0.0), (1.0, 0, 0.7, 0.0), (1.0, 0, 1.0, 0.1)]
    T, k, p, mp = map(list, zip(*s))
    P, tok, lp, _, _, noise = _run(x, T, k, p, mp)
    spoiled = torch.where(P > 0, noise, math.nan)
    _, tok2, lp2, *_ = _run(x, T, k, p, mp, noise=spoiled)
    assert torch.equal(tok, tok2) and torch.equal(lp, lp2)


def test_sample_follows_its_distribution():
    """20,000 draws from one row of five tokens that stay: each count within five standard deviations."""
    R, V = 20000, 37
    x = torch.full((V,), -5.0, device="cuda")
    x[[3, 8, 20, 21, 36]] = torch.tensor([1.0, 0.5, 0.0, -0.5, 2.0], device="cuda")
    noise = torch.empty((R, V), device="cuda").exponential_(1.0, generator=_gen(9))
    _, tok, *_ = _run(x.repeat(R, 1), [0.9] * R, [5] * R, noise=noise)
    order, prob = _keep(x.double(), 0.9, 5, 1.0, 0.0)
    for i, q in zip(order.tolist(), prob.tolist()):
        assert abs(int((tok == i).sum()) - R * q) <= 5 * math.sqrt(R * q * (1 - q))
    assert bool(torch.isin(tok.long(), order).all())


def test_sample_in_a_graph_and_on_two_streams():
    R, V = 33, 20003
    x = _logits("ranked", R, V, 11, torch.bfloat16)
    noise = torch.empty((R, V), device="cuda").exponential_(1.0, generator=_gen(12))
    d = rf.rf_sample_desc(n_rows=R, vocab=V, ld_logits=V, ld_noise=V, ld_probs=V, dtype=rf.RF_BF16)
    T, k = torch.full((R,), 0.8, device="cuda"), torch.full((R,), 40, dtype=torch.int32, device="cuda")
    k[::2] = 0
    p = torch.full((R,), 0.9, device="cuda")
    out = [(torch.empty((R, V), device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")) for _ in range(3)]

    def call(i):
        rf.rf_sample(d, x, T, k, p, None, noise, *out[i])

    call(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0)
    x.copy_(_logits("ranked", R, V, 13, torch.bfloat16))
    k.add_(3)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in (1, 2):
        with torch.cuda.stream(streams[i - 1]):
            call(i)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out[0], out[1]):
        assert torch.equal(a, b)
    for a, b in zip(out[0], out[2]):
        assert torch.equal(a, b)


def test_sample_probabilities_are_what_verification_takes():
    """Filtered target and draft probabilities, then a chain whose draft equals the target: every token is accepted."""
    B, n, V = 3, 4, 9000
    g = _gen(21)
    x = torch.empty((B * n, V), device="cuda").normal_(0.0, 2.0, generator=g)
    P, *_ = _run(x, [0.8] * (B * n), [30] * (B * n), [0.9] * (B * n), draw=False)
    target = P.view(B, n, V)
    tokens = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    for i in range(1, n):
        tokens[:, i] = target[:, i - 1].argmax(-1)
    par = torch.tensor([[-1, 0, 1, 2]] * B, dtype=torch.int32, device="cuda")
    ints = lambda: torch.zeros(B, dtype=torch.int32, device="cuda")  # noqa: E731
    path, cnt, nxt = torch.zeros((B, n), dtype=torch.int32, device="cuda"), ints(), ints()
    u = torch.rand((B, n), generator=g, device="cuda") * 0.999
    noise = torch.empty((B, V), device="cuda").exponential_(1.0, generator=g)
    rf.rf_verify_draft(rf.rf_verify_desc(n_seqs=B, n_nodes=n, vocab=V, ld_target=V, ld_draft=V, ld_noise=V), target, target,
                       tokens, par, u, noise, path, cnt, nxt)
    torch.cuda.synchronize()
    assert cnt.tolist() == [n] * B
    for b in range(B):
        assert float(target[b, n - 1, nxt[b]]) > 0
