"""Workloads of the operators of a batched decoding step over one filled prompt: what each
one computes, in a plain form and through the library.

A prompt is filled once and many sequences continue it. At every step their queries and
keys are normalised head by head and rotated in one pass (norm_rope; its gradient trains
such a model), attend to the shared prompt, to their own rows and to their drafted rows
(prefix), and the logits become tokens, or the probabilities that drafts are verified
against, by temperature, top-k, top-p and min-p (sample).

``own = False`` computes the operators from elementary torch operations in 32 bits (64
where a border decides: angles, cumulative masses); ``own = True`` calls the library.
``exact`` computes them in 64 bits, apart from both. Head counts, head sizes, lengths and
vocabularies are those of this repository's synthetic deployments and decoding workloads
(8 KV heads of 128 under 32 or 40 query heads, 2 under 20, prompts up to 32,768 rows,
32,000 and 131,072 tokens) or generic.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
_SCALING = {"none": 0, "base": 2, "wavelength": 3}


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # One token of each of 8 sequences: queries and keys of a fused projection row, given positions. Latency.
        dict(name="norm rope step", op="norm_rope", rows=8, q_heads=40, k_heads=8, spare=8, hd=128, rot=128,
             layout="half", dtype="bf16", backward=False, given=True, scaling="wavelength", theta=5.0e5, offset=20000),
        # A whole prompt, as the fill's exact rows run it.
        dict(name="norm rope prompt", op="norm_rope", rows=32768, q_heads=40, k_heads=8, spare=8, hd=128, rot=128,
             layout="half", dtype="bf16", backward=False, given=False, scaling="base", theta=1.0e6, offset=0),
        # Training: gradients of the rows and of both gains, odd row count.
        dict(name="norm rope gradient", op="norm_rope", rows=8191, q_heads=32, k_heads=8, spare=8, hd=128, rot=128,
             layout="half", dtype="bf16", backward=True, given=False, scaling="none", theta=1.0e6, offset=0),
        # The same in 32 bits, interleaved pairs, part of each head turning.
        dict(name="norm rope gradient f32", op="norm_rope", rows=2047, q_heads=20, k_heads=2, spare=0, hd=128, rot=96,
             layout="interleaved", dtype="f32", backward=True, given=True, scaling="none", theta=1.0e4, offset=513),
        # Four answers to one full-length prompt, a token each: the prompt's bytes.
        dict(name="prefix few", op="prefix", seqs=4, nodes=1, branch=1, kv=8, group=5, hd=128, prefix=32767, length=200,
             cap=256),
        # A batch of 64 over a shared prompt, a token each, with up to 1,024 rows of their own.
        dict(name="prefix batch", op="prefix", seqs=64, nodes=1, branch=1, kv=8, group=4, hd=128, prefix=16384,
             length=1024, cap=1040),
        # Drafted trees of 64 nodes for 16 sequences over a long shared prompt: matrix products.
        dict(name="prefix trees", op="prefix", seqs=16, nodes=64, branch=4, kv=8, group=4, hd=128, prefix=28672,
             length=300, cap=384),
        # Narrow heads, three rows in order for each of 100 sequences, own parts as long as the prompt.
        dict(name="prefix narrow", op="prefix", seqs=100, nodes=3, branch=0, kv=2, group=10, hd=64, prefix=4099,
             length=4000, cap=4003),
        # One token of one sequence, every filter on. Latency.
        dict(name="sample one", op="sample", rows=1, vocab=32000, dtype="f32", filters="all", probs=False),
        # A batch's next tokens from bf16 logits, nucleus sampling: ties among rounded logits.
        dict(name="sample batch", op="sample", rows=64, vocab=131072, dtype="bf16", filters="top_p", probs=False),
        # Target probabilities of drafted trees (16 sequences of 16 nodes), every filter on.
        dict(name="sample probabilities", op="sample", rows=256, vocab=131072, dtype="f32", filters="all", probs=True),
        # Temperature alone, odd vocabulary: every token stays in the race.
        dict(name="sample unfiltered", op="sample", rows=48, vocab=100003, dtype="f32", filters="none", probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "prefix", "sample"])
    if op == "norm_rope":
        hd, kv = rng.choice([64, 96, 128, 256]), rng.choice([1, 2, 8])
        group = rng.choice([1, 2, 4, 5])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        top = 32768 * 48 * 128 * 2 // ((kv * group + kv) * hd * (2 if dtype == "bf16" else 4))
        backward = rng.random() < 0.5
        return dict(op=op, rows=_log(rng, 1, min(32768, top * 2 // 3 if backward else top)), q_heads=kv * group, k_heads=kv,
                    spare=rng.choice([0, kv]), hd=hd, rot=rng.choice([hd, hd // 2, hd // 4 * 3, 20]),
                    layout=rng.choice(["half", "interleaved"]), dtype=dtype, backward=backward,
                    given=rng.random() < 0.5, scaling=rng.choice(sorted(_SCALING)), theta=rng.choice([1.0e4, 5.0e5, 1.0e6]),
                    offset=rng.randint(0, 30000))
    if op == "prefix":
        kv, hd = rng.choice([1, 2, 8]), rng.choice([64, 128])
        group = rng.choice([1, 2, 4, 5, 10]) if kv < 8 else rng.choice([1, 2, 4, 5])
        seqs = _log(rng, 1, 64)
        nodes = _log(rng, 1, min(16, 512 // seqs))
        length = _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, nodes=nodes, branch=rng.randint(0, 4), kv=kv, group=group, hd=hd,
                    prefix=_log(rng, 1, 28672), length=length, cap=length + rng.randint(0, 50))
    vocab = _log(rng, 1000, 131072)
    return dict(op=op, rows=_log(rng, 1, 256), vocab=vocab, dtype=rng.choice(["f32", "bf16"]),
                filters=rng.choice(["all", "top_p", "top_k", "min_p", "none"]), probs=rng.random() < 0.5)


def _lengths(case):
    """Ragged lengths of the sequences' own rows, the first the longest; a new sequence has none yet."""
    top = case["length"]
    return [max(0, int(top * (1.0 - (0.61803399 * b) % 1.0))) for b in range(case["seqs"])]


# ------------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFF)
    return g


def _randn(shape, g, dtype=BF16, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tree(case, seed):
    """Which drafted nodes a node sees (itself and its ancestors): bool [B][n][n], and as mask words."""
    B, n, branch = case["seqs"], case["nodes"], case["branch"]
    g = torch.Generator()
    g.manual_seed(int(seed) * 7919 + 17)
    jitter = torch.randint(0, branch, (B, n), generator=g).tolist()
    seen = torch.zeros((B, n, n), dtype=torch.bool)
    for b in range(B):
        for i in range(n):
            if i:
                seen[b, i] = seen[b, min(i - 1, max(0, (i - 1 + jitter[b][i]) // branch))]
            seen[b, i, i] = True
    w = (n + 63) // 64
    bits = torch.zeros((B, n, w * 64), dtype=torch.int64)
    bits[:, :, :n] = seen.long()
    return seen.cuda(), (bits.view(B, n, w, 64) << torch.arange(64)).sum(-1).cuda()


def prepare(case, seed):
    g = _gen(seed, sum(ord(c) for c in case["op"]))
    s = {"case": case}
    if case["op"] == "norm_rope":
        dtype = BF16 if case["dtype"] == "bf16" else F32
        rows, heads, hd = case["rows"], case["q_heads"] + case["k_heads"], case["hd"]
        # projections of unequal rows, gains around one
        s["x"] = _randn((rows, (heads + case["spare"]) * hd), g, dtype)
        s["x"] *= torch.rand((rows, 1), generator=g, device="cuda").add_(0.25).to(dtype)
        s["q_gain"] = _randn((hd,), g, F32, 0.2).add_(1.0).to(dtype)
        s["k_gain"] = _randn((hd,), g, F32, 0.2).add_(1.0).to(dtype)
        s["positions"] = None
        if case["given"]:
            s["positions"] = torch.randint(0, 32768, (rows,), generator=g, device="cuda").to(torch.int32)
        if case["backward"]:
            s["dy"] = _randn((rows, heads * hd), g, dtype)
            s["dx"] = torch.zeros_like(s["x"])
            s["dq_gain"], s["dk_gain"] = (torch.zeros((hd,), dtype=F32, device="cuda") for _ in range(2))
        else:
            s["y"] = torch.empty((rows, heads * hd), dtype=dtype, device="cuda")
    elif case["op"] == "prefix":
        B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
        # queries, keys and values of the drafted rows come from one projection
        fused = _randn((B, n, (G * H + 2 * H), hd), g)
        fused[:, :, :G * H] *= 2.0
        s["q"], s["kd"], s["vd"] = fused[:, :, :G * H], fused[:, :, G * H:G * H + H], fused[:, :, G * H + H:]
        s["kp"], s["vp"] = _randn((case["prefix"], H, hd), g), _randn((case["prefix"], H, hd), g)
        s["k"], s["v"] = _randn((B, case["cap"], H, hd), g), _randn((B, case["cap"], H, hd), g)
        s["prefix_len"], s["lens"] = _ints([case["prefix"]]), _ints(_lengths(case))
        s["seen"], s["mask"] = _tree(case, seed) if case["branch"] else (None, None)
        s["out"] = torch.empty((B, n, G * H, hd), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((B, n, G * H), dtype=F32, device="cuda")
    else:
        R, V = case["rows"], case["vocab"]
        # the r-th largest of V exponentials is about ln(V/r): token frequencies that fall as a power of their rank
        x = torch.empty((R, V), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        x.mul_(1.2).add_(_randn((R, V), g, F32, 0.5))
        # every fifth row is held to a grammar that allows a tenth of the vocabulary
        x[4::5] = x[4::5].masked_fill_(torch.rand(x[4::5].shape, generator=g, device="cuda") > 0.1, -math.inf)
        s["logits"] = x.to(BF16 if case["dtype"] == "bf16" else F32)
        s["noise"] = torch.empty((R, V), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        i = torch.arange(R, device="cuda")

        def cycle(values, kind, dtype):
            if case["filters"] not in ("all", kind):
                return None
            return torch.tensor(values, dtype=dtype, device="cuda")[(i + seed) % len(values)].contiguous()

        # requests of their own settings; one in seven is greedy
        s["temperature"] = torch.tensor([1.0, 0.7, 0.6, 1.0, 1.3, 0.8, 0.0], device="cuda")[i % 7].contiguous()
        s["top_k"] = cycle([50, 0, 20, 1000], "top_k", torch.int32)
        s["top_p"] = cycle([0.95, 0.9, 0.8], "top_p", F32)
        s["min_p"] = cycle([0.0, 0.05, 0.0, 0.01, 0.001], "min_p", F32)
        s["probs"] = torch.empty((R, V), dtype=F32, device="cuda") if case["probs"] else None
        s["token"], s["kept"] = _ints([0] * R), _ints([0] * R)
        s["logprob"] = torch.zeros(R, dtype=F32, device="cuda")
    return s


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work of a pass
def work(case):
    if case["op"] == "norm_rope":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * (case["q_heads"] + case["k_heads"]) * case["hd"]
        extra = 2 * case["hd"] * (size + (4 if case["backward"] else 0)) + (4 * case["rows"] if case["given"] else 0)
        return {"bytes": (3 if case["backward"] else 2) * n * size + extra, "flops": (14 if case["backward"] else 7) * n}
    if case["op"] == "prefix":
        B, n, H, G, hd, P = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd", "prefix"))
        rows = sum(_lengths(case))
        among = n * (n + 1) // 2 if not case["branch"] else n * max(1, n.bit_length())
        mask = B * n * ((n + 63) // 64) * 8 if case["branch"] else 0
        return {"bytes": 4 * B * n * G * H * hd + 4 * H * hd * (P + rows + B * n) + 4 * B * n * G * H + mask,
                "flops": 4 * G * H * hd * (B * n * P + n * rows + B * among)}
    n = case["rows"] * case["vocab"]
    size = 2 if case["dtype"] == "bf16" else 4
    every = 4 * n if case["filters"] == "none" else 0  # noise of tokens that are filtered out decides nothing
    return {"bytes": n * size + every + (4 * n if case["probs"] else 0) + 20 * case["rows"], "flops": 4 * n}


# -------------------------------------------------------------------- plain forms
_FACTOR, _ORIGINAL, _LOW, _HIGH, _EPS = 4.0, 8192.0, 1.0, 4.0, 1.0e-5


def _frequencies(case):
    """Angular frequency of each rotated pair, 64 bits (a table that a program keeps)."""
    r, theta = case["rot"], case["theta"]
    i = torch.arange(r // 2, dtype=F64, device="cuda")
    if case["scaling"] == "base":
        theta = theta * _FACTOR ** (r / (r - 2.0))
    f = theta ** (-2.0 * i / r)
    if case["scaling"] == "wavelength":
        t = ((_ORIGINAL * f / (2.0 * math.pi) - _LOW) / (_HIGH - _LOW)).clamp(0.0, 1.0)
        return f * (t + (1.0 - t) / _FACTOR)
    return f


def _cos_sin(s):
    """Angles in 64 bits: one of 32 is off by 2e-3 at row 32768."""
    case = s["case"]
    p = s["positions"] if case["given"] else case["offset"] + torch.arange(case["rows"], device="cuda")
    angle = p.double()[:, None] * _frequencies(case)
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _turned(x, c, s, case):
    """x [rows][heads][hd]; s negated gives the transpose."""
    r, y = case["rot"], x.clone()
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    return y


def _plain_norm_rope(s):
    case = s["case"]
    Hq, Hk, hd = case["q_heads"], case["k_heads"], case["hd"]
    w = (Hq + Hk) * hd
    x = s["x"][:, :w].float().view(-1, Hq + Hk, hd)
    gain = torch.cat([s["q_gain"].float().expand(Hq, hd), s["k_gain"].float().expand(Hk, hd)])
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    c, t = _cos_sin(s)
    if not case["backward"]:
        s["y"].copy_(_turned(x * r * gain, c, t, case).view_as(s["y"]))
        return {"y": s["y"]}
    u = _turned(s["dy"].float().view(-1, Hq + Hk, hd), c, -t, case)
    dg = (u * x * r).sum(0)
    u *= gain
    s["dx"][:, :w] = (r * (u - x * (r * r * (u * x).mean(-1, keepdim=True)))).view(-1, w).to(s["dx"].dtype)
    s["dq_gain"].copy_(dg[:Hq].sum(0))
    s["dk_gain"].copy_(dg[Hq:].sum(0))
    return {k: s[k] for k in ("dx", "dq_gain", "dk_gain")}


def _plain_prefix(s):
    case = s["case"]
    B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
    cap = max(1, case["length"])  # the longest sequence
    q = s["q"].float().view(B, n, H, G, hd) * hd ** -0.5
    # the prompt, all sequences at once
    shared = q.permute(2, 0, 1, 3, 4).reshape(H, B * n * G, hd) @ s["kp"].float().permute(1, 2, 0)
    top = shared.amax(-1, keepdim=True)
    top_s = top.view(H, B, n, G, 1).permute(1, 0, 3, 2, 4)
    # own rows and drafted rows
    k = torch.cat([s["k"][:, :cap], s["kd"]], 1).float().permute(0, 2, 3, 1)
    v = torch.cat([s["v"][:, :cap], s["vd"]], 1).float().permute(0, 2, 1, 3)
    mine = (q.permute(0, 2, 3, 1, 4).reshape(B, H, G * n, hd) @ k).view(B, H, G, n, cap + n)
    cached = (torch.arange(cap, device="cuda") < s["lens"][:, None])[:, None].expand(B, n, cap)
    among = s["seen"] if case["branch"] else torch.ones((n, n), dtype=torch.bool, device="cuda").tril().expand(B, n, n)
    mine.masked_fill_(~torch.cat([cached, among], 2)[:, None, None], -math.inf)
    top_m = mine.amax(-1, keepdim=True)
    both = torch.maximum(top_s, top_m)  # [B][H][G][n][1]
    shared.sub_(both.permute(1, 0, 3, 2, 4).reshape(H, B * n * G, 1)).exp_()
    mine.sub_(both).exp_()
    total = shared.sum(-1).view(H, B, n, G).permute(1, 0, 3, 2) + mine.sum(-1)
    out = (shared @ s["vp"].float().permute(1, 0, 2)).view(H, B, n, G, hd).permute(1, 2, 0, 3, 4)
    out = out + (mine.view(B, H, G * n, cap + n) @ v).view(B, H, G, n, hd).permute(0, 3, 1, 2, 4)
    s["out"].copy_((out / total.permute(0, 3, 1, 2)[..., None]).reshape(B, n, G * H, hd))
    s["lse"].copy_((total.log() + both[..., 0]).permute(0, 3, 1, 2).reshape(B, n, G * H))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_sample(s):
    case = s["case"]
    V = case["vocab"]
    x = s["logits"].float()
    greedy = (s["temperature"] == 0)[:, None]
    t = torch.where(greedy, 1.0, s["temperature"][:, None])
    top, index = torch.sort(x, dim=1, descending=True, stable=True)
    i = torch.arange(V, device="cuda")
    keep = top > -math.inf
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (i < k) | (k == 0)
    # cumulative masses and borders in 64 bits
    far = (top.double() - top[:, :1].double()) / t.double()
    if s["top_p"] is not None:
        mass = torch.where(keep, far.exp(), 0.0)
        before = torch.zeros_like(mass)
        before[:, 1:] = mass.cumsum(1)[:, :-1]
        p = s["top_p"][:, None].double()
        keep &= (before < p * (before[:, -1:] + mass[:, -1:])) | (p >= 1.0) | (i == 0)
    if s["min_p"] is not None:
        keep &= far >= s["min_p"][:, None].double().log()
    keep = torch.where(greedy, i == 0, keep)
    there = torch.zeros_like(keep).scatter_(1, index, keep)
    away = (x - top[:, :1]) / t
    w = torch.where(there, away.exp(), 0.0)
    total = w.sum(1, keepdim=True)
    w /= total
    token = torch.where(there, w / s["noise"], -1.0).argmax(1)
    s["token"].copy_(token)
    s["logprob"].copy_((away.gather(1, token[:, None]) - total.log())[:, 0])
    s["kept"].copy_(keep.sum(1))
    if s["probs"] is not None:
        s["probs"].copy_(w)
    return _sampled(s)


def _sampled(s):
    return {k: s[k] for k in ("token", "logprob", "kept", "probs") if s[k] is not None}


_PLAIN = {"norm_rope": _plain_norm_rope, "prefix": _plain_prefix, "sample": _plain_sample}


# ---------------------------------------------------------------- the library's calls
def _kept(s, name, make):
    """What a program makes once and keeps: a descriptor, a workspace."""
    if name not in s:
        s[name] = make()
    return s[name]


def _scratch(size):
    return torch.empty(max(256, size), dtype=torch.uint8, device="cuda")


def _norm_rope_desc(rf, case):
    heads = case["q_heads"] + case["k_heads"]
    rope = rf.rf_rope_desc(
        n_rows=case["rows"], n_heads=heads, head_dim=case["hd"], rot_dim=case["rot"],
        ld_in=(heads + case["spare"]) * case["hd"], ld_out=heads * case["hd"], pos_offset=case["offset"],
        theta=case["theta"], factor=_FACTOR, original_rows=_ORIGINAL, low_turns=_LOW, high_turns=_HIGH, amplitude=1.0,
        layout=rf.RF_ROPE_HALF if case["layout"] == "half" else rf.RF_ROPE_INTERLEAVED,
        dtype=rf.RF_BF16 if case["dtype"] == "bf16" else rf.RF_F32, transpose=0, scaling=_SCALING[case["scaling"]])
    return rf.rf_norm_rope_desc(rope=rope, n_q_heads=case["q_heads"], eps=_EPS)


def _own_norm_rope(s):
    import ridge_map_kv_gb300 as rf
    desc = _kept(s, "desc", lambda: _norm_rope_desc(rf, s["case"]))
    if not s["case"]["backward"]:
        rf.rf_norm_rope(desc, s["x"], s["q_gain"], s["k_gain"], s["y"], s["positions"])
        return {"y": s["y"]}
    ws = _kept(s, "ws", lambda: _scratch(rf.rf_norm_rope_backward_workspace_bytes(desc)))
    rf.rf_norm_rope_backward(desc, s["x"], s["q_gain"], s["k_gain"], s["dy"], s["positions"], s["dx"], s["dq_gain"],
                             s["dk_gain"], ws, ws.numel())
    return {k: s[k] for k in ("dx", "dq_gain", "dk_gain")}


def _own_prefix(s):
    import ridge_map_kv_gb300 as rf
    case, q, k, kp, kd, out = s["case"], s["q"], s["k"], s["kp"], s["kd"], s["out"]
    desc = _kept(s, "desc", lambda: rf.rf_prefix_attn_desc(
        attn=rf.rf_attn_desc(n_seqs=case["seqs"], n_q_heads=case["kv"] * case["group"], n_kv_heads=case["kv"],
                             head_dim=case["hd"], n_nodes=case["nodes"], capacity=case["cap"], q_row_stride=q.stride(1),
                             q_seq_stride=q.stride(0), draft_row_stride=kd.stride(1), draft_seq_stride=kd.stride(0),
                             cache_row_stride=k.stride(1), cache_seq_stride=k.stride(0), out_row_stride=out.stride(1),
                             out_seq_stride=out.stride(0), scale=case["hd"] ** -0.5),
        prefix_capacity=kp.shape[0], prefix_row_stride=kp.stride(0)))
    ws = _kept(s, "ws", lambda: _scratch(rf.rf_prefix_attn_workspace_bytes(desc)))
    rf.rf_prefix_attention(desc, q, kp, s["vp"], s["prefix_len"], k, s["v"], s["lens"], kd, s["vd"], s["mask"], out,
                           s["lse"], None, ws, ws.numel())
    return {"out": out, "lse": s["lse"]}


def _own_sample(s):
    import ridge_map_kv_gb300 as rf
    case = s["case"]
    V = case["vocab"]
    desc = _kept(s, "desc", lambda: rf.rf_sample_desc(
        n_rows=case["rows"], vocab=V, ld_logits=V, ld_noise=V, ld_probs=V,
        dtype=rf.RF_BF16 if case["dtype"] == "bf16" else rf.RF_F32))
    rf.rf_sample(desc, s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["noise"], s["probs"],
                 s["token"], s["logprob"], s["kept"])
    return _sampled(s)


_OWN = {"norm_rope": _own_norm_rope, "prefix": _own_prefix, "sample": _own_sample}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "prefix": _exact_prefix, "sample": _exact_sample}[case["op"]](s)


def _exact_norm_rope(s):
    """Each pair as a complex number times exp(i angle); the gradient from the norm's Jacobian."""
    case = s["case"]
    Hq, hd, r = case["q_heads"], case["hd"], case["rot"]
    heads = Hq + case["k_heads"]
    rows = case["rows"]
    p = s["positions"].double() if case["given"] else torch.arange(rows, dtype=F64, device="cuda") + case["offset"]
    angle = torch.outer(p, _frequencies(case))
    turn = torch.polar(torch.ones_like(angle), angle)

    def rotate(x, by):
        y = x.clone()
        one, two = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
        z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * by
        y[..., one], y[..., two] = z.real, z.imag
        return y

    y = None if case["backward"] else torch.zeros((rows, heads, hd), dtype=F64, device="cuda")
    dx = s["dx"].double() if case["backward"] else None
    dg = torch.zeros((2, hd), dtype=F64, device="cuda")
    for h in range(heads):  # one head after another
        x = s["x"][:, h * hd:(h + 1) * hd].double()
        gain = (s["q_gain"] if h < Hq else s["k_gain"]).double()
        size = torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / hd + _EPS)
        unit = x / size
        if not case["backward"]:
            y[:, h] = rotate(unit * gain, turn)
            continue
        back = rotate(s["dy"][:, h * hd:(h + 1) * hd].double(), turn.conj())
        dg[0 if h < Hq else 1] += (back * unit).sum(0)
        back = back * gain
        along = torch.einsum("rc,rc->r", back, unit)[:, None] / hd
        dx[:, h * hd:(h + 1) * hd] = (back - along * unit) / size
    if not case["backward"]:
        return {"y": y.view(rows, heads * hd)}
    return {"dx": dx, "dq_gain": dg[0], "dk_gain": dg[1]}


def _exact_prefix(s):
    """One sequence and KV head after another, over the rows in use alone."""
    case = s["case"]
    B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
    out = torch.zeros((B, n, H, G, hd), dtype=F64, device="cuda")
    lse = torch.zeros((B, n, H, G), dtype=F64, device="cuda")
    order = torch.ones((n, n), device="cuda").tril().bool()
    for h in range(H):
        kp, vp = s["kp"][:, h].double(), s["vp"][:, h].double()
        for b, m in enumerate(_lengths(case)):
            k = torch.cat([kp, s["k"][b, :m, h].double(), s["kd"][b, :, h].double()])
            v = torch.cat([vp, s["v"][b, :m, h].double(), s["vd"][b, :, h].double()])
            x = torch.einsum("igc,tc->igt", s["q"][b, :, h * G:(h + 1) * G].double(), k) / math.sqrt(hd)
            x[..., len(k) - n:].masked_fill_(~(s["seen"][b] if case["branch"] else order)[:, None], -math.inf)
            lse[b, :, h] = torch.logsumexp(x, -1)
            out[b, :, h] = torch.softmax(x, -1) @ v
    return {"out": out.view(B, n, H * G, hd), "lse": lse.view(B, n, H * G)}


def _exact_sample(s):
    """One request after another: its tokens by falling logit, cut three times."""
    case = s["case"]
    setting = {k: None if s[k] is None else s[k].tolist() for k in ("temperature", "top_k", "top_p", "min_p")}
    probs = torch.zeros((case["rows"], case["vocab"]), dtype=F64, device="cuda") if case["probs"] else None
    logprob = torch.zeros(case["rows"], dtype=F64, device="cuda")
    for row in range(case["rows"]):
        x = s["logits"][row].double()
        order = torch.argsort(-x, stable=True)
        if setting["temperature"][row] == 0.0:
            if case["probs"]:
                probs[row, order[0]] = 1.0
            continue
        order = order[:int((x > -math.inf).sum())]
        if setting["top_k"] and setting["top_k"][row] > 0:
            order = order[:setting["top_k"][row]]
        p = torch.softmax(x[order] / setting["temperature"][row], 0)
        if setting["top_p"] and setting["top_p"][row] < 1.0:
            reach = torch.searchsorted(p.cumsum(0), torch.tensor([setting["top_p"][row]], dtype=F64, device="cuda"))
            p = p[:int(reach) + 1]
        if setting["min_p"]:
            p = p[p >= setting["min_p"][row] * p[0]]
        order, p = order[:len(p)], p / p.sum()
        if case["probs"]:
            probs[row, order] = p
        logprob[row] = p[torch.argmax(p / s["noise"][row, order].double())].log()
    out = {"token": None, "logprob": logprob, "kept": None}
    return {**out, "probs": probs} if case["probs"] else out
