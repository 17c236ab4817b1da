"""Workloads of the serving operators: what each one computes, in a plain form and
through the library.

A filled KV cache is decoded from by drafting a tree of tokens and checking it in one
pass: the tree's queries and keys are rotated (rope), every node attends to the cache
and to its ancestors (attention), the drafted tokens are accepted or refused against
the target's probabilities and the accepted rows join the cache (verify), each cached
row's attention weight is added up (weights), and rows of little weight leave the cache
(evict).

``own = False`` computes the operators from elementary torch operations in 32 bits;
``own = True`` calls the library. ``exact`` computes them in 64 bits, apart from both.
Head counts, head sizes, widths and lengths are those of this repository's synthetic
deployments (8 KV heads of 128 under 32 or 40 query heads, 2 under 20, prompts up to
32,768 rows with 4,096 tail rows) or generic.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
_SCALING = {"none": 0, "linear": 1, "base": 2, "wavelength": 3, "ramp": 4}


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # A decoding step's rotation: one tree of 16 nodes for each of 8 sequences, query and key heads of a fused
        # row, frequencies stretched by wavelength; the tree's masks and positions are built in the same step.
        dict(name="rope step", op="rope", seqs=8, nodes=16, branch=3, heads=40, spare=8, hd=128, rot=128,
             layout="half", dtype="bf16", transpose=False, scaling="wavelength", factor=8.0, theta=5.0e5, offset=20000),
        # A whole prompt's queries and keys, base stretched for a long context.
        dict(name="rope prompt", op="rope", seqs=1, nodes=32768, branch=0, heads=48, spare=8, hd=128, rot=128,
             layout="half", dtype="bf16", transpose=False, scaling="base", factor=4.0, theta=1.0e6, offset=0),
        # The gradient of an interleaved rotation of part of each head, in 32 bits, odd row count.
        dict(name="rope gradient", op="rope", seqs=1, nodes=8191, branch=0, heads=40, spare=0, hd=128, rot=96,
             layout="interleaved", dtype="f32", transpose=True, scaling="ramp", factor=16.0, theta=1.0e4, offset=513),
        # One token of one sequence at the end of a full-length prompt: latency and the cache's bytes.
        dict(name="attention token", op="attention", seqs=1, nodes=1, branch=1, kv=8, group=5, hd=128, length=32767,
             cap=32768),
        # Trees of 64 nodes for 16 sequences of ragged lengths.
        dict(name="attention trees", op="attention", seqs=16, nodes=64, branch=4, kv=8, group=4, hd=128, length=16384,
             cap=16512),
        # The exact tail of a filled prompt: 4,096 rows in order over 28,672 filled ones.
        dict(name="attention tail", op="attention", seqs=1, nodes=4096, branch=0, kv=8, group=5, hd=128, length=28672,
             cap=32768),
        # Each accepted path's weights over its sequence's cache, once per layer and step.
        dict(name="weights path", op="weights", seqs=16, nodes=64, path=7, kv=8, group=4, hd=128, length=16384,
             cap=16512, decay=1.0),
        # The last 64 prompt rows' weights over the whole prompt, older sums decayed.
        dict(name="weights window", op="weights", seqs=1, nodes=64, path=0, kv=2, group=10, hd=128, length=32768,
             cap=32768, decay=0.5),
        # Steady state: a few rows over the budget leave each head at every step.
        dict(name="evict step", op="evict", layers=20, seqs=2, kv=8, hd=128, length=4103, keep=4096, cap=4224, sink=4,
             recent=256),
        # After the prompt: a quarter of the rows stays.
        dict(name="evict prompt", op="evict", layers=20, seqs=1, kv=8, hd=128, length=16384, keep=4096, cap=16512,
             sink=4, recent=512),
        # A chain of four drafted tokens behind the last one, drafted without probabilities.
        dict(name="verify chain", op="verify", seqs=1, nodes=5, branch=1, vocab=32000, draft=False, layers=32, kv=8,
             hd=128, length=1000, cap=1024),
        # Trees of 64 nodes for 16 sequences with the draft's probabilities.
        dict(name="verify trees", op="verify", seqs=16, nodes=64, branch=4, vocab=131072, draft=True, layers=32, kv=8,
             hd=128, length=300, cap=384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "weights", "evict", "verify"])
    if op == "rope":
        hd = rng.choice([64, 128])
        heads = rng.choice([4, 10, 22, 40, 48])
        tree = rng.random() < 0.4
        nodes = _log(rng, 1, 64) if tree else _log(rng, 1, 32768)
        return dict(op=op, seqs=_log(rng, 1, 16) if tree else 1, nodes=nodes, branch=rng.randint(1, 4) if tree else 0,
                    heads=heads, spare=rng.choice([0, 2, 8]), hd=hd, rot=rng.choice([hd, hd // 2, hd // 4 * 3, 20]),
                    layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if nodes <= 8192 else "bf16", transpose=rng.random() < 0.5,
                    scaling=rng.choice(sorted(_SCALING)), factor=rng.choice([2.0, 4.0, 8.0]),
                    theta=rng.choice([1.0e4, 5.0e5, 1.0e6]), offset=rng.randint(0, 30000))
    if op == "attention":
        kv, hd = rng.choice([1, 2, 8]), rng.choice([64, 128])
        group = rng.choice([1, 2, 4, 5, 10]) if kv < 8 else rng.choice([1, 2, 4, 5])
        if rng.random() < 0.3:
            seqs, nodes, branch = 1, _log(rng, 64, 4096), 0
        else:
            seqs, nodes, branch = _log(rng, 1, 16), _log(rng, 1, 64), rng.randint(1, 4)
        length = _log(rng, 1, 28672 if seqs == 1 else 16384)
        return dict(op=op, seqs=seqs, nodes=nodes, branch=branch, kv=kv, group=group, hd=hd, length=length,
                    cap=length + rng.randint(0, 200))
    if op == "weights":
        kv, hd = rng.choice([1, 2, 8]), rng.choice([64, 128])
        nodes = _log(rng, 1, 64)
        length = nodes + _log(rng, 1, 16000)
        return dict(op=op, seqs=_log(rng, 1, 16), nodes=nodes, path=rng.choice([0, max(1, nodes // 4), max(1, nodes // 9)]),
                    kv=kv, group=rng.choice([1, 2, 4, 5]), hd=hd, length=length, cap=length + rng.randint(0, 200),
                    decay=rng.choice([1.0, 0.9, 0.5]))
    if op == "evict":
        length = _log(rng, 64, 16384)
        keep = max(1, int(length * rng.choice([0.25, 0.5, 0.9, 0.99, 1.0])))
        return dict(op=op, layers=rng.choice([1, 4, 20]), seqs=1 if length > 4096 else rng.randint(1, 2),
                    kv=rng.choice([2, 8]), hd=rng.choice([64, 128]), length=length, keep=keep,
                    cap=length + rng.randint(0, 100), sink=rng.choice([0, 4]), recent=rng.choice([0, keep // 8]))
    length = _log(rng, 1, 300)
    nodes = _log(rng, 1, 64)
    return dict(op=op, seqs=_log(rng, 1, 16), nodes=nodes, branch=rng.randint(1, 4), vocab=_log(rng, 1000, 131072),
                draft=rng.random() < 0.6, layers=rng.choice([1, 4, 32]), kv=rng.choice([2, 8]), hd=rng.choice([64, 128]),
                length=length, cap=length + nodes + rng.randint(0, 40))


def _lengths(case):
    """Ragged lengths of the sequences, the first the longest."""
    top = case["length"]
    return [max(1, int(top * (1.0 - (0.61803399 * b) % 1.0))) for b in range(case["seqs"])]


def _path_lengths(case):
    """How many of a sequence's nodes add their weights; path = 0: all of them, in order."""
    if case["path"] == 0:
        return [case["nodes"]] * case["seqs"]
    return [1 + (case["path"] - 1 + b) % case["path"] for b in range(case["seqs"])]


def _weight_lengths(case):
    return [max(n, p) for n, p in zip(_lengths(case), _path_lengths(case))]


# ------------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFF)
    return g


def _randn(shape, g, dtype=BF16, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _parents(case, seed):
    """Parents of each sequence's nodes: node 0 is the root, node i hangs under one of the
    `branch` nodes' worth before it, so every tree of a case has its own shape."""
    n, b = case["nodes"], max(1, case["branch"])
    g = torch.Generator()
    g.manual_seed(int(seed) * 7919 + 17)
    i = torch.arange(n)
    jitter = torch.randint(0, b, (case["seqs"], n), generator=g)
    p = torch.clamp(torch.div(i - 1 + jitter, b, rounding_mode="floor"), min=0)
    p = torch.minimum(p, torch.clamp(i - 1, min=0)).to(torch.int32)
    p[:, 0] = -1
    return p.cuda()


def _ancestors(parents):
    """bool [B][n][n]: node j is node i or an ancestor of it, by repeated squaring."""
    B, n = parents.shape
    step = torch.eye(n, device=parents.device, dtype=F32).repeat(B, 1, 1)
    has = (parents >= 0).to(F32)
    step.scatter_add_(2, parents.clamp(min=0).long()[..., None], has[..., None])
    for _ in range(max(1, (n - 1).bit_length())):
        step = (step @ step).clamp(max=1.0)
    return step > 0


def _words(seen):
    """bool [B][n][n] -> the mask words: bit j % 64 of word j / 64 of node i."""
    B, n, _ = seen.shape
    w = (n + 63) // 64
    bits = torch.zeros((B, n, w * 64), dtype=torch.int64, device=seen.device)
    bits[:, :, :n] = seen.long()
    return (bits.view(B, n, w, 64) << torch.arange(64, device=seen.device)).sum(-1)


def _bits(words, n):
    """The inverse of _words."""
    B, m, w = words.shape
    return ((words[..., None] >> torch.arange(64, device=words.device)) & 1).view(B, m, w * 64)[:, :, :n].bool()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed, sum(ord(c) for c in case["op"]))
    s = {"case": case}
    if case["op"] == "rope":
        rows = case["seqs"] * case["nodes"]
        width = (case["heads"] + case["spare"]) * case["hd"]
        dtype = BF16 if case["dtype"] == "bf16" else F32
        s["x"] = _randn((rows, width), g, dtype)
        s["y"] = torch.empty((rows, case["heads"] * case["hd"]), dtype=dtype, device="cuda")
        s["next_pos"] = _ints([case["offset"] + 97 * b for b in range(case["seqs"])])
        if case["branch"]:
            s["parents"] = _parents(case, seed)
            s["mask"] = torch.zeros((case["seqs"], case["nodes"], (case["nodes"] + 63) // 64), dtype=torch.int64, device="cuda")
            s["positions"] = torch.zeros((case["seqs"], case["nodes"]), dtype=torch.int32, device="cuda")
    elif case["op"] == "attention":
        B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
        # queries, keys and values of the drafted rows come from one projection
        fused = _randn((B, n, (G * H + 2 * H), hd), g)
        fused[:, :, :G * H] *= 2.0
        s["q"], s["kd"], s["vd"] = fused[:, :, :G * H], fused[:, :, G * H:G * H + H], fused[:, :, G * H + H:]
        s["k"], s["v"] = _randn((B, case["cap"], H, hd), g), _randn((B, case["cap"], H, hd), g)
        s["lens"] = _ints(_lengths(case))
        s["mask"] = _words(_ancestors(_parents(case, seed))) if case["branch"] else None
        s["out"] = torch.empty((B, n, G * H, hd), dtype=BF16, device="cuda")
        s["lse"] = torch.empty((B, n, G * H), dtype=F32, device="cuda")
    elif case["op"] == "weights":
        B, n, H, G, hd, cap = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd", "cap"))
        s["q"] = _randn((B, n, G * H, hd), g, std=2.0)
        s["k"] = _randn((B, cap, H, hd), g)
        lens, sel = _weight_lengths(case), _path_lengths(case)
        s["lens"], s["n_path"] = _ints(lens), _ints(sel)
        # an accepted path: ascending nodes from the root
        order = torch.rand((B, n), generator=g, device="cuda")
        order[:, 0] = -1.0
        rank = order.argsort(1).argsort(1)
        taken = rank < s["n_path"][:, None]
        s["path"] = torch.where(taken, torch.arange(n, device="cuda")[None], n).sort(1).values.to(torch.int32)
        s["path"][s["path"] == n] = -1
        # the statistics that the path's attention left behind
        s["lse"] = _randn((B, n, G * H), g, F32)
        m = case["path"] or n
        j = s["path"][:, :m].clamp(min=0).long()[..., None].expand(B, m, G * H)
        stat = torch.logsumexp(_path_scores(s), dim=4).permute(0, 2, 1, 3).reshape(B, m, G * H)
        there = (s["path"][:, :m] >= 0)[..., None].expand_as(stat)
        s["lse"].scatter_(1, torch.where(there, j, 0), torch.where(there, stat, stat[:, :1].expand_as(stat)))
        s["score"] = torch.empty((B, H, cap), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        s["score_out"] = torch.zeros((B, H, cap), dtype=F32, device="cuda")
    elif case["op"] == "evict":
        L, B, H, cap, hd = (case[k] for k in ("layers", "seqs", "kv", "cap", "hd"))
        s["k"], s["v"] = _randn((L, B, cap, H, hd), g), _randn((L, B, cap, H, hd), g)
        s["lens"] = _ints(_lengths(case))
        s["next_pos"] = _ints([n + 3 for n in _lengths(case)])
        s["score"] = torch.empty((L, B, H, cap), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        # earlier evictions left every head's positions in an order of its own
        s["pos"] = torch.rand((L, B, H, cap), generator=g, device="cuda").argsort(-1).to(torch.int32)
        s["score_out"], s["pos_out"] = torch.zeros_like(s["score"]), torch.zeros_like(s["pos"])
        s["new_lens"] = torch.zeros_like(s["lens"])
    else:
        B, n, V, L, H, hd, cap = (case[k] for k in ("seqs", "nodes", "vocab", "layers", "kv", "hd", "cap"))
        logits = _randn((B, n, V), g, F32, 3.0)
        s["target"] = torch.softmax(logits, -1)
        s["parents"] = _parents(case, seed)
        if case["draft"]:  # a smaller model that mostly agrees
            drafted = torch.softmax(logits.add_(_randn((B, n, V), g, F32, 0.8)), -1)
            s["draft"] = drafted
        else:
            s["draft"], drafted = None, s["target"]
        at = s["parents"].clamp(min=0).long()[..., None].expand(B, n, V)
        race = torch.empty((B, n, V), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        s["tokens"] = (drafted.gather(1, at) / race).argmax(-1).to(torch.int32)
        del logits, drafted, at, race
        s["u"] = torch.rand((B, n), generator=g, device="cuda")
        s["noise"] = torch.empty((B, V), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        s["path"] = torch.zeros((B, n), dtype=torch.int32, device="cuda")
        s["n_path"], s["token"] = _ints([0] * B), _ints([0] * B)
        s["kd"], s["vd"] = _randn((L, B, n, H, hd), g), _randn((L, B, n, H, hd), g)
        s["k"], s["v"] = _randn((L, B, cap, H, hd), g), _randn((L, B, cap, H, hd), g)
        s["lens"] = _ints(_lengths(case))
        s["next_pos"] = _ints([m + 5 for m in _lengths(case)])
        s["score"] = torch.empty((L, B, H, cap), dtype=F32, device="cuda").exponential_(1.0, generator=g)
        s["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(L, B, H, 1)
        s["new_lens"], s["new_next_pos"] = torch.zeros_like(s["lens"]), torch.zeros_like(s["lens"])
    return s


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work of a pass
def work(case):
    op = case["op"]
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        rows = case["seqs"] * case["nodes"]
        extra = rows * (4 + 4 + 8 * ((case["nodes"] + 63) // 64)) if case["branch"] else 0
        return {"bytes": 2 * rows * case["heads"] * case["hd"] * size + extra,
                "flops": 3 * rows * case["heads"] * case["rot"]}
    if op == "attention":
        B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
        rows = sum(_lengths(case))
        among = n * (n + 1) // 2 if not case["branch"] else n * max(1, n.bit_length())
        mask = B * n * ((n + 63) // 64) * 8 if case["branch"] else 0
        return {"bytes": 2 * (2 * B * n * G * H * hd + 2 * H * hd * (rows + B * n)) + 4 * B * n * G * H + mask,
                "flops": 4 * G * H * hd * (n * rows + B * among)}
    if op == "weights":
        H, G, hd = case["kv"], case["group"], case["hd"]
        lens, sel = _weight_lengths(case), _path_lengths(case)
        return {"bytes": sum(lens) * H * (2 * hd + 8) + sum(sel) * G * H * (2 * hd + 4),
                "flops": 2 * G * H * hd * sum(n * j for n, j in zip(lens, sel))}
    if op == "evict":
        L, H, hd, keep = case["layers"], case["kv"], case["hd"], case["keep"]
        # scores and positions in, the kept ones out; a kept row beyond the budget moves into a hole below it
        total = 0
        for n in _lengths(case):
            total += 8 * n + 8 * min(n, keep)
            if n > keep:
                total += 2 * 2 * 2 * hd * keep * (n - keep) // n
        return {"bytes": L * H * total, "flops": L * H * sum(_lengths(case))}
    B, n, V, L, H, hd = (case[k] for k in ("seqs", "nodes", "vocab", "layers", "kv", "hd"))
    # the last row's distribution (and the draft's) and the noise; the root's rows join the cache at the least
    return {"bytes": B * (V * 4 * (3 if case["draft"] else 2) + 20 * n + L * H * (8 * hd + 8)), "flops": 3 * B * V}


# -------------------------------------------------------------------- plain forms
def _frequencies(case):
    """Angular frequency of each rotated pair, 64 bits (a table that a program keeps)."""
    r, theta, s = case["rot"], case["theta"], case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    kind, original, low, high = case["scaling"], 8192.0, 1.0, 4.0 if case["scaling"] == "wavelength" else 32.0
    if kind == "base":
        theta = theta * s ** (r / (r - 2.0))
    f = theta ** (-2.0 * i / r)
    if kind == "linear":
        return f / s
    if kind == "wavelength":
        turns = original * f / (2.0 * math.pi)
        return f * ((t := ((turns - low) / (high - low)).clamp(0.0, 1.0)) + (1.0 - t) / s)
    if kind == "ramp":
        at = lambda turns: r * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - t) + f / s * t
    return f


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


def _rope_positions(s):
    case = s["case"]
    if not case["branch"]:
        return s["next_pos"][:1] + torch.arange(case["nodes"], device="cuda", dtype=torch.int32)
    return s["positions"].reshape(-1)


def _rotate(x, positions, case, dtype):
    """x [rows][heads][hd] in `dtype`; angles in 64 bits, since one of 32 is off by 2e-3 at row 32768."""
    angle = positions.double()[:, None] * _frequencies(case)
    sign = -1.0 if case["transpose"] else 1.0
    c = (angle.cos() * _amplitude(case)).to(dtype)[:, None]
    t = (angle.sin() * (sign * _amplitude(case))).to(dtype)[:, None]
    r = case["rot"]
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * t, b * c + a * t
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * t, b * c + a * t
    return y


def _plain_rope(s):
    case = s["case"]
    out = {}
    if case["branch"]:
        seen = _ancestors(s["parents"])
        s["mask"].copy_(_words(seen))
        s["positions"].copy_(s["next_pos"][:, None] + seen.sum(-1) - 1)
        out = {"mask": s["mask"], "positions": s["positions"]}
    x = s["x"][:, :case["heads"] * case["hd"]].float().view(-1, case["heads"], case["hd"])
    s["y"].copy_(_rotate(x, _rope_positions(s), case, F32).view_as(s["y"]))
    return {"y": s["y"], **out}


def _seen(s, cap):
    """bool [B][n][cap + n]: which cache rows and drafted rows a node sees."""
    case = s["case"]
    B, n = case["seqs"], case["nodes"]
    cached = (torch.arange(cap, device="cuda") < s["lens"][:, None])[:, None].expand(B, n, cap)
    if s["mask"] is None:
        among = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()[None].expand(B, n, n)
    else:
        among = _bits(s["mask"], n)
    return torch.cat([cached, among], 2)


def _attend(s, dtype):
    case = s["case"]
    B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
    cap = case["length"]  # the longest sequence
    q = s["q"].to(dtype).view(B, n, H, G, hd).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, hd)
    k = torch.cat([s["k"][:, :cap], s["kd"]], 1).to(dtype).permute(0, 2, 1, 3)
    v = torch.cat([s["v"][:, :cap], s["vd"]], 1).to(dtype).permute(0, 2, 1, 3)
    hidden = ~_seen(s, cap)[:, None, None]
    p = (q @ k.transpose(2, 3)).mul_(hd ** -0.5).view(B, H, G, n, cap + n).masked_fill_(hidden, -math.inf)
    top = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, G * n, cap + n) @ v).view(B, H, G, n, hd) / total
    lse = (total.log() + top).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, G * H, hd), lse.permute(0, 3, 1, 2).reshape(B, n, G * H)


def _plain_attention(s):
    out, lse = _attend(s, F32)
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _path_scores(s, dtype=F32):
    """Scaled scores [B][H][longest path][G][cap] of the paths' nodes, -inf past a path's end and at unseen rows.
    The j-th node of a path sees the rows before it and its own, the last node every row."""
    case = s["case"]
    B, H, G, hd, cap = (case[k] for k in ("seqs", "kv", "group", "hd", "cap"))
    n = case["path"] or case["nodes"]  # the longest path
    at = s["path"][:, :n].clamp(min=0).long()
    q = s["q"].to(dtype).gather(1, at[..., None, None].expand(B, n, G * H, hd)).view(B, n, H, G, hd)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, n * G, hd)
    k = s["k"].to(dtype).permute(0, 2, 3, 1)
    x = (q @ k).mul_(hd ** -0.5).view(B, H, n, G, cap)
    last = s["lens"][:, None] - s["n_path"][:, None] + torch.arange(n, device="cuda")
    last = torch.where(s["path"][:, :n] >= 0, last, -1)
    hidden = torch.arange(cap, device="cuda") > last[..., None]
    return x.masked_fill_(hidden[:, None, :, None], -math.inf)


def _weights(s, dtype):
    case = s["case"]
    B, H, G = (case[k] for k in ("seqs", "kv", "group"))
    n = case["path"] or case["nodes"]
    at = s["path"][:, :n].clamp(min=0).long()
    lse = s["lse"].to(dtype).gather(1, at[..., None].expand(B, n, G * H)).view(B, n, H, G).permute(0, 2, 1, 3)
    return s["score"].to(dtype) * case["decay"] + _path_scores(s, dtype).sub_(lse[..., None]).exp_().sum((2, 3))


def _plain_weights(s):
    there = torch.arange(s["case"]["cap"], device="cuda") < s["lens"][:, None, None]
    s["score_out"].copy_(torch.where(there, _weights(s, F32), s["score_out"]))
    return s["score_out"]


def _plain_evict(s):
    case = s["case"]
    cap, keep = case["cap"], min(case["keep"], case["cap"])
    slot = torch.arange(cap, device="cuda")
    n = s["lens"][None, :, None, None].long()
    sure = (s["pos"] < case["sink"]) | (s["pos"] >= s["next_pos"][None, :, None, None] - case["recent"])
    key = torch.where(sure, math.inf, s["score"].nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf))
    # order: rows in use, by weight, the lowest slot first among equals
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort((order >= n).byte(), dim=-1, stable=True).indices)
    kept = torch.zeros_like(sure).scatter_(-1, order[..., :keep], True) & (slot < n)
    hole, mover = ~kept & (slot < n.clamp(max=keep)), kept & (slot >= keep)
    rank = (mover.cumsum(-1) - 1).masked_fill_(~mover, cap)
    by_rank = torch.zeros(kept.shape[:-1] + (cap + 1,), dtype=torch.int64, device="cuda")
    by_rank.scatter_(-1, rank, slot.expand_as(rank))
    src = torch.where(hole, by_rank.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), slot)[..., :keep]
    live = slot[:keep] < n
    s["score_out"][..., :keep] = torch.where(live, s["score"].gather(-1, src), s["score_out"][..., :keep])
    s["pos_out"][..., :keep] = torch.where(live, s["pos"].gather(-1, src), s["pos_out"][..., :keep])
    rows = src.permute(0, 1, 3, 2)[..., None].expand(-1, -1, -1, -1, case["hd"])
    s["k"][:, :, :keep] = s["k"].gather(2, rows)
    s["v"][:, :, :keep] = s["v"].gather(2, rows)
    s["new_lens"].copy_(s["lens"].clamp(max=keep))
    return {k: s[k] for k in ("k", "v", "score_out", "pos_out", "new_lens")}


def _walk(s, dtype):
    """Walks each sequence's tree from its root: a child x of the current node is accepted when u q(x) Z < r(x),
    where r starts as the node's target row (Z = 1) and becomes max(r / Z - q, 0), with Z its sum, after a refusal.
    Where no child is left, the next token is the first argmax of r / noise. Children come in index order."""
    case = s["case"]
    B, n, V = case["seqs"], case["nodes"], case["vocab"]
    target, draft = s["target"].to(dtype), None if s["draft"] is None else s["draft"].to(dtype)
    u, noise = s["u"].to(dtype), s["noise"].to(dtype)
    b = torch.arange(B, device="cuda")
    at = torch.zeros(B, dtype=torch.int64, device="cuda")
    r, total = target[:, 0], torch.ones((B, 1), dtype=dtype, device="cuda")
    q = None if draft is None else draft[:, 0]
    taken = torch.zeros((B, n), dtype=torch.bool, device="cuda")
    taken[:, 0] = True
    for c in range(1, n):  # one node after another: what a node's row is depends on those before it
        x = s["tokens"][:, c].long()[:, None]
        child = s["parents"][:, c].long() == at
        qx = 1.0 if q is None else q.gather(1, x)
        yes = child & (u[:, c:c + 1] * qx * total < r.gather(1, x))[:, 0]
        left = r.scatter(1, x, 0.0) if q is None else (r / total - q).clamp(min=0.0)
        mass = left.sum(1, keepdim=True)
        no = (child & ~yes)[:, None] & (mass > 0)
        r = torch.where(yes[:, None], target[:, c], torch.where(no, left, r))
        total = torch.where(yes[:, None], 1.0, torch.where(no, mass, total))
        if q is not None:
            q = torch.where(yes[:, None], draft[:, c], q)
        taken[b, c] = yes
        at = torch.where(yes, c, at)
    token = torch.where(r > 0, r / noise, 0.0).argmax(1)
    return taken, token


def _commit(s, taken):
    """The accepted rows of every layer follow the cache's, with weight 0 and their own positions."""
    case = s["case"]
    n, cap = case["nodes"], case["cap"]
    i = torch.arange(n, device="cuda")
    path = torch.where(taken, i, n).sort(1).values
    count = taken.sum(1)
    row = torch.arange(cap, device="cuda")[None] - s["lens"][:, None]
    fresh = (row >= 0) & (row < count[:, None])
    src = path.gather(1, row.clamp(0, n - 1)).clamp(max=n - 1)
    shape = s["k"].shape
    rows = src[None, :, :, None, None].expand(shape)
    there = fresh[None, :, :, None, None]
    s["k"].copy_(torch.where(there, s["kd"].gather(2, rows), s["k"]))
    s["v"].copy_(torch.where(there, s["vd"].gather(2, rows), s["v"]))
    s["score"].copy_(torch.where(fresh[None, :, None], 0.0, s["score"]))
    s["pos"].copy_(torch.where(fresh[None, :, None], (s["next_pos"][:, None] + row)[None, :, None].int(), s["pos"]))
    s["path"].copy_(torch.where(path < n, path, -1))
    s["n_path"].copy_(count)
    s["new_lens"].copy_(s["lens"] + count)
    s["new_next_pos"].copy_(s["next_pos"] + count)


_ACCEPTED = ("path", "n_path", "token", "k", "v", "score", "pos", "new_lens", "new_next_pos")


def _plain_verify(s):
    taken, token = _walk(s, F32)
    s["token"].copy_(token)
    _commit(s, taken)
    return {k: s[k] for k in _ACCEPTED}


_PLAIN = {"rope": _plain_rope, "attention": _plain_attention, "weights": _plain_weights, "evict": _plain_evict,
          "verify": _plain_verify}


# ---------------------------------------------------------------- the library's calls
def _kept(s, name, make):
    """What a program makes once and keeps: a descriptor, a workspace."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own_rope(s):
    import ridge_map_kv_gb300 as rf
    case = s["case"]
    desc = _kept(s, "desc", lambda: rf.rf_rope_desc(
        n_rows=case["seqs"] * case["nodes"], n_heads=case["heads"], head_dim=case["hd"], rot_dim=case["rot"],
        ld_in=(case["heads"] + case["spare"]) * case["hd"], ld_out=case["heads"] * case["hd"],
        pos_offset=case["offset"], theta=case["theta"], factor=case["factor"], original_rows=8192.0, low_turns=1.0,
        high_turns=4.0 if case["scaling"] == "wavelength" else 32.0, amplitude=_amplitude(case),
        layout=rf.RF_ROPE_HALF if case["layout"] == "half" else rf.RF_ROPE_INTERLEAVED,
        dtype=rf.RF_BF16 if case["dtype"] == "bf16" else rf.RF_F32, transpose=int(case["transpose"]),
        scaling=_SCALING[case["scaling"]]))
    if case["branch"]:
        rf.rf_tree_build(case["seqs"], case["nodes"], s["parents"], s["next_pos"], s["mask"], s["positions"])
        rf.rf_rope(desc, s["x"], s["y"], s["positions"])
        return {"y": s["y"], "mask": s["mask"], "positions": s["positions"]}
    rf.rf_rope(desc, s["x"], s["y"])
    return {"y": s["y"]}


def _attn_desc(rf, s):
    case = s["case"]
    q, k = s["q"], s["k"]
    kd = s.get("kd", k[:, :1])
    out = s.get("out", q)
    return rf.rf_attn_desc(n_seqs=case["seqs"], n_q_heads=case["kv"] * case["group"], n_kv_heads=case["kv"],
                           head_dim=case["hd"], n_nodes=case["nodes"], capacity=case["cap"],
                           q_row_stride=q.stride(1), q_seq_stride=q.stride(0), draft_row_stride=kd.stride(1),
                           draft_seq_stride=kd.stride(0), cache_row_stride=k.stride(1), cache_seq_stride=k.stride(0),
                           out_row_stride=out.stride(1), out_seq_stride=out.stride(0), scale=case["hd"] ** -0.5)


def _scratch(size):
    return torch.empty(max(256, size), dtype=torch.uint8, device="cuda")


def _own_attention(s):
    import ridge_map_kv_gb300 as rf
    desc = _kept(s, "desc", lambda: _attn_desc(rf, s))
    ws = _kept(s, "ws", lambda: _scratch(rf.rf_attn_workspace_bytes(desc)))
    rf.rf_tree_attention(desc, s["q"], s["k"], s["v"], s["lens"], s["kd"], s["vd"], s["mask"], s["out"], s["lse"],
                         None, ws, ws.numel())
    return {"out": s["out"], "lse": s["lse"]}


def _own_weights(s):
    import ridge_map_kv_gb300 as rf
    desc = _kept(s, "desc", lambda: _attn_desc(rf, s))
    ws = _kept(s, "ws", lambda: _scratch(rf.rf_attn_weights_workspace_bytes(desc)))
    every = s["case"]["path"] == 0
    rf.rf_attn_weights(desc, s["q"], s["lse"], None if every else s["path"], None if every else s["n_path"], s["k"],
                       s["lens"], s["case"]["decay"], s["score"], s["score_out"], None, ws, ws.numel())
    return s["score_out"]


def _cache_desc(rf, s):
    case, k = s["case"], s["k"]
    return rf.rf_cache_desc(n_layers=case["layers"], n_seqs=case["seqs"], n_kv_heads=case["kv"], head_dim=case["hd"],
                            capacity=case["cap"], row_stride=k.stride(2), seq_stride=k.stride(1),
                            layer_stride=k.stride(0))


def _own_evict(s):
    import ridge_map_kv_gb300 as rf
    case = s["case"]
    desc = _kept(s, "desc", lambda: _cache_desc(rf, s))
    ws = _kept(s, "ws", lambda: _scratch(rf.rf_evict_workspace_bytes(desc, case["keep"])))
    rf.rf_evict(desc, case["keep"], case["sink"], case["recent"], s["lens"], s["next_pos"], s["k"], s["v"], s["score"],
                s["pos"], s["score_out"], s["pos_out"], s["new_lens"], None, ws, ws.numel())
    return {k: s[k] for k in ("k", "v", "score_out", "pos_out", "new_lens")}


def _own_verify(s):
    import ridge_map_kv_gb300 as rf
    case = s["case"]
    V, n = case["vocab"], case["nodes"]
    desc = _kept(s, "desc", lambda: rf.rf_verify_desc(n_seqs=case["seqs"], n_nodes=n, vocab=V, ld_target=V, ld_draft=V,
                                                      ld_noise=V))
    cache = _kept(s, "cache", lambda: _cache_desc(rf, s))
    rf.rf_verify_draft(desc, s["target"], s["draft"], s["tokens"], s["parents"], s["u"], s["noise"], s["path"],
                       s["n_path"], s["token"])
    kd = s["kd"]
    rf.rf_commit_draft(cache, n, kd.stride(2), kd.stride(1), kd.stride(0), s["path"], s["n_path"], s["lens"],
                       s["next_pos"], kd, s["vd"], s["k"], s["v"], s["score"], s["pos"], s["new_lens"],
                       s["new_next_pos"])
    return {k: s[k] for k in _ACCEPTED}


_OWN = {"rope": _own_rope, "attention": _own_attention, "weights": _own_weights, "evict": _own_evict,
        "verify": _own_verify}


# ------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(s)
    if op == "attention":
        return _exact_attention(s)
    if op == "weights":
        return _exact_weights(s)
    return _exact_evict(s) if op == "evict" else _exact_verify(s)


def _exact_rope(s):
    """Each pair as a complex number times exp(i angle)."""
    case = s["case"]
    heads, hd, r = case["heads"], case["hd"], case["rot"]
    out = {}
    if case["branch"]:
        up = s["parents"].tolist()
        B, n = case["seqs"], case["nodes"]
        depth = [[0] * n for _ in range(B)]
        for b in range(B):
            for i in range(1, n):
                depth[b][i] = depth[b][up[b][i]] + 1
        pos = torch.tensor(depth, device="cuda") + s["next_pos"][:, None]
        out = {"mask": None, "positions": None}
    else:
        pos = case["offset"] + torch.arange(case["nodes"], device="cuda")
    angle = pos.reshape(-1).double()[:, None] * _frequencies(case)
    turn = torch.polar(torch.full_like(angle, _amplitude(case)), -angle if case["transpose"] else angle)[:, None]
    x = s["x"][:, :heads * hd].double().view(-1, heads, hd)
    y = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    return {"y": y.view(-1, heads * hd), **out}


def _exact_attention(s):
    """One sequence and KV head after another, over the rows in use alone."""
    case = s["case"]
    B, n, H, G, hd = (case[k] for k in ("seqs", "nodes", "kv", "group", "hd"))
    out = torch.zeros((B, n, H, G, hd), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, n, H, G), dtype=torch.float64, device="cuda")
    for b, m in enumerate(_lengths(case)):
        among = torch.ones((n, n), device="cuda").tril().bool() if s["mask"] is None else _bits(s["mask"][b:b + 1], n)[0]
        for h in range(H):
            k = torch.cat([s["k"][b, :m, h], s["kd"][b, :, h]]).double()
            v = torch.cat([s["v"][b, :m, h], s["vd"][b, :, h]]).double()
            for g in range(G):
                x = s["q"][b, :, h * G + g].double() @ k.T / math.sqrt(hd)
                x[:, m:] = torch.where(among, x[:, m:], -math.inf)
                lse[b, :, h, g] = torch.logsumexp(x, 1)
                out[b, :, h, g] = torch.softmax(x, 1) @ v
    return {"out": out.view(B, n, H * G, hd), "lse": lse.view(B, n, H * G)}


def _exact_weights(s):
    case = s["case"]
    H, G, hd = case["kv"], case["group"], case["hd"]
    out = torch.zeros(s["score"].shape, dtype=torch.float64, device="cuda")
    path = s["path"].tolist()
    for b, (m, c) in enumerate(zip(_weight_lengths(case), _path_lengths(case))):
        at = torch.tensor(path[b][:c], device="cuda")
        last = m - c + torch.arange(c, device="cuda")
        seen = torch.arange(m, device="cuda") <= last[:, None]
        for h in range(H):
            q = s["q"][b, at, h * G:(h + 1) * G].double()
            x = torch.einsum("jgd,td->jgt", q, s["k"][b, :m, h].double()) / math.sqrt(hd)
            w = torch.exp(x - s["lse"][b, at, h * G:(h + 1) * G].double()[..., None]) * seen[:, None]
            out[b, h, :m] = s["score"][b, h, :m].double() * case["decay"] + w.sum((0, 1))
    return out


def _exact_evict(s):
    """One head after another: its rows in use as a sorted list of (sure or not, weight, slot)."""
    case = s["case"]
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    k, v, score_out, pos_out = (s[x].double() for x in ("k", "v", "score_out", "pos_out"))
    score, pos = s["score"].double().cpu().numpy(), s["pos"].cpu().numpy()
    for layer in range(case["layers"]):
        for b, n in enumerate(_lengths(case)):
            newest = n + 3
            for h in range(case["kv"]):
                w, at = score[layer, b, h, :n], pos[layer, b, h, :n]
                free = (at >= sink) & (at < newest - recent)
                best = np.lexsort((np.arange(n), -w, free))[:keep]
                holes = np.setdiff1d(np.arange(min(n, keep)), best)
                movers = np.sort(best[best >= keep])
                src = np.arange(min(n, keep))
                src[holes] = movers
                to = torch.from_numpy(src).cuda()
                m = len(src)
                k[layer, b, :m, h], v[layer, b, :m, h] = k[layer, b, to, h], v[layer, b, to, h]
                score_out[layer, b, h, :m] = s["score"][layer, b, h, to].double()
                pos_out[layer, b, h, :m] = s["pos"][layer, b, h, to].double()
    return {"k": k, "v": v, "score_out": score_out, "pos_out": None, "new_lens": None}


def _exact_verify(s):
    """One sequence after another, from each node to its accepted child."""
    case = s["case"]
    k, v, score = (s[x].double() for x in ("k", "v", "score"))
    n = case["nodes"]
    for b, m in enumerate(_lengths(case)):
        up, tokens, u = s["parents"][b].tolist(), s["tokens"][b].tolist(), s["u"][b].double().tolist()
        path, here = [0], 0
        while here is not None:
            r = s["target"][b, here].double()
            q = None if s["draft"] is None else s["draft"][b, here].double()
            total, here_next = 1.0, None
            for c in (c for c in range(n) if up[c] == here):
                x = tokens[c]
                if u[c] * (1.0 if q is None else float(q[x])) * total < float(r[x]):
                    here_next = c
                    path.append(c)
                    break
                r = r.index_fill(0, torch.tensor([x], device="cuda"), 0.0) if q is None else (r / total - q).clamp(min=0.0)
                total = float(r.sum())
            here = here_next
        to, at = torch.tensor(path, device="cuda"), m + len(path)
        k[:, b, m:at], v[:, b, m:at] = s["kd"][:, b, to].double(), s["vd"][:, b, to].double()
        score[:, b, :, m:at] = 0.0
    return {x: {"k": k, "v": v, "score": score}.get(x) for x in _ACCEPTED}
