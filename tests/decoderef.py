"""Plain 64-bit definitions of the decoding operators and their derived error bounds,
shared by the tests. Everything runs on the device of its inputs."""
from __future__ import annotations

import math

import torch

U24, U8 = 2.0 ** -24, 2.0 ** -8      # unit roundoffs: fp32 has 24 significant bits, bf16 has 8


def randn(shape, seed, dtype=torch.bfloat16, std=1.0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=device).normal_(0.0, std, generator=g)


# ------------------------------------------------------------------------- rope
def frequencies(rot, theta, scaling=0, factor=1.0, original=0.0, low=0.0, high=0.0):
    out = []
    if scaling == 2:
        theta = theta * factor ** (rot / (rot - 2.0))
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if scaling == 1:
            f /= factor
        elif scaling == 3:
            w = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f * w + f * (1.0 - w) / factor
        elif scaling == 4:
            d = lambda x: rot * math.log(original / (2 * math.pi * x)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(math.floor(d(high)), 0), min(math.ceil(d(low)), rot - 1)
            w = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1.0 - w) + f * w / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rope(x, pos, freqs, interleaved, transpose=False, amplitude=1.0):
    """x [rows][heads][hd] float64, pos [rows]; also each element's |x1| + |x2|."""
    r = 2 * len(freqs)
    ang = pos.double()[:, None] * freqs.to(x.device)
    if transpose:
        ang = -ang
    c, s = amplitude * ang.cos()[:, None], amplitude * ang.sin()[:, None]
    y, mag = x.clone(), torch.zeros_like(x)
    i1 = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    i2 = i1 + (1 if interleaved else r // 2)
    a, b = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = a * c - b * s, b * c + a * s
    mag[..., i1] = mag[..., i2] = amplitude * (a.abs() + b.abs())
    return y, mag


# ------------------------------------------------------------------------- trees
def random_parents(n, seed, reach=4):
    g = torch.Generator()
    g.manual_seed(seed)
    p = [-1]
    for i in range(1, n):
        lo = max(0, i - reach)
        p.append(int(torch.randint(lo, i, (1,), generator=g)))
    return p


def ancestors(parents):
    """bool [n][n]"""
    n = len(parents)
    seen = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = parents[j]
    return seen


def words(seen):
    """bool [..., n, n] -> int64 [..., n, ceil(n/64)]"""
    n = seen.shape[-1]
    w = (n + 63) // 64
    bits = torch.zeros(seen.shape[:-1] + (w * 64,), dtype=torch.int64)
    bits[..., :n] = seen.long()
    return (bits.view(seen.shape[:-1] + (w, 64)) << torch.arange(64)).sum(-1)


# --------------------------------------------------------------------- attention
def attention(q, k, v, kd, vd, lens, seen, scale):
    """float64 outputs, lse, and bounds on the kernel's errors.
    q [B][n][Hq][hd], k, v [B][cap][H][hd], kd, vd [B][n][H][hd], seen bool [B][n][n] or None (rows in order).

    A score is a sum of hd products in fp32: its error is at most hd 2^-22 sum |q||k| scale (the tensor cores may
    truncate), so a weight is off by that much and the exponential's 2^-21, relatively, twice (numerator and
    denominator); a weight is rounded to bf16 for its product with v, and the result once more."""
    B, n, Hq, hd = q.shape
    H = kd.shape[2]
    G = Hq // H
    out = torch.zeros((B, n, Hq, hd), dtype=torch.float64, device=q.device)
    lse = torch.full((B, n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    tril = torch.ones((n, n), device=q.device).tril().bool()
    for b in range(B):
        m = int(lens[b])
        among = tril if seen is None else seen[b].to(q.device)
        vis = torch.cat([torch.ones((n, m), dtype=torch.bool, device=q.device), among], 1)
        for h in range(H):
            kk = torch.cat([k[b, :m, h], kd[b, :, h]]).double()
            vv = torch.cat([v[b, :m, h], vd[b, :, h]]).double()
            used = vis.any(0)
            kk, vv = torch.where(used[:, None], kk, 0.0), torch.where(used[:, None], vv, 0.0)
            for g in range(G):
                a = h * G + g
                qq = q[b, :, a].double()
                s = torch.where(vis, qq @ kk.nan_to_num(0.0, 0.0, 0.0).T * scale, -math.inf)
                poison = vis & ~torch.isfinite(kk).all(1)[None]
                s = torch.where(poison, math.nan, s)
                ln = torch.logsumexp(s, 1)
                w = torch.where(vis, torch.exp(s - ln[:, None]), 0.0)
                w = torch.where(torch.isneginf(ln)[:, None], 0.0, w)
                o = w @ vv.nan_to_num(0.0, 0.0, 0.0)
                fin = torch.isfinite(vv)
                if not bool(fin.all()):     # what is seen and is not finite decides
                    for j in (~fin).any(1).nonzero()[:, 0].tolist():
                        o = torch.where(vis[:, j, None] & ~fin[j], o + vv[j], o)
                out[b, :, a], lse[b, :, a] = o, ln
                eps = hd * 2.0 ** -22 * scale * (qq.abs() @ kk.nan_to_num(0.0, 0.0, 0.0).abs().T).amax(1) + 2.0 ** -20
                mag = w.nan_to_num(0.0) @ vv.nan_to_num(0.0, 0.0, 0.0).abs()
                b_out[b, :, a] = (U8 + 2 * eps + 2.0 ** -19)[:, None] * mag + U8 * o.abs().nan_to_num(0.0, 0.0, 0.0) + 1e-30
                b_lse[b, :, a] = eps + 2.0 ** -19 + 2.0 ** -21 * ln.abs().nan_to_num(0.0, 0.0, 0.0)
    return out, lse, b_out, b_lse


def within(got, want, bound):
    """Largest error in units of its bound; NaN, infinities and finiteness have to agree."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]) and torch.equal(torch.isinf(got), inf)
    ok = torch.isfinite(want)
    if not bool(ok.any()):
        return 0.0
    return float(((got - want).abs()[ok] / bound[ok]).max())


# ----------------------------------------------------------------------- weights
def weights(q, lse, k, lens, path, decay, score, scale):
    """float64 score_out (entries beyond a length are score_out's own: NaN here) and its bound. path: list of lists."""
    B, cap, H, hd = k.shape
    G = q.shape[2] // H
    out = torch.full((B, H, cap), math.nan, dtype=torch.float64, device=q.device)
    bound = torch.ones_like(out)
    for b in range(B):
        m, p = int(lens[b]), path[b]
        for h in range(H):
            kk = k[b, :m, h].double()
            base = score[b, h, :m].double() * decay if decay != 0.0 else torch.zeros(m, dtype=torch.float64, device=q.device)
            tot, err = base.clone(), U24 * base.abs()
            for j, node in enumerate(p):
                last = m - len(p) + j
                for g in range(G):
                    ln = float(lse[b, node, h * G + g])
                    if ln == -math.inf:
                        continue
                    qq = q[b, node, h * G + g].double()
                    s = kk[:last + 1] @ qq * scale
                    w = torch.exp(s - ln)
                    tot[:last + 1] += w
                    e = hd * 2.0 ** -22 * scale * (kk[:last + 1].abs() @ qq.abs()) + 2.0 ** -20 + 2.0 ** -22 * (s.abs() + abs(ln))
                    err[:last + 1] += w * e
            out[b, h, :m] = tot
            bound[b, h, :m] = err + (len(p) * G + 2) * U24 * tot.abs() + 1e-30
    return out, bound


# ------------------------------------------------------------------------ verify
def verify(target, draft, tokens, parents, u, noise):
    """One sequence, float64 rows: (path, next token, how near to a tie the closest decision was)."""
    n = len(parents)
    path, cur, near = [0], 0, math.inf
    while True:
        r = target[cur].double()
        q = None if draft is None else draft[cur].double()
        z, found = 1.0, None
        for c in (c for c in range(n) if parents[c] == cur):
            t = int(tokens[c])
            lhs, rhs = float(u[c]) * (1.0 if q is None else float(q[t])) * z, float(r[t])
            near = min(near, abs(lhs - rhs) / max(lhs, rhs, 1e-30))
            if lhs < rhs:
                found = c
                break
            left = r.clone()
            if q is None:
                left[t] = 0.0
            else:
                left = (r / z - q).clamp(min=0.0)
            if float(left.sum()) > 0.0:
                r, z = left, float(left.sum())
        if found is None:
            score = torch.where(r > 0, r / noise.double(), torch.zeros_like(r))
            top = score.topk(min(2, score.numel())).values
            if top.numel() > 1 and float(top[0]) > 0:
                near = min(near, float((top[0] - top[1]) / top[0]))
            return path, int(score.argmax()), near
        path.append(found)
        cur = found


# ------------------------------------------------------------------------- evict
def evict_order(score, pos, n, keep, sink, newest):
    """Which of rows 0..n-1 stay: python floats, NaN as -inf, the lowest row first among equals."""
    rank = []
    for t in range(n):
        s = score[t]
        s = -math.inf if s != s else s
        if pos[t] < sink or pos[t] >= newest:
            s = math.inf
        rank.append((-s, t))
    return sorted(t for _, t in sorted(rank)[:keep])


def evict_moves(stay, n, keep):
    stay_set = set(stay)
    holes = [t for t in range(min(n, keep)) if t not in stay_set]
    movers = [t for t in stay if t >= keep]
    assert len(holes) == len(movers)
    return holes, movers
