"""Several answers to one filled prompt, a step of drafted trees: rf_fill_kv fills the prompt's cache, rf_norm_rope
writes its exact tail's keys and turns the step's queries and keys, rf_prefix_attention runs them in every layer,
rf_sample turns logits into the probabilities that rf_verify_draft takes, and rf_commit_draft appends what is kept.
Each call's outputs against its definition in 64 bits on the inputs that it had; then the step as CUDA graphs."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf
import synth
import test_sample_gpu as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
CFG = synth.FillConfig(name="fill, then answers", index=92, d=512, L=4, S=2, N=400, T=37, H=2, hd=128, rope_theta=5e5,
                       exact="uniform10", lam=0.03, calib_n=0)
B, G, V, CAP = 5, 5, 1003, 160
LENS = [0, 7, 64, 1, 130]
PARENTS = [-1, 0, 0, 2]
n = len(PARENTS)
HEADS = CFG.H * G
EPS = 1e-5


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _norm_desc(rows, n_q, n_k, ld_in, ld_out, offset=0):
    rope = rf.rf_rope_desc(n_rows=rows, n_heads=n_q + n_k, head_dim=CFG.hd, rot_dim=CFG.hd, ld_in=ld_in, ld_out=ld_out,
                           pos_offset=offset, theta=CFG.rope_theta)
    return rf.rf_norm_rope_desc(rope=rope, n_q_heads=n_q, eps=EPS)


def _check_norm_rope(x, gain, pos, y):
    """x, y [rows][heads][hd], gain [heads][hd]; the bounds of rf_norm_rope's own test."""
    x = x.double()
    want, mag = R.rope(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.double(), pos,
                       R.frequencies(CFG.hd, CFG.rope_theta), False)
    assert R.within(y, want, (2.0 ** -19.5 + 1.4e-6) * mag + R.U8 * want.abs() + 1e-30) <= 1.0


def _prompt():
    """The prompt's caches [L][N][H][hd] and the gains of its keys' norms: layers below S drawn, the others filled
    and, in the tail, written from projections. Exact rows among the filled ones stay as drawn."""
    c = CFG
    inp = {k: None if v is None else v.cuda() for k, v in synth.fill_inputs(c, device="cpu").items()}
    gains = R.randn((c.L, c.hd), 3, torch.float32, 0.2).add_(1.0).bfloat16()
    k, v = (R.randn((c.L, c.N, c.H, c.hd), seed) for seed in (1, 2))
    before = k.clone()
    d = rf.rf_fill_desc(d=c.d, L=c.L, S=c.S, N=c.N, T=c.T, n_kv_heads=c.H, head_dim=c.hd, rope_theta=c.rope_theta,
                        rms_eps=c.rms_eps, pos_offset=0, k_norm_gain=gains[c.S:].data_ptr())
    ws = torch.empty(rf.rf_fill_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    count, st = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    rf.rf_fill_kv(d, inp["x_S"], c.d, inp["mask"], inp["A"], inp["b"], inp["gain"], inp["Wk"], inp["Wv"], k, v, k.stride(0),
                  k.stride(1), count, st, ws, ws.numel())
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and int(count.item()) > 300
    tail = torch.arange(c.N - c.T, c.N, device=DEV)
    assert torch.equal(k[:, tail], before[:, tail]) and not torch.equal(k[c.S:, :c.N - c.T], before[c.S:, :c.N - c.T])
    filled = (k[c.S:] != before[c.S:]).flatten(2).any(-1)
    assert int(filled[0].sum()) == int(count.item())
    raw = R.randn((c.L, c.T, c.H, c.hd), 4, std=3.0)
    for l in range(c.L):
        rf.rf_norm_rope(_norm_desc(c.T, 0, c.H, raw.stride(1), k.stride(1), c.N - c.T), raw[l], None, gains[l], k[l, c.N - c.T:])
    torch.cuda.synchronize()
    for l in range(c.L):
        _check_norm_rope(raw[l], gains[l].expand(c.H, c.hd), tail, k[l, tail])
    assert torch.equal(k[:c.S, :c.N - c.T], before[:c.S, :c.N - c.T])
    return k, v, gains


class Step:
    """One step over the prompt and the sequences' own caches, everything allocated beforehand."""

    def __init__(self, kp, vp, gains, ws=None):
        c = CFG
        self.kp, self.vp, self.gk = kp, vp, gains
        self.gq = R.randn((c.L, c.hd), 6, torch.float32, 0.2).add_(1.0).bfloat16()
        self.k, self.v = (torch.full((c.L, B, CAP, c.H, c.hd), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        for i, x in enumerate((self.k, self.v)):
            for b, m in enumerate(LENS):
                x[:, b, :m] = R.randn((c.L, m, c.H, c.hd), 20 + 2 * b + i)
        self.raw = R.randn((c.L, B * n, (HEADS + 2 * c.H) * c.hd), 7, std=2.0)      # query, key and value heads of a row
        self.qkv = self.raw.clone()
        self.parents, self.plen, self.lens, self.status = _ints([PARENTS] * B), _ints([c.N]), _ints(LENS), _ints([0])
        self.next_pos = self.lens + c.N
        self.mask = torch.zeros((B, n, 1), dtype=torch.int64, device=DEV)
        self.positions = torch.zeros((B, n), dtype=torch.int32, device=DEV)
        self.out = torch.zeros((c.L, B, n, HEADS, c.hd), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros((c.L, B, n, HEADS), device=DEV)
        self.head = R.randn((HEADS * c.hd, V), 8, torch.float32, 0.3)
        self.logits, self.probs = torch.zeros((B * n, V), device=DEV), torch.zeros((B * n, V), device=DEV)
        f = lambda x: torch.tensor(x, device=DEV).repeat_interleave(n).contiguous()  # noqa: E731
        self.settings = dict(temperature=f([1.0, 0.7, 1.3, 0.0, 0.9]), top_k=f([0, 40, 300, 0, 1]).int(),
                             top_p=f([0.95, 1.0, 0.9, 1.0, 0.5]), min_p=f([0.0, 0.02, 0.0, 0.0, 0.0]))
        gen = torch.Generator(DEV).manual_seed(9)
        self.noise = torch.empty((B, V), device=DEV).exponential_(1.0, generator=gen).clamp_(min=1e-30)
        self.u = torch.rand((B, n), device=DEV, generator=gen)
        self.tokens = torch.randint(0, V, (B, n), device=DEV, generator=gen).int()
        self.path, self.n_path, self.token = _ints([[-9] * n] * B), _ints([-9] * B), _ints([-9] * B)
        qkv, s = self.qkv.view(c.L, B, n, HEADS + 2 * c.H, c.hd), self.k.stride()
        self.q, self.kd, self.vd = qkv[..., :HEADS, :], qkv[..., HEADS:HEADS + c.H, :], qkv[..., HEADS + c.H:, :]
        self.attn = rf.rf_prefix_attn_desc(
            attn=rf.rf_attn_desc(n_seqs=B, n_q_heads=HEADS, n_kv_heads=c.H, head_dim=c.hd, n_nodes=n, capacity=CAP,
                                 q_row_stride=self.q.stride(2), q_seq_stride=self.q.stride(1),
                                 draft_row_stride=self.kd.stride(2), draft_seq_stride=self.kd.stride(1), cache_row_stride=s[2],
                                 cache_seq_stride=s[1], out_row_stride=HEADS * c.hd, out_seq_stride=n * HEADS * c.hd,
                                 scale=c.hd ** -0.5),
            prefix_capacity=c.N, prefix_row_stride=kp.stride(1))
        self.norm = _norm_desc(B * n, HEADS, c.H, self.raw.stride(1), self.qkv.stride(1))
        self.sample = rf.rf_sample_desc(n_rows=B * n, vocab=V, ld_logits=V, ld_noise=V, ld_probs=V, dtype=rf.RF_F32)
        self.verify = rf.rf_verify_desc(n_seqs=B, n_nodes=n, vocab=V, ld_target=V, ld_draft=V, ld_noise=V)
        self.cache = rf.rf_cache_desc(n_layers=c.L, n_seqs=B, n_kv_heads=c.H, head_dim=c.hd, capacity=CAP, row_stride=s[2],
                                      seq_stride=s[1], layer_stride=s[0])
        need = rf.rf_prefix_attn_workspace_bytes(self.attn)
        self.ws = torch.empty(need, dtype=torch.uint8, device=DEV) if ws is None else ws

    def attend(self):
        rf.rf_tree_build(B, n, self.parents, self.next_pos, self.mask, self.positions, self.status)
        for l in range(CFG.L):
            rf.rf_norm_rope(self.norm, self.raw[l], self.gq[l], self.gk[l], self.qkv[l], self.positions)
            rf.rf_prefix_attention(self.attn, self.q[l], self.kp[l], self.vp[l], self.plen, self.k[l], self.v[l], self.lens,
                                   self.kd[l], self.vd[l], self.mask, self.out[l], self.lse[l], self.status, self.ws,
                                   self.ws.numel())
        torch.matmul(self.out.view(CFG.L, B * n, -1).sum(0).float(), self.head, out=self.logits)

    def choose(self):
        rf.rf_sample(self.sample, self.logits, **self.settings, probs=self.probs, dev_status=self.status)
        rf.rf_verify_draft(self.verify, self.probs, None, self.tokens, self.parents, self.u, self.noise, self.path,
                           self.n_path, self.token, self.status)

    def keep(self):
        rf.rf_commit_draft(self.cache, n, self.kd.stride(2), self.kd.stride(1), self.kd.stride(0), self.path, self.n_path,
                           self.lens, self.next_pos, self.kd, self.vd, self.k, self.v, None, None, self.lens, self.next_pos,
                           self.status)

    def all(self):
        self.attend()
        self.choose()
        self.keep()

    def state(self):
        names = ("k", "v", "qkv", "out", "lse", "logits", "probs", "path", "n_path", "token", "lens", "next_pos", "status")
        return [getattr(self, x) for x in names]


def test_answers_to_one_prompt():
    c = CFG
    kp, vp, gains = _prompt()
    s = Step(kp, vp, gains)
    s.attend()
    torch.cuda.synchronize()
    assert s.positions.tolist() == [[c.N + m + d for d in (0, 1, 1, 2)] for m in LENS]
    seen = R.ancestors(PARENTS)[None].expand(B, -1, -1)
    rows = lambda x: x.reshape(B * n, -1, c.hd)  # noqa: E731
    for l in range(c.L):
        raw = s.raw[l].view(B * n, HEADS + 2 * c.H, c.hd)
        gain = torch.cat([s.gq[l].expand(HEADS, c.hd), gains[l].expand(c.H, c.hd)])
        _check_norm_rope(raw[:, :HEADS + c.H], gain, s.positions.flatten(), torch.cat([rows(s.q[l]), rows(s.kd[l])], 1))
        assert torch.equal(rows(s.vd[l]), raw[:, HEADS + c.H:])
        long = [torch.zeros((B, c.N + CAP, c.H, c.hd), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        for x, p, own in zip(long, (kp[l], vp[l]), (s.k[l], s.v[l])):
            x[:, :c.N] = p
            for b, m in enumerate(LENS):
                x[b, c.N:c.N + m] = own[b, :m]
        want, wl, bo, bl = R.attention(s.q[l], *long, s.kd[l], s.vd[l], [c.N + m for m in LENS], seen, c.hd ** -0.5)
        assert R.within(s.out[l], want, bo) <= 1.0 and R.within(s.lse[l], wl, bl) <= 1.0
    s.choose()
    torch.cuda.synchronize()
    t = {k: v.tolist() for k, v in s.settings.items()}
    for r in range(B * n):
        order, p = S._keep(s.logits[r].double(), t["temperature"][r], t["top_k"][r], t["top_p"][r], t["min_p"][r])
        want = torch.zeros(V, dtype=torch.float64, device=DEV).index_put_((order,), p)
        big = want > 2.0 ** -100
        assert torch.equal((s.probs[r] > 0) & big, big) and bool((s.probs[r][want == 0] == 0).all())
        assert bool(((s.probs[r].double() - want).abs()[big] <= ((2.0 ** -21 + (V / 512 + 32) * R.U24) * want)[big]).all())
    path, count, token = s.path.tolist(), s.n_path.tolist(), s.token.tolist()
    old_k, old_v = s.k.clone(), s.v.clone()
    s.keep()
    torch.cuda.synchronize()
    for b, m in enumerate(LENS):
        nodes = path[b][:count[b]]
        assert count[b] >= 1 and nodes[0] == 0 and path[b][count[b]:] == [-1] * (n - count[b])
        assert float(s.probs[b * n + nodes[-1], token[b]]) > 0.0               # the next token is one that stayed
        assert s.lens[b].item() == m + count[b] and s.next_pos[b].item() == c.N + m + count[b]
        assert torch.equal(s.k[:, b, m:m + count[b]], s.kd[:, b, nodes]) and torch.equal(s.v[:, b, m:m + count[b]], s.vd[:, b, nodes])
        assert torch.equal(s.k[:, b, :m], old_k[:, b, :m]) and torch.equal(s.v[:, b, :m], old_v[:, b, :m])
        assert bool(torch.isnan(s.k[:, b, m + count[b]:].float()).all())
    assert int(s.status.item()) == 0


def _bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


def test_steps_in_cuda_graphs_that_share_a_workspace_give_the_same_bits():
    kp, vp, gains = _prompt()
    plain, first = Step(kp, vp, gains), Step(kp, vp, gains)
    second = Step(kp, vp, gains, ws=first.ws)
    second.raw.neg_()                                   # another step's rows
    other = Step(kp, vp, gains)
    other.raw.neg_()
    start = [x.clone() for x in first.state()]
    for x in (plain, other):
        x.all()
    torch.cuda.synchronize()
    graphs = []
    for x in (first, second):
        x.all()                                         # first calls set kernel attributes, outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.all()
        graphs.append(g)
    for turn in range(3):
        for x in (first, second):
            for y, z in zip(x.state(), start):
                y.copy_(z)
        first.ws.fill_(0xFF)
        for g in graphs if turn != 1 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for x, want in ((first, plain), (second, other)):
            for y, z in zip(x.state(), want.state()):
                assert torch.equal(_bits(y), _bits(z))
    assert int(plain.status.item()) == 0 and not torch.equal(_bits(plain.out), _bits(other.out))


def test_a_step_on_another_stream_gives_the_same_bits():
    kp, vp, gains = _prompt()
    plain, aside = Step(kp, vp, gains), Step(kp, vp, gains)
    plain.all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        aside.all()
    side.synchronize()
    for y, z in zip(aside.state(), plain.state()):
        assert torch.equal(_bits(y), _bits(z))
