"""rf_fill_kv fills a cache, and the decoding operators take it from there: attention of a drafted tree in every layer,
verification, commit, accumulated weights, eviction, and attention over what is left; call by call, and as one CUDA
graph with the same bits."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
CFG = synth.FillConfig(name="fill, then decode", index=91, d=512, L=4, S=2, N=400, T=37, H=2, hd=128, rope_theta=5e5,
                       exact="uniform10", lam=0.03, calib_n=0)
G, SPARE, KEEP, V = 3, 16, 256, 64
PARENTS = [-1, 0, 0, 2, 3, 3]
ACCEPTED = [0, 2, 3, 5]
N_NODES = len(PARENTS)


def _filled():
    """Caches [L][1][N + SPARE][H][hd], exact rows drawn, the others filled; what lies beyond N rows is NaN."""
    c = CFG
    inp = {k: None if v is None else v.cuda() for k, v in synth.fill_inputs(c, device="cpu").items()}
    caches = []
    for seed in (1, 2):
        x = torch.full((c.L, 1, c.N + SPARE, c.H, c.hd), math.nan, dtype=torch.bfloat16, device=DEV)
        x[:, :, :c.N] = R.randn((c.L, 1, c.N, c.H, c.hd), seed)
        caches.append(x)
    before = [x.clone() for x in caches]
    d = rf.rf_fill_desc(d=c.d, L=c.L, S=c.S, N=c.N, T=c.T, n_kv_heads=c.H, head_dim=c.hd, rope_theta=c.rope_theta,
                        rms_eps=c.rms_eps, pos_offset=0)
    ws = torch.empty(rf.rf_fill_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    n, st = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    rf.rf_fill_kv(d, inp["x_S"], c.d, inp["mask"], inp["A"], inp["b"], inp["gain"], inp["Wk"], inp["Wv"], *caches,
                  caches[0].stride(0), caches[0].stride(2), n, st, ws, ws.numel())
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and int(n.item()) > 300
    for x, y in zip(caches, before):                    # it did fill, up to the last prefix row and no further
        assert not torch.equal(x[c.S:, :, :c.N], y[c.S:, :, :c.N]) and bool(torch.isfinite(x[:, :, :c.N].float()).all())
        assert torch.equal(x[:c.S, :, :c.N], y[:c.S, :, :c.N]) and bool(torch.isnan(x[:, :, c.N:].float()).all())
    return caches


class Step:
    """One decoding step over a cache, everything allocated beforehand."""

    def __init__(self, k, v):
        c, n = CFG, N_NODES
        self.k, self.v = k.clone(), v.clone()
        cap, heads = k.shape[2], c.H * G
        self.q, self.kd, self.vd = (R.randn((c.L, 1, n, h, c.hd), 10 + i) for i, h in enumerate((heads, c.H, c.H)))
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        self.lens, self.next_pos, self.parents, self.status = ints([c.N]), ints([c.N]), ints([PARENTS]), ints([0])
        self.mask = torch.zeros((1, n, 1), dtype=torch.int64, device=DEV)
        self.positions = torch.zeros((1, n), dtype=torch.int32, device=DEV)
        self.out = torch.zeros((2, c.L, 1, n, heads, c.hd), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros((2, c.L, 1, n, heads), device=DEV)
        self.tokens = ints([[0] + [10 + i for i in range(1, n)]])
        self.target = torch.zeros((1, n, V), device=DEV)
        for a, b in zip(ACCEPTED, ACCEPTED[1:]):
            self.target[0, a, 10 + b] = 1.0
        self.target[0, ACCEPTED[-1], 7] = 1.0
        self.u, self.noise = torch.full((1, n), 0.5, device=DEV), torch.ones((1, V), device=DEV)
        self.path, self.n_path, self.token = ints([[-9] * n]), ints([-9]), ints([-9])
        self.score = torch.rand((c.L, 1, c.H, cap), device=DEV, generator=torch.Generator(DEV).manual_seed(3))
        self.pos = torch.arange(cap, dtype=torch.int32, device=DEV).expand(c.L, 1, c.H, cap).contiguous()
        s = k.stride()
        self.cache = rf.rf_cache_desc(n_layers=c.L, n_seqs=1, n_kv_heads=c.H, head_dim=c.hd, capacity=cap, row_stride=s[2],
                                      seq_stride=s[1], layer_stride=s[0])
        self.attn = rf.rf_attn_desc(
            n_seqs=1, n_q_heads=heads, n_kv_heads=c.H, head_dim=c.hd, n_nodes=n, capacity=cap, q_row_stride=heads * c.hd,
            q_seq_stride=n * heads * c.hd, draft_row_stride=c.H * c.hd, draft_seq_stride=n * c.H * c.hd,
            cache_row_stride=s[2], cache_seq_stride=s[1], out_row_stride=heads * c.hd, out_seq_stride=n * heads * c.hd,
            scale=c.hd ** -0.5)
        self.verify = rf.rf_verify_desc(n_seqs=1, n_nodes=n, vocab=V, ld_target=V, ld_draft=V, ld_noise=V)
        self.ws = torch.empty(max(rf.rf_attn_workspace_bytes(self.attn), rf.rf_evict_workspace_bytes(self.cache, KEEP)),
                              dtype=torch.uint8, device=DEV)

    def attend(self, turn):
        for l in range(CFG.L):
            rf.rf_tree_attention(self.attn, self.q[l], self.k[l], self.v[l], self.lens, self.kd[l], self.vd[l], self.mask,
                                 self.out[turn, l], self.lse[turn, l], self.status, self.ws, self.ws.numel())

    def accept(self):
        rf.rf_verify_draft(self.verify, self.target, None, self.tokens, self.parents, self.u, self.noise, self.path,
                           self.n_path, self.token, self.status)
        rf.rf_commit_draft(self.cache, N_NODES, self.kd.stride(2), self.kd.stride(1), self.kd.stride(0), self.path,
                           self.n_path, self.lens, self.next_pos, self.kd, self.vd, self.k, self.v, self.score, self.pos,
                           self.lens, self.next_pos, self.status)

    def weigh(self):
        for l in range(CFG.L):
            rf.rf_attn_weights(self.attn, self.q[l], self.lse[0, l], self.path, self.n_path, self.k[l], self.lens, 0.5,
                               self.score[l], self.score[l], self.status, self.ws, self.ws.numel())

    def evict(self):
        rf.rf_evict(self.cache, KEEP, 4, 40, self.lens, self.next_pos, self.k, self.v, self.score, self.pos, self.score,
                    self.pos, self.lens, self.status, self.ws, self.ws.numel())

    def build(self):
        rf.rf_tree_build(1, N_NODES, self.parents, self.next_pos, self.mask, self.positions, self.status)

    def all(self):
        self.build()
        self.attend(0)
        self.accept()
        self.weigh()
        self.evict()
        self.attend(1)

    def state(self):
        names = ("k", "v", "out", "lse", "path", "n_path", "token", "score", "pos", "lens", "next_pos", "positions", "status")
        return [getattr(self, x) for x in names]


def _check_attention(s, turn, lens):
    seen = R.ancestors(PARENTS)[None]
    for l in range(CFG.L):
        want, wl, bo, bl = R.attention(s.q[l], s.k[l], s.v[l], s.kd[l], s.vd[l], lens, seen, CFG.hd ** -0.5)
        assert R.within(s.out[turn, l], want, bo) <= 1.0 and R.within(s.lse[turn, l], wl, bl) <= 1.0


def test_decoding_takes_over_where_the_fill_ends():
    c = CFG
    k, v = _filled()
    s = Step(k, v)
    s.build()
    s.attend(0)
    torch.cuda.synchronize()
    _check_attention(s, 0, [c.N])
    assert s.positions.tolist() == [[c.N + d for d in (0, 1, 1, 2, 3, 3)]]
    s.accept()
    torch.cuda.synchronize()
    m = c.N + len(ACCEPTED)
    assert s.path.tolist() == [ACCEPTED + [-1, -1]] and s.token.tolist() == [7] and s.lens.tolist() == [m]
    assert torch.equal(s.k[:, :, :c.N], k[:, :, :c.N]) and torch.equal(s.k[:, 0, c.N:m], s.kd[:, 0, ACCEPTED])
    assert torch.equal(s.v[:, 0, c.N:m], s.vd[:, 0, ACCEPTED]) and bool(torch.isnan(s.v[:, 0, m:].float()).all())
    before = s.score.clone()
    s.weigh()
    torch.cuda.synchronize()
    for l in range(c.L):
        want, bound = R.weights(s.q[l], s.lse[0, l], s.k[l], [m], [ACCEPTED], 0.5, before[l], c.hd ** -0.5)
        assert R.within(s.score[l][..., :m], want[..., :m], bound[..., :m]) <= 1.0
    score, pos, old = s.score.tolist(), s.pos.tolist(), (s.k.clone(), s.v.clone())
    s.evict()
    torch.cuda.synchronize()
    assert s.lens.tolist() == [KEEP]
    for l in range(c.L):
        for h in range(c.H):
            stay = R.evict_order(score[l][0][h], pos[l][0][h], m, KEEP, 4, m - 40)
            assert sorted(s.pos[l, 0, h, :KEEP].tolist()) == [pos[l][0][h][t] for t in stay]
            rows = s.pos[l, 0, h, :KEEP].long()         # positions were row numbers
            assert torch.equal(s.k[l, 0, :KEEP, h], old[0][l, 0, rows, h]) and torch.equal(s.v[l, 0, :KEEP, h], old[1][l, 0, rows, h])
    s.attend(1)
    torch.cuda.synchronize()
    _check_attention(s, 1, [KEEP])
    assert int(s.status.item()) == 0


def test_a_whole_step_in_a_cuda_graph_gives_the_same_bits():
    k, v = _filled()
    plain, captured = Step(k, v), Step(k, v)
    plain.all()
    torch.cuda.synchronize()
    start = [x.clone() for x in captured.state()]
    captured.all()                                      # first calls set kernel attributes, outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured.all()
    for _ in range(3):
        for x, y in zip(captured.state(), start):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured.state(), plain.state()):
            t = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(x.view(t), y.view(t))
    assert int(plain.status.item()) == 0
