"""Decoding from a KV cache by drafting trees: rotation, attention, verification, cache,
accumulated weights and eviction in one loop.

A small random transformer (RMSNorm, attention with grouped heads, a gated feed-forward
block) decodes for a few sequences of different lengths. Each step drafts a tree of
tokens per sequence, runs the tree through every layer in one pass, keeps the branch
that the model itself would have taken, and appends its rows to the cache. Where a budget
is given, rows of little accumulated attention weight leave the cache after each step.

    python examples/decode_draft.py [--tokens 24] [--nodes 8] [--budget 0]

Drafts come from a table of what followed each token before: cheap, and often wrong. With
``sample=False`` the model's distribution is the argmax alone, so any tree gives the
tokens that decoding one by one gives.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import ridge_map_kv_gb300 as rf  # noqa: E402


@dataclasses.dataclass(frozen=True)
class Config:
    vocab: int = 211
    layers: int = 4
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    width: int = 256
    theta: float = 1.0e4

    @property
    def group(self) -> int:
        return self.q_heads // self.kv_heads


class Model:
    """Random weights; everything but attention and rotation is plain torch."""

    def __init__(self, cfg: Config, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device=device).mul_(s[-1] ** -0.5).bfloat16()  # noqa: E731
        c = self.cfg = cfg
        heads = c.q_heads + 2 * c.kv_heads
        self.embed = torch.randn((c.vocab, c.width), generator=g, device=device).bfloat16()
        self.qkv = [rand(heads * c.head_dim, c.width) for _ in range(c.layers)]
        self.out = [rand(c.width, c.q_heads * c.head_dim) for _ in range(c.layers)]
        self.up = [rand(4 * c.width, c.width) for _ in range(c.layers)]
        self.down = [rand(c.width, 2 * c.width) for _ in range(c.layers)]
        self.head = torch.randn((c.vocab, c.width), generator=g, device=device).mul_(0.3).bfloat16()

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-5).to(x.dtype)


class Decoder:
    """A cache of all layers for a batch of sequences, and the step that extends it."""

    def __init__(self, model: Model, seqs: int, capacity: int, max_nodes: int, budget: int = 0, sink: int = 4,
                 recent: int = 16, device: str = "cuda"):
        c, self.model = model.cfg, model
        self.seqs, self.capacity, self.max_nodes = seqs, capacity, max_nodes
        self.budget, self.sink, self.recent = budget, sink, recent
        cache = (c.layers, seqs, capacity, c.kv_heads, c.head_dim)
        self.k = torch.zeros(cache, dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        draft = (c.layers, seqs, max_nodes, c.kv_heads, c.head_dim)
        self.kd = torch.empty(draft, dtype=torch.bfloat16, device=device)
        self.vd = torch.empty_like(self.kd)
        self.score = torch.zeros((c.layers, seqs, c.kv_heads, capacity), device=device)
        self.pos = torch.zeros((c.layers, seqs, c.kv_heads, capacity), dtype=torch.int32, device=device)
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self.lens, self.next_pos, self.n_path, self.token, self.status = (ints(seqs), ints(seqs), ints(seqs),
                                                                          ints(seqs), ints(1))
        self.cache_desc = rf.rf_cache_desc(
            n_layers=c.layers, n_seqs=seqs, n_kv_heads=c.kv_heads, head_dim=c.head_dim, capacity=capacity,
            row_stride=self.k.stride(2), seq_stride=self.k.stride(1), layer_stride=self.k.stride(0))
        size = max(rf.rf_attn_workspace_bytes(self._attn_desc(n)) for n in (1, max_nodes))
        if budget:
            size = max(size, rf.rf_evict_workspace_bytes(self.cache_desc, budget))
        self.ws = torch.empty(max(size, 256), dtype=torch.uint8, device=device)

    def _attn_desc(self, n: int) -> rf.rf_attn_desc:
        c = self.model.cfg
        w = (c.q_heads + c.kv_heads) * c.head_dim      # rows of rotated queries and keys
        return rf.rf_attn_desc(
            n_seqs=self.seqs, n_q_heads=c.q_heads, n_kv_heads=c.kv_heads, head_dim=c.head_dim, n_nodes=n,
            capacity=self.capacity, q_row_stride=w, q_seq_stride=n * w, draft_row_stride=self.kd.stride(2),
            draft_seq_stride=self.kd.stride(1), cache_row_stride=self.k.stride(2), cache_seq_stride=self.k.stride(1),
            out_row_stride=c.q_heads * c.head_dim, out_seq_stride=n * c.q_heads * c.head_dim, scale=c.head_dim ** -0.5)

    def forward(self, tokens, parents):
        """The model's logits [seqs][n][vocab] after each node of the trees; the nodes' K and V wait in kd, vd."""
        c, m = self.model.cfg, self.model
        B, n = tokens.shape
        mask = torch.empty((B, n, (n + 63) // 64), dtype=torch.int64, device=tokens.device)
        positions = torch.empty((B, n), dtype=torch.int32, device=tokens.device)
        rf.rf_tree_build(B, n, parents, self.next_pos, mask, positions, self.status)
        desc = self._attn_desc(n)
        qk_heads = c.q_heads + c.kv_heads
        turn = rf.rf_rope_desc(n_rows=B * n, n_heads=qk_heads, head_dim=c.head_dim, rot_dim=c.head_dim,
                               ld_in=(qk_heads + c.kv_heads) * c.head_dim, ld_out=qk_heads * c.head_dim, theta=c.theta)
        x = m.embed[tokens.long()]
        self.kept = []                                   # per layer: queries and statistics, for the weights
        for l in range(c.layers):
            qkv = m.norm(x) @ m.qkv[l].T
            qk = torch.empty((B, n, qk_heads, c.head_dim), dtype=torch.bfloat16, device=x.device)
            rf.rf_rope(turn, qkv, qk, positions)
            self.kd[l, :, :n] = qk[:, :, c.q_heads:]
            self.vd[l, :, :n] = qkv.view(B, n, -1, c.head_dim)[:, :, qk_heads:]
            out = torch.empty((B, n, c.q_heads * c.head_dim), dtype=torch.bfloat16, device=x.device)
            lse = torch.empty((B, n, c.q_heads), device=x.device)
            rf.rf_tree_attention(desc, qk, self.k[l], self.v[l], self.lens, self.kd[l], self.vd[l], mask, out, lse,
                                 self.status, self.ws, self.ws.numel())
            self.kept.append((qk, lse))
            x = x + out @ m.out[l].T
            gate, val = (m.norm(x) @ m.up[l].T).chunk(2, -1)
            x = x + (torch.nn.functional.silu(gate) * val) @ m.down[l].T
        return (m.norm(x) @ m.head.T).float()

    def commit(self, path, n_path, n: int):
        """The accepted nodes' rows join the cache; their weights are added up; light rows leave."""
        c = self.model.cfg
        rf.rf_commit_draft(self.cache_desc, n, self.kd.stride(2), self.kd.stride(1), self.kd.stride(0), path, n_path,
                           self.lens, self.next_pos, self.kd, self.vd, self.k, self.v, self.score, self.pos, self.lens,
                           self.next_pos, self.status)
        if not self.budget:
            return
        desc = self._attn_desc(n)
        for l in range(c.layers):
            q, lse = self.kept[l]
            rf.rf_attn_weights(desc, q, lse, path, n_path, self.k[l], self.lens, 1.0, self.score[l], self.score[l],
                               self.status, self.ws, self.ws.numel())
        rf.rf_evict(self.cache_desc, self.budget, self.sink, self.recent, self.lens, self.next_pos, self.k, self.v,
                    self.score, self.pos, self.score, self.pos, self.lens, self.status, self.ws, self.ws.numel())

    def prompt(self, tokens):
        """Takes prompts of one length, [seqs][n], rows in order; returns the next tokens."""
        B, n = tokens.shape
        chain = torch.arange(-1, n - 1, dtype=torch.int32, device=tokens.device).expand(B, n).contiguous()
        logits = self.forward(tokens, chain)
        path = torch.arange(n, dtype=torch.int32, device=tokens.device).expand(B, n).contiguous()
        self.commit(path, torch.full((B,), n, dtype=torch.int32, device=tokens.device), n)
        return logits[:, -1].argmax(-1).to(torch.int32)

    def step(self, tokens, parents, generator=None, sample: bool = False):
        """One step: tokens [seqs][n] int32 with node 0 the last token of each sequence. Returns the accepted nodes
        [seqs][n] (-1 behind the last), their numbers and each sequence's next token."""
        B, n = tokens.shape
        logits = self.forward(tokens, parents)
        if sample:
            probs = torch.softmax(logits, -1)
        else:
            probs = torch.nn.functional.one_hot(logits.argmax(-1), logits.shape[-1]).float()
        u = torch.rand((B, n), generator=generator, device=tokens.device)
        noise = torch.empty((B, probs.shape[-1]), device=tokens.device).exponential_(1.0, generator=generator)
        path = torch.empty((B, n), dtype=torch.int32, device=tokens.device)
        V = probs.shape[-1]
        desc = rf.rf_verify_desc(n_seqs=B, n_nodes=n, vocab=V, ld_target=V, ld_draft=V, ld_noise=V)
        # drafted outright, without probabilities of their own
        rf.rf_verify_draft(desc, probs, None, tokens, parents, u, noise, path, self.n_path, self.token, self.status)
        self.commit(path, self.n_path, n)
        return path, self.n_path, self.token


def tree(table, token: int, n: int, vocab: int):
    """Tokens and parents of a tree of n nodes: what followed each token before, breadth first, the most recent first;
    other tokens where nothing is known."""
    tok, par = [int(token)], [-1]
    at = 0
    while len(tok) < n:
        known = table.get(tok[at], [])[-2:][::-1] or [(tok[at] * 7 + 3) % min(97, vocab)]
        for x in known[: n - len(tok)]:
            tok.append(int(x))
            par.append(at)
        at += 1
    return tok, par


def draft(table, last, n: int, vocab: int):
    """A tree of n nodes for each sequence."""
    tokens, parents = zip(*(tree(table, int(t), n, vocab) for t in last))
    return (torch.tensor(tokens, dtype=torch.int32, device="cuda"), torch.tensor(parents, dtype=torch.int32, device="cuda"))


def capacity(n0: int, n_tokens: int, nodes: int, budget: int) -> int:
    """Cache rows that any sequence may need. Every step gives the slowest sequence a token at least, so there are fewer
    than n_tokens; each may add all nodes to the fastest, of which a budget leaves its rows until the next step."""
    most = n0 + n_tokens * nodes
    return min(most, max(n0, budget + nodes)) if budget else most


def generate(model: Model, prompts, n_tokens: int, nodes: int, budget: int = 0, sample: bool = False, seed: int = 1):
    """Decodes n_tokens (or a few more) for every prompt; returns lists of tokens, the steps taken and the decoder."""
    B, n0 = prompts.shape
    dec = Decoder(model, B, capacity(n0, n_tokens, nodes, budget), max(nodes, n0), budget)
    g = torch.Generator(device="cuda").manual_seed(seed)
    last = dec.prompt(prompts)
    out = [[int(x)] for x in last]
    table: dict[int, list[int]] = {}
    steps = 0
    while min(len(o) for o in out) < n_tokens:
        tokens, parents = draft(table, last, nodes, model.cfg.vocab)
        path, n_path, nxt = dec.step(tokens, parents, g, sample)
        steps += 1
        tok, pth, cnt, last = tokens.tolist(), path.tolist(), n_path.tolist(), nxt.clone()
        for b in range(B):
            new = [tok[b][i] for i in pth[b][1:cnt[b]]] + [int(last[b])]
            for a, x in zip([tok[b][0]] + new, new):
                known = table.setdefault(a, [])
                if x in known:
                    known.remove(x)
                known.append(x)
            out[b] += new
    assert int(dec.status.item()) == 0, rf.rf_status_string(int(dec.status.item()))
    return [o[:n_tokens] for o in out], steps, dec


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--nodes", type=int, default=8)
    ap.add_argument("--budget", type=int, default=0, help="cache rows per head that stay after a step (0: all)")
    ap.add_argument("--sample", action="store_true")
    a = ap.parse_args()
    model = Model(Config())
    prompts = torch.randint(0, model.cfg.vocab, (3, 40), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    out, steps, dec = generate(model, prompts, a.tokens, a.nodes, a.budget, a.sample)
    for o in out:
        print(*o)
    print(f"{a.tokens} tokens of each sequence in {steps} steps; cache rows {dec.lens.tolist()}")


if __name__ == "__main__":
    main()
