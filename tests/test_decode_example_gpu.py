"""The decoding operators together, as examples/decode_draft.py runs them."""
import os
import sys

import pytest
import torch

import ridge_map_kv_gb300 as rf

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import decode_draft
    return decode_draft


def _logits(model, tokens):
    """The model's logits after the last of a list of tokens: the whole sequence in fp32 torch."""
    c = model.cfg
    inv = c.theta ** (-torch.arange(0, c.head_dim, 2, device="cuda").double() / c.head_dim)
    f = lambda x: x.float()  # noqa: E731
    x = f(model.embed[torch.tensor(tokens, device="cuda")])
    T = len(tokens)
    ang = torch.arange(T, device="cuda").double()[:, None] * inv
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    for l in range(c.layers):
        h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)
        qkv = (h @ f(model.qkv[l]).T).view(T, -1, c.head_dim)
        a, b = qkv[..., :c.head_dim // 2], qkv[..., c.head_dim // 2:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        q, k, v = rot[:, :c.q_heads], rot[:, c.q_heads:c.q_heads + c.kv_heads], qkv[:, c.q_heads + c.kv_heads:]
        k, v = k.repeat_interleave(c.group, 1), v.repeat_interleave(c.group, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * c.head_dim ** -0.5
        s = s.masked_fill(~torch.ones((T, T), device="cuda").tril().bool(), float("-inf"))
        o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(T, -1)
        x = x + o @ f(model.out[l]).T
        gate, val = ((x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)) @ f(model.up[l]).T).chunk(2, -1)
        x = x + (torch.nn.functional.silu(gate) * val) @ f(model.down[l]).T
    return (x[-1] * torch.rsqrt(x[-1].square().mean() + 1e-5)) @ f(model.head).T


def test_every_node_of_a_tree_sees_its_own_sequence(ex):
    """Logits after each node of random trees, over two steps with an accepted branch between them, against the whole
    sequence of that node in fp32. About ten bf16 roundings of 2^-8 / sqrt(3) each in every one of four layers add up to
    1.5 % of the logits' norm; 5 % is allowed. A wrong mask, position, row or length changes them altogether."""
    model = ex.Model(ex.Config())
    g = torch.Generator().manual_seed(4)
    B, n0, n = 3, 37, 11
    prompts = torch.randint(0, model.cfg.vocab, (B, n0), generator=g).to(torch.int32).cuda()
    dec = ex.Decoder(model, B, n0 + 30, n0)
    dec.prompt(prompts)
    seqs = [p.tolist() for p in prompts]
    for _ in range(2):
        tokens = torch.randint(0, model.cfg.vocab, (B, n), generator=g).to(torch.int32)
        parents = [[-1] + [int(torch.randint(max(0, i - 3), i, (1,), generator=g)) for i in range(1, n)] for _ in range(B)]
        got = dec.forward(tokens.cuda(), torch.tensor(parents, dtype=torch.int32).cuda())
        lines = []
        for b in range(B):
            line = [[0]]
            for i in range(1, n):
                line.append(line[parents[b][i]] + [i])
            lines.append(line)
            for i in range(n):
                want = _logits(model, seqs[b] + [int(tokens[b, j]) for j in line[i]])
                assert float((got[b, i] - want).norm() / want.norm()) <= 0.05, (b, i)
        path = torch.full((B, n), -1, dtype=torch.int32)
        for b in range(B):
            keep = lines[b][n - 1 - b]
            path[b, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            seqs[b] += [int(tokens[b, j]) for j in keep]
        dec.commit(path.cuda(), (path >= 0).sum(1).int().cuda(), n)
        assert dec.lens.tolist() == [len(s) for s in seqs] == dec.next_pos.tolist()
    assert int(dec.status.item()) == 0


def test_a_step_accepts_the_models_own_branch(ex):
    """Without sampling a tree that holds the tokens of one-by-one decoding (the model's own, fed back) is accepted along
    that branch, and the next token is the one that follows."""
    model = ex.Model(ex.Config())
    prompt = torch.randint(0, model.cfg.vocab, (1, 30), generator=torch.Generator().manual_seed(7)).to(torch.int32).cuda()
    dec = ex.Decoder(model, 1, 60, 30)
    first = int(dec.prompt(prompt)[0])
    probe = ex.Decoder(model, 1, 60, 30)
    probe.prompt(prompt)
    # the branch: each token is the argmax after the ones before, as a tree pass of this shape gives it
    branch = [first]
    parents = torch.tensor([[-1, 0, 0, 2, 3, 3]], dtype=torch.int32).cuda()
    where = [0, 2, 3, 5]                    # the branch's nodes among others
    for depth in range(4):
        tok = torch.full((1, 6), 1, dtype=torch.int32)
        for i, w in enumerate(where[:len(branch)]):
            tok[0, w] = branch[i]
        logits = probe.forward(tok.cuda(), parents)
        branch.append(int(logits[0, where[depth]].argmax()))
    tok = torch.zeros((1, 6), dtype=torch.int32)
    for i, w in enumerate(where):
        tok[0, w] = branch[i]
    for w in (1, 4):                        # siblings that are not the model's choice
        tok[0, w] = (branch[1 if w == 1 else 3] + 1) % model.cfg.vocab
    path, cnt, nxt = dec.step(tok.cuda(), parents)
    assert path.tolist() == [where + [-1, -1]] and cnt.tolist() == [4] and nxt.tolist() == [branch[4]]


def test_decoding_with_a_budget_keeps_sinks_recent_rows_and_the_budget(ex):
    model = ex.Model(ex.Config())
    prompts = torch.randint(0, model.cfg.vocab, (2, 50), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    out, steps, dec = ex.generate(model, prompts, 30, 6, budget=40, sample=True)
    assert all(len(o) == 30 for o in out) and all(0 <= t < model.cfg.vocab for o in out for t in o)
    assert dec.lens.tolist() == [40, 40]
    nxt = dec.next_pos.tolist()
    for b in range(2):
        for l in range(model.cfg.layers):
            for h in range(model.cfg.kv_heads):
                held = set(dec.pos[l, b, h, :40].tolist())
                assert len(held) == 40 and max(held) < nxt[b]
                assert set(range(dec.sink)) <= held and set(range(nxt[b] - dec.recent, nxt[b])) <= held
                score = dec.score[l, b, h, :40]
                assert bool(torch.isfinite(score).all()) and float(score.min()) >= 0.0


def test_sampled_decoding_repeats_with_its_seed(ex):
    model = ex.Model(ex.Config())
    prompts = torch.randint(0, model.cfg.vocab, (2, 20), generator=torch.Generator().manual_seed(6)).to(torch.int32).cuda()
    a = ex.generate(model, prompts, 12, 7, sample=True, seed=3)
    b = ex.generate(model, prompts, 12, 7, sample=True, seed=3)
    assert a[0] == b[0] and a[1] == b[1] and rf.rf_last_error() == ""


@pytest.mark.parametrize("budget", [0, 32])
def test_sequences_that_accept_unevenly_fit_the_cache(ex, monkeypatch, budget):
    """Sequence 0 accepts every node of every step, sequence 1 only its last token: the model's logits are replaced, the
    rows are its own. The cache holds both until the slow one is done."""
    nodes, n0, n_tokens = 8, 40, 24
    forward = ex.Decoder.forward

    def steered(self, tokens, parents):
        logits = torch.zeros_like(forward(self, tokens, parents))
        follow = torch.cat([tokens[0, 1:], tokens.new_zeros(1)]).long()
        logits[0, torch.arange(tokens.shape[1]), follow] = 10.0
        logits[1, :, 200] = 10.0                    # never drafted
        return logits

    def chain(table, last, n, vocab):
        tokens = [[int(t)] + list(range(1, n)) for t in last]
        parents = [list(range(-1, n - 1))] * len(tokens)
        return torch.tensor(tokens, dtype=torch.int32).cuda(), torch.tensor(parents, dtype=torch.int32).cuda()

    monkeypatch.setattr(ex.Decoder, "forward", steered)
    monkeypatch.setattr(ex, "draft", chain)
    model = ex.Model(ex.Config())
    prompts = torch.randint(0, 200, (2, n0), generator=torch.Generator().manual_seed(8)).to(torch.int32).cuda()
    out, steps, dec = ex.generate(model, prompts, n_tokens, nodes, budget)
    assert steps == n_tokens - 1
    assert out[0] == ([0] + (list(range(1, nodes)) + [0]) * n_tokens)[:n_tokens]
    assert out[1] == [200] * n_tokens
    rows = [n0 + steps * nodes, n0 + steps]
    assert dec.next_pos.tolist() == rows and dec.lens.tolist() == ([budget, budget] if budget else rows)


def test_a_small_vocabulary_decodes(ex):
    model = ex.Model(ex.Config(vocab=23))
    prompts = torch.randint(0, 23, (2, 10), generator=torch.Generator().manual_seed(9)).to(torch.int32).cuda()
    out, _, dec = ex.generate(model, prompts, 12, 9, sample=True)
    assert all(0 <= t < 23 for o in out for t in o) and int(dec.status.item()) == 0
