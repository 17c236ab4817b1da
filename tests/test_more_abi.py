"""Refusals of the operators of a batched decoding step: all on the host, before any launch, so no
GPU is touched. Pointers are aligned numbers that nothing dereferences."""
import os

import pytest

import ridge_map_kv_gb300 as rf

P = 256       # an aligned address
INV, SHAPE, ALIGN, WS = rf.RF_ERR_INVALID_ARG, rf.RF_ERR_SHAPE, rf.RF_ERR_ALIGN, rf.RF_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(rf.LIB_PATH):
        from ridge_map_kv_gb300 import build
        build.build()
    rf.lib()


def _refused(status, call, *a, **kw):
    with pytest.raises(rf.RFError) as ei:
        call(*a, **kw, stream=0)
    assert ei.value.status == status, str(ei.value)
    assert rf.rf_last_error()


# ------------------------------------------------------------------ norm and rotation
def _norm(n_q_heads=1, eps=1e-5, **kw):
    d = dict(n_rows=4, n_heads=2, head_dim=64, rot_dim=64, ld_in=128, ld_out=128, pos_offset=0, theta=1e4, factor=2.0,
             original_rows=4096.0, low_turns=1.0, high_turns=4.0, amplitude=1.0, layout=0, dtype=0, transpose=0, scaling=0)
    d.update(kw)
    return rf.rf_norm_rope_desc(rope=rf.rf_rope_desc(**d), n_q_heads=n_q_heads, eps=eps)


@pytest.mark.parametrize("bad,status", [
    (dict(n_rows=-1), INV), (dict(n_heads=0), INV), (dict(theta=0.0), INV), (dict(layout=2), INV), (dict(dtype=2), INV),
    (dict(transpose=1), INV), (dict(n_q_heads=-1), INV), (dict(n_q_heads=3), INV), (dict(eps=0.0), INV),
    (dict(eps=-1e-5), INV), (dict(eps=1e-40), INV), (dict(eps=float("inf")), INV), (dict(eps=float("nan")), INV),
    (dict(head_dim=60, rot_dim=60), SHAPE), (dict(head_dim=264, rot_dim=64, ld_in=528, ld_out=528), SHAPE),
    (dict(rot_dim=63), SHAPE), (dict(n_rows=(1 << 24) + 1), SHAPE), (dict(ld_in=120), ALIGN), (dict(ld_out=132), ALIGN)])
def test_norm_rope_refuses_bad_descriptors(bad, status):
    d = _norm(**bad)
    assert rf.rf_norm_rope_backward_workspace_bytes(d) == 0
    _refused(status, rf.rf_norm_rope, d, P, P, P, 2 * P)
    _refused(status, rf.rf_norm_rope_backward, d, P, P, P, P, P, P, P, 2 * P, P, 1 << 40)


def test_norm_rope_refuses_pointers():
    _refused(INV, rf.rf_norm_rope, _norm(), None, P, P, P)
    _refused(INV, rf.rf_norm_rope, _norm(), P, P, P, None)
    for i in range(4):
        a = [P, P, P, 2 * P]
        a[i] += 8
        _refused(ALIGN, rf.rf_norm_rope, _norm(), *a)
    _refused(ALIGN, rf.rf_norm_rope, _norm(), P, P, P, P, P + 2)
    _refused(INV, rf.rf_norm_rope, _norm(ld_out=136), P, P, P, P)       # in place with another stride
    rf.rf_norm_rope(_norm(n_rows=0), None, None, None, None, stream=0)


def test_norm_rope_backward_refuses_pointers():
    d, far = _norm(), 1 << 20
    need = rf.rf_norm_rope_backward_workspace_bytes(d)
    good = [P, P, P, 2 * P, P, 3 * P, P, far, P, need]                    # in, gains, d_out, positions, d_in, sums, workspace
    for i in (0, 3, 5):
        _refused(INV, rf.rf_norm_rope_backward, d, *good[:i], None, *good[i + 1:])
    for i, off in ((0, 8), (1, 8), (2, 8), (3, 8), (5, 8), (4, 2), (6, 2), (7, 2)):
        _refused(ALIGN, rf.rf_norm_rope_backward, d, *good[:i], good[i] + off, *good[i + 1:])
    _refused(WS, rf.rf_norm_rope_backward, d, *good[:8], None, need)
    _refused(WS, rf.rf_norm_rope_backward, d, *good[:8], P, need - 1)
    _refused(WS, rf.rf_norm_rope_backward, d, *good[:8], P + 128, need)
    _refused(INV, rf.rf_norm_rope_backward, d, *good[:7], P + 4, P, need)  # the gains' gradients overlap
    _refused(INV, rf.rf_norm_rope_backward, _norm(ld_out=136), *good[:5], good[3], *good[6:])
    rf.rf_norm_rope_backward(_norm(n_rows=0), None, None, None, None, None, None, stream=0)


# ------------------------------------------------------------------------ sampling
def _sample(**kw):
    d = dict(n_rows=2, vocab=100, ld_logits=100, ld_noise=100, ld_probs=100, dtype=rf.RF_F32, reserved=0)
    d.update(kw)
    return rf.rf_sample_desc(**d)


FAR = 1 << 20
GOOD = [P, P, P, P, P, P, FAR, P, P, P]     # logits, temperature, top_k, top_p, min_p, noise, probs, token, logprob, n_kept


@pytest.mark.parametrize("bad,status", [
    (dict(n_rows=-1), INV), (dict(vocab=0), INV), (dict(dtype=2), INV), (dict(reserved=1), INV),
    (dict(vocab=(1 << 20) + 1, ld_logits=1 << 21, ld_noise=1 << 21, ld_probs=1 << 21), SHAPE),
    (dict(n_rows=(1 << 24) + 1), SHAPE), (dict(ld_logits=1 << 37), SHAPE), (dict(ld_probs=1 << 62), SHAPE),
    (dict(ld_logits=99), ALIGN), (dict(ld_noise=99), ALIGN), (dict(ld_probs=99), ALIGN)])
def test_sample_refuses_bad_descriptors(bad, status):
    _refused(status, rf.rf_sample, _sample(**bad), *GOOD)


def test_sample_refuses_pointers():
    d = _sample()
    _refused(INV, rf.rf_sample, d, None, *GOOD[1:])
    _refused(INV, rf.rf_sample, d, P)                                        # neither token nor probabilities
    _refused(INV, rf.rf_sample, d, *GOOD[:5], None, *GOOD[6:])                # a token without noise
    _refused(INV, rf.rf_sample, d, *GOOD[:7], None, None, P)                  # noise without a token
    _refused(INV, rf.rf_sample, d, *GOOD[:5], None, FAR, None, P, P)          # a log-probability without a token
    for i in range(10):
        _refused(ALIGN, rf.rf_sample, d, *GOOD[:i], GOOD[i] + 2, *GOOD[i + 1:])
    _refused(ALIGN, rf.rf_sample, _sample(dtype=rf.RF_BF16), P + 1, *GOOD[1:])
    for shift in (4, 4 * 199, -4 * 199):                                      # probabilities over the logits in part
        _refused(INV, rf.rf_sample, d, FAR, *GOOD[1:6], FAR + shift, *GOOD[7:])
    _refused(INV, rf.rf_sample, _sample(ld_probs=104), FAR, *GOOD[1:6], FAR, *GOOD[7:])
    _refused(INV, rf.rf_sample, _sample(dtype=rf.RF_BF16), FAR, *GOOD[1:6], FAR, *GOOD[7:])
    rf.rf_sample(_sample(n_rows=0), None, stream=0)


# ------------------------------------------------------------ attention over a shared prefix
def _prefix(prefix_capacity=50, prefix_row_stride=256, **kw):
    d = dict(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=128, n_nodes=4, capacity=100, q_row_stride=1024,
             q_seq_stride=4096, draft_row_stride=256, draft_seq_stride=1024, cache_row_stride=256, cache_seq_stride=25600,
             out_row_stride=1024, out_seq_stride=4096, scale=0.1)
    d.update(kw)
    return rf.rf_prefix_attn_desc(attn=rf.rf_attn_desc(**d), prefix_capacity=prefix_capacity,
                                  prefix_row_stride=prefix_row_stride)


@pytest.mark.parametrize("bad,status", [
    (dict(n_seqs=-1), INV), (dict(n_nodes=0), INV), (dict(capacity=0), INV), (dict(scale=0.0), INV), (dict(flags=1), INV),
    (dict(head_dim=96), SHAPE), (dict(n_q_heads=7), SHAPE), (dict(q_row_stride=1016), ALIGN),
    (dict(cache_row_stride=260), ALIGN), (dict(prefix_capacity=0), INV), (dict(prefix_capacity=(1 << 30) + 1), SHAPE),
    (dict(prefix_row_stride=248), ALIGN), (dict(prefix_row_stride=260), ALIGN), (dict(prefix_row_stride=1 << 39), SHAPE),
    (dict(n_seqs=1 << 20, n_nodes=64), SHAPE)])
def test_prefix_attention_refuses_bad_descriptors(bad, status):
    d = _prefix(**bad)
    assert rf.rf_prefix_attn_workspace_bytes(d) == 0
    _refused(status, rf.rf_prefix_attention, d, *[P] * 12, None, P, 1 << 50)


def test_prefix_attention_refuses_pointers():
    d = _prefix()
    need = rf.rf_prefix_attn_workspace_bytes(d)
    # q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, lens, k_draft, v_draft, tree_mask, out, lse
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 10):
        a = [P] * 12
        a[i] = None
        _refused(INV, rf.rf_prefix_attention, d, *a, None, P, need)
    for i in range(12):
        a = [P] * 12
        a[i] += 2
        _refused(ALIGN, rf.rf_prefix_attention, d, *a, None, P, need)
    _refused(WS, rf.rf_prefix_attention, d, *[P] * 12, None, None, need)
    _refused(WS, rf.rf_prefix_attention, d, *[P] * 12, None, P, need - 1)
    _refused(WS, rf.rf_prefix_attention, d, *[P] * 12, None, P + 128, need)
    wide = _prefix(n_nodes=1025, q_seq_stride=1 << 21, draft_seq_stride=1 << 19, out_seq_stride=1 << 21)
    _refused(SHAPE, rf.rf_prefix_attention, wide, *[P] * 12, None, P, 1 << 50)            # with a mask
    rf.rf_prefix_attention(_prefix(n_seqs=0), *[None] * 12, stream=0)
