"""Refusals of the decoding operators: all on the host, before any launch, so no GPU is
touched. Pointers are aligned numbers that nothing dereferences."""
import os
import random
import re

import pytest

import ridge_map_kv_gb300 as rf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def _rope(**kw):
    d = dict(n_rows=4, n_heads=2, head_dim=64, rot_dim=64, ld_in=128, ld_out=128, pos_offset=0, theta=1e4, factor=2.0,
             original_rows=4096.0, low_turns=1.0, high_turns=4.0, amplitude=1.0, layout=0, dtype=0, transpose=0, scaling=0)
    d.update(kw)
    return rf.rf_rope_desc(**d)


@pytest.mark.parametrize("bad,status", [
    (dict(n_rows=-1), INV), (dict(n_heads=0), INV), (dict(theta=0.0), INV), (dict(theta=float("nan")), INV),
    (dict(layout=2), INV), (dict(dtype=2), INV), (dict(scaling=5), INV), (dict(scaling=1, factor=0.5), INV),
    (dict(scaling=3, high_turns=1.0), INV), (dict(scaling=4, original_rows=0.0), INV), (dict(scaling=4, theta=1.0), INV),
    (dict(amplitude=float("inf")), INV), (dict(head_dim=60, rot_dim=60), SHAPE),
    (dict(head_dim=264, rot_dim=64, ld_in=528, ld_out=528), SHAPE), (dict(rot_dim=63), SHAPE), (dict(rot_dim=66), SHAPE),
    (dict(scaling=2, rot_dim=2), SHAPE), (dict(n_rows=(1 << 24) + 1), SHAPE), (dict(ld_in=120), ALIGN),
    (dict(ld_out=132), ALIGN)])
def test_rope_refusals(bad, status):
    _refused(status, rf.rf_rope, _rope(**bad), P, 2 * P)


def test_rope_pointer_refusals_and_nothing_to_do():
    _refused(INV, rf.rf_rope, _rope(), None, P)
    _refused(ALIGN, rf.rf_rope, _rope(), P + 8, P)
    _refused(ALIGN, rf.rf_rope, _rope(), P, 2 * P, P + 2)
    _refused(INV, rf.rf_rope, _rope(ld_out=136), P, P)          # in place with another stride
    rf.rf_rope(_rope(n_rows=0), None, None, stream=0)


def test_tree_build_refusals():
    _refused(INV, rf.rf_tree_build, -1, 4, P)
    _refused(INV, rf.rf_tree_build, 1, 0, P)
    _refused(SHAPE, rf.rf_tree_build, 1, 1025, P, P, P, P)
    _refused(INV, rf.rf_tree_build, 1, 4, None, P, P, P)
    _refused(INV, rf.rf_tree_build, 1, 4, P, None, P, P)        # positions need next_pos
    _refused(ALIGN, rf.rf_tree_build, 1, 4, P, P, P + 4, P)
    rf.rf_tree_build(0, 4, None, stream=0)


def _attn(**kw):
    d = dict(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=128, n_nodes=4, capacity=100, q_row_stride=1024,
             q_seq_stride=4096, draft_row_stride=256, draft_seq_stride=1024, cache_row_stride=256, cache_seq_stride=25600,
             out_row_stride=1024, out_seq_stride=4096, scale=0.1)
    d.update(kw)
    return rf.rf_attn_desc(**d)


BAD_ATTN = [
    (dict(n_seqs=-1), INV), (dict(n_nodes=0), INV), (dict(capacity=0), INV), (dict(scale=0.0), INV),
    (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=1e39), INV), (dict(scale=1e-60), INV),
    (dict(flags=1), INV), (dict(head_dim=96), SHAPE), (dict(n_q_heads=7), SHAPE), (dict(n_q_heads=258), SHAPE),
    (dict(n_nodes=(1 << 20) + 1), SHAPE), (dict(q_row_stride=1016), ALIGN), (dict(cache_row_stride=260), ALIGN),
    (dict(cache_seq_stride=0), ALIGN), (dict(draft_seq_stride=-8), ALIGN), (dict(out_row_stride=8), ALIGN)]


@pytest.mark.parametrize("bad,status", BAD_ATTN)
def test_attention_and_weights_refuse_bad_descriptors(bad, status):
    d = _attn(**bad)
    assert rf.rf_attn_workspace_bytes(d) == 0 and rf.rf_attn_weights_workspace_bytes(d) == 0
    _refused(status, rf.rf_tree_attention, d, P, P, P, P, P, P, P, P, P, None, P, 1 << 40)
    _refused(status, rf.rf_attn_weights, d, P, P, P, P, P, P, 1.0, P, P, None, P, 1 << 40)


def test_attention_refuses_pointers_workspaces_and_long_masks():
    d = _attn()
    need = rf.rf_attn_workspace_bytes(d)
    assert need > 0
    names = ["q", "k", "v", "lens", "kd", "vd", "mask", "out", "lse"]
    for i, name in enumerate(names):
        a = [P] * 9
        a[i] = None
        if name in ("mask", "lse"):            # may be NULL: the workspace is looked at next
            _refused(WS, rf.rf_tree_attention, d, *a, None, P, need - 1)
        else:
            _refused(INV, rf.rf_tree_attention, d, *a, None, P, need)
        a[i] = P + 2
        _refused(ALIGN, rf.rf_tree_attention, d, *a, None, P, need)
    _refused(WS, rf.rf_tree_attention, d, *[P] * 9, None, None, need)
    _refused(WS, rf.rf_tree_attention, d, *[P] * 9, None, P + 128, need)
    _refused(SHAPE, rf.rf_tree_attention, _attn(n_nodes=1025, q_seq_stride=1 << 24, draft_seq_stride=1 << 24,
                                                out_seq_stride=1 << 24), *[P] * 9, None, P, 1 << 40)
    rf.rf_tree_attention(_attn(n_seqs=0), *[None] * 9, None, None, 0, stream=0)
    # a wider row tile needs more scratch
    assert rf.rf_attn_workspace_bytes(_attn(n_nodes=64)) > need


def test_weights_refuse_pointers_and_workspaces():
    d = _attn()
    full = dict(q=P, lse=P, path=P, n_path=P, k=P, lens=P, score_in=P, score_out=P)

    def call(decay=1.0, ws=P, wsb=256, **kw):
        a = dict(full, **kw)
        return (d, a["q"], a["lse"], a["path"], a["n_path"], a["k"], a["lens"], decay, a["score_in"], a["score_out"],
                None, ws, wsb)
    for name in ("q", "lse", "path", "n_path", "k", "lens", "score_in", "score_out"):
        _refused(INV, rf.rf_attn_weights, *call(**{name: None}))
        _refused(ALIGN, rf.rf_attn_weights, *call(**{name: P + 2}))
    _refused(INV, rf.rf_attn_weights, *call(decay=float("inf")))
    _refused(WS, rf.rf_attn_weights, *call(ws=None))
    _refused(WS, rf.rf_attn_weights, *call(wsb=255))
    _refused(WS, rf.rf_attn_weights, *call(decay=0.0, score_in=None, wsb=0))    # decay 0: no score_in needed
    _refused(SHAPE, rf.rf_attn_weights, _attn(n_seqs=1025), *call()[1:])


def _verify(**kw):
    d = dict(n_seqs=2, n_nodes=4, vocab=100, ld_target=100, ld_draft=100, ld_noise=100)
    d.update(kw)
    return rf.rf_verify_desc(**d)


@pytest.mark.parametrize("bad,status", [(dict(n_seqs=-1), INV), (dict(n_nodes=0), INV), (dict(vocab=0), INV),
                                        (dict(n_nodes=1025), SHAPE), (dict(vocab=1 << 31, ld_target=1 << 31,
                                                                           ld_draft=1 << 31, ld_noise=1 << 31), SHAPE),
                                        (dict(ld_target=99), ALIGN), (dict(ld_draft=99), ALIGN), (dict(ld_noise=99), ALIGN)])
def test_verify_refuses_bad_descriptors(bad, status):
    _refused(status, rf.rf_verify_draft, _verify(**bad), *[P] * 9)


def test_verify_refuses_pointers():
    for i in (0, 2, 3, 4, 5, 6, 7, 8):          # all but the draft
        a = [P] * 9
        a[i] = None
        _refused(INV, rf.rf_verify_draft, _verify(), *a)
        a[i] = P + 1
        _refused(ALIGN, rf.rf_verify_draft, _verify(), *a)
    rf.rf_verify_draft(_verify(n_seqs=0), *[None] * 9, stream=0)


def _cache(**kw):
    d = dict(n_layers=2, n_seqs=2, n_kv_heads=2, head_dim=64, capacity=50, row_stride=128, seq_stride=6400,
             layer_stride=12800)
    d.update(kw)
    return rf.rf_cache_desc(**d)


BAD_CACHE = [(dict(n_layers=-1), INV), (dict(n_kv_heads=0), INV), (dict(capacity=0), INV), (dict(head_dim=12), SHAPE),
             (dict(head_dim=264, row_stride=528), SHAPE), (dict(capacity=(1 << 24) + 1), SHAPE), (dict(n_seqs=65536), SHAPE),
             (dict(row_stride=120), ALIGN), (dict(seq_stride=6404), ALIGN), (dict(layer_stride=0), ALIGN),
             (dict(seq_stride=0), ALIGN), (dict(seq_stride=128, layer_stride=256), ALIGN)]


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_commit_and_evict_refuse_bad_caches(bad, status):
    d = _cache(**bad)
    assert rf.rf_evict_workspace_bytes(d, 10) == 0
    _refused(status, rf.rf_evict, d, 10, 0, 0, *[P] * 9, None, P, 1 << 40)
    _refused(status, rf.rf_commit_draft, d, 4, 128, 512, 1024, *[P] * 12)


def test_evict_refuses_arguments():
    d = _cache()
    need = rf.rf_evict_workspace_bytes(d, 10)
    assert need >= 256 and rf.rf_evict_workspace_bytes(d, 0) == 0
    assert rf.rf_evict_workspace_bytes(d, 50) == 256             # nothing can move
    _refused(INV, rf.rf_evict, d, 0, 0, 0, *[P] * 9, None, P, need)
    _refused(INV, rf.rf_evict, d, 10, -1, 0, *[P] * 9, None, P, need)
    _refused(INV, rf.rf_evict, d, 10, 0, 1 << 31, *[P] * 9, None, P, need)
    for i in range(9):
        a = [P] * 9
        a[i] = None
        _refused(INV, rf.rf_evict, d, 10, 0, 0, *a, None, P, need)
        a[i] = P + 2
        _refused(ALIGN, rf.rf_evict, d, 10, 0, 0, *a, None, P, need)
    _refused(WS, rf.rf_evict, d, 10, 0, 0, *[P] * 9, None, P, need - 1)
    _refused(SHAPE, rf.rf_evict, _cache(n_layers=300, n_kv_heads=128, row_stride=8192, seq_stride=409600,
                                        layer_stride=819200), 10, 0, 0, *[P] * 9, None, P, 1 << 40)


def test_commit_refuses_arguments():
    d = _cache()
    args = (4, 128, 512, 1024)
    _refused(INV, rf.rf_commit_draft, d, 0, 128, 512, 1024, *[P] * 12)
    _refused(SHAPE, rf.rf_commit_draft, d, (1 << 20) + 1, 128, 512, 1024, *[P] * 12)
    _refused(ALIGN, rf.rf_commit_draft, d, 4, 120, 512, 1024, *[P] * 12)
    _refused(ALIGN, rf.rf_commit_draft, d, 4, 128, 516, 1024, *[P] * 12)
    for i in (0, 1, 2, 3, 4, 5, 6, 7):
        a = [P] * 12
        a[i] = None
        _refused(INV, rf.rf_commit_draft, d, *args, *a)          # 3: next_pos, wanted by pos
    for i in range(12):
        a = [P] * 12
        a[i] = P + 2
        _refused(ALIGN, rf.rf_commit_draft, d, *args, *a)


def test_constants_and_stage_names_match_the_header():
    txt = open(os.path.join(ROOT, "include", "rf.h")).read()
    for name, val in re.findall(r"#define (RF_(?:ROPE|BF16|F32|TREE_MAX)\w*) (\d+)\b", txt):
        assert getattr(rf, name) == int(val), name
    stages = re.findall(r"RF_STAGE_(\w+) = (\d+)", txt)
    for name, val in stages:
        assert rf.rf_stage_name(int(val)) != "unknown", name
    assert [rf.rf_stage_name(i) for i in (22, 24, 26, 28, 29)] == ["rope", "attention", "verify", "attention_weights",
                                                                  "evict_select"]


def test_evict_refuses_lengths_that_overlap_in_part():
    d = _cache()
    need = rf.rf_evict_workspace_bytes(d, 10)
    for shift in (-4, 4):                       # two sequences: 8 bytes
        _refused(INV, rf.rf_evict, d, 10, 0, 0, P, 2 * P, *[P] * 6, P + shift, None, P, need)


def test_commit_refuses_lengths_that_overlap_in_part():
    d = _cache()
    far = [P << 4, P << 5, P << 6, P << 7]      # path, n_path, lens, next_pos
    for i in range(4):                          # two sequences: 8 bytes; the path: 32
        for shift in (-4, 4) if i else (-4, 0, 28):
            for out in ([far[i] + shift, P << 8], [P << 8, far[i] + shift]):
                _refused(INV, rf.rf_commit_draft, d, 4, 128, 512, 1024, *far, *[P] * 6, *out)


W = 128          # elements of a row of _cache(): 2 heads of 64 channels; 50 rows, 2 sequences, 2 layers


@pytest.mark.parametrize("strides,legal", [
    # (row, sequence, layer), and whether rows of the whole cache lie apart
    ((W, 50 * W, 100 * W), True), ((W, 100 * W, 50 * W), True),          # layers of sequences, sequences of layers
    ((2 * W, W, 100 * W), True), ((4 * W, W, 2 * W), True), ((4 * W, 2 * W, W), True),     # rows of both, between and outside
    ((2 * W, 100 * W, W), True), ((3 * W, 200 * W, 3 * 49 * W + W), True),
    ((W, 50 * W, 50 * W), False), ((W, 50 * W, 99 * W), False), ((W, 49 * W, 100 * W), False), ((W, 100 * W, 49 * W), False),
    ((2 * W, W, 99 * W), False), ((2 * W, W - 8, 100 * W), False), ((3 * W, W, 2 * W), False), ((4 * W, W, W), False)])
def test_caches_may_be_nested_in_any_order_but_not_overlap(strides, legal):
    names = ("row_stride", "seq_stride", "layer_stride")
    d = _cache(**dict(zip(names, strides)))
    assert (rf.rf_evict_workspace_bytes(d, 10) > 0) == legal
    at = {r * strides[0] + b * strides[1] + l * strides[2] for r in range(50) for b in range(2) for l in range(2)}
    places = sorted(at)
    apart = len(places) == 200 and all(y - x >= W for x, y in zip(places, places[1:]))
    assert apart == legal                                                # the parameters themselves
    if not legal:
        _refused(ALIGN, rf.rf_evict, d, 10, 0, 0, *[P] * 9, None, P, 1 << 40)
        _refused(ALIGN, rf.rf_commit_draft, d, 4, 128, 512, 1024, *[P] * 12)


@pytest.mark.parametrize("stride,legal", [(50 * W, True), (50 * W - 8, False), (8, False)])
def test_layers_of_a_single_sequence_may_not_overlap(stride, legal):
    d = _cache(n_seqs=1, layer_stride=stride, seq_stride=0)
    assert (rf.rf_evict_workspace_bytes(d, 10) > 0) == legal
    assert rf.rf_evict_workspace_bytes(_cache(n_layers=1, n_seqs=1, layer_stride=0, seq_stride=0), 10) > 0
    # strides whose spans pass 64 bits
    assert rf.rf_evict_workspace_bytes(_cache(n_layers=65535, layer_stride=1 << 61, seq_stride=1 << 61), 10) == 0


def test_small_caches_are_accepted_exactly_where_no_two_rows_overlap():
    r = random.Random(1)
    for _ in range(3000):
        n_layers, n_seqs, rows, w = r.randint(1, 4), r.randint(1, 4), r.randint(1, 5), r.choice([8, 16])
        row, seq, layer = r.randint(w // 8, 14) * 8, r.randint(0, 14) * 8, r.randint(0, 14) * 8
        d = rf.rf_cache_desc(n_layers=n_layers, n_seqs=n_seqs, n_kv_heads=1, head_dim=w, capacity=rows, row_stride=row,
                             seq_stride=seq, layer_stride=layer)
        at = sorted(t * row + b * seq + l * layer for t in range(rows) for b in range(n_seqs) for l in range(n_layers))
        assert (rf.rf_evict_workspace_bytes(d, 3) > 0) == all(y - x >= w for x, y in zip(at, at[1:]))


def test_scales_whose_base_2_form_overflows_are_refused():
    """Scores are taken to base 2, where the largest fp32 numbers turn infinite (and 0 times that NaN)."""
    for scale, legal in ((2.3e38, True), (2.4e38, False), (3.4e38, False)):
        d = _attn(scale=scale)
        assert (rf.rf_attn_workspace_bytes(d) > 0) == legal
        if not legal:
            _refused(INV, rf.rf_tree_attention, d, P, P, P, P, P, P, P, P, P, None, P, 1 << 40)
            _refused(INV, rf.rf_attn_weights, d, P, P, P, P, P, P, 1.0, P, P, None, P, 1 << 40)


def test_the_header_states_the_limits_of_the_decoding_calls():
    """What the calls refuse by size alone is found in the header beside them."""
    text = re.sub(r"\n \* ?", " ", open(os.path.join(ROOT, "include", "rf.h")).read())
    assert "n_layers * n_seqs * n_kv_heads <= 65535" in text and "with n_seqs <= 1024" in text
    ok = dict(n_kv_heads=15, row_stride=960, seq_stride=48000, layer_stride=96000)
    assert rf.rf_evict_workspace_bytes(_cache(n_layers=2184, **ok), 10) > 0
    assert rf.rf_evict_workspace_bytes(_cache(n_layers=2185, **ok), 10) == 0            # 65,550
    assert rf.rf_attn_weights_workspace_bytes(_attn(n_seqs=1024)) == 256
    assert rf.rf_attn_weights_workspace_bytes(_attn(n_seqs=1025)) == 0
