"""rf_sample at the largest vocabulary, 2^20 tokens, with every filter: counts, masses and token numbers at their limits.
What is compared, and how closely, is as in test_sample_gpu."""
import pytest
import torch

import test_sample_gpu as S

pytestmark = pytest.mark.gpu
V = 1 << 20
HOT = 2.0 ** 100                                        # brings any finite logits into one bin
ONE_BIN = [(50, 1.0), (256, 0.51234), (1000, 1.0), (300000, 1.0), (V - 1, 1.0), (V, 1.0)]
NUCLEI = [(0, 0.3000051), (0, 0.9000155), (0, 1e-9), (500000, 0.7000121), (0, 0.99999994)]


def _one_bin(kind, dtype, rows):
    x = S._logits("normal" if kind == "hot" else "equal", rows, V, 5, dtype)
    if kind == "near":                                  # distinct logits, all weights within 1/128 octave
        x = S._logits("normal", rows, V, 6, dtype) * 1e-5
    return x, (HOT if kind == "hot" else 1.0)


def _check(x, T, k, p, mp):
    P, tok, lp, cnt, st, noise = S._run(x, T, k, p, mp)
    assert st == 0
    for r in range(len(T)):
        S._check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["equal", "near", "hot"])
@pytest.mark.parametrize("settings", [ONE_BIN, NUCLEI], ids=["top_k", "top_p"])
def test_sample_all_tokens_in_one_bin(settings, kind, dtype):
    x, T = _one_bin(kind, dtype, len(settings))
    k, p = map(list, zip(*settings))
    _check(x, [T] * len(k), k, p, [0.0] * len(k))


@pytest.mark.parametrize("vocab", [V - 1, V - 7])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_all_tokens_in_one_bin_of_a_little_fewer(vocab, dtype):
    x = torch.full((4, vocab), 1.5, device="cuda", dtype=dtype)
    k = [50, 1000, vocab - 1, vocab]
    P, tok, lp, cnt, st, noise = S._run(x, [1.0] * 4, k, [1.0] * 4, [0.0] * 4)
    assert st == 0
    for r in range(4):
        S._check_row(vocab, x[r], 1.0, k[r], 1.0, 0.0, P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["normal", "ranked", "flat", "steps", "far", "masked", "lowest"])
def test_sample_every_setting_of_the_largest_vocabulary(kind, dtype):
    settings = S.SETTINGS + [(1.0, 300000, 0.95, 0.0), (HOT, 700001, 1.0, 0.0)]
    x = S._logits(kind, len(settings), V, 17, dtype)
    T, k, p, mp = map(list, zip(*settings))
    if kind in ("steps", "lowest", "flat"):             # (borders between equal masses, as in test_sample_gpu)
        p = [min(1.0, q * 1.0000172) if 0.0 < q < 1.0 else q for q in p]
    _check(x, T, k, p, mp)


def test_sample_the_last_token_of_the_largest_vocabulary():
    x = torch.full((3, V), -1.0, device="cuda")
    x[:, V - 1] = 4.0
    P, tok, _, cnt, st, _ = S._run(x, [1.0, 0.0, 1.0], [1, 0, 0], [1.0, 1.0, 1e-9], [0.0] * 3)
    assert st == 0 and tok.tolist() == [V - 1] * 3 and cnt.tolist() == [1] * 3
    assert bool((P[:, V - 1] == 1).all()) and not bool(P[:, :V - 1].any())
