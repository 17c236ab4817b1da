"""rf_sample where logits are so much smaller than the greatest one that their difference from it is no fp32 number.

A border is decided by masses that are off by less than 2^-29 of themselves, and their sums over a bin by 2^-42 of the
greatest weight. Of 2^20 tokens whose weights are e^-20 that is (2^20 2^-29 + 2 2^-42 e^20) < 2^-8 tokens; a difference
from the greatest logit that is rounded to fp32 moves the borders here by a third of a token."""
import math

import numpy as np
import pytest
import torch

import test_sample_gpu as S

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
# 1 - ABOVE and 1 - BELOW are both 1 in fp32, by the most that 8-bit logits allow
ABOVE, BELOW = 1.9921875 * 2.0 ** -26, -1.9921875 * 2.0 ** -25


@pytest.mark.parametrize("dtype", DTYPES)
def test_sample_borders_among_logits_next_to_zero(dtype):
    V, R = 1 << 20, 64
    half = V // 2
    x = torch.empty((R, V), device="cuda", dtype=dtype)
    x[:, :half], x[:, half:] = ABOVE, BELOW
    x[:, V - 1] = 1.0
    p = np.array([1.0 - (i + 0.5) / R * 1.05e-3 for i in range(R)], dtype=np.float32)
    T = float(np.float32(0.05))
    # the run: the greatest one, the half above 0, then k of the others
    a, b = (math.exp((v - 1.0) / T) for v in (ABOVE, BELOW))
    total = 1.0 + half * a + (half - 1) * b
    border = (p.astype(np.float64) * total - 1.0 - half * a) / b
    clear = np.abs(border - np.rint(border)) > 2.0 ** -7
    assert clear.sum() >= R // 2 and border.min() > 0 and border.max() < half - 2
    P, _, _, cnt, st, _ = S._run(x, [T] * R, [0] * R, p.tolist(), [0.0] * R, draw=False)
    assert st == 0
    want = 1 + half + np.ceil(border).astype(np.int64)
    assert (cnt.cpu().numpy() == want)[clear].all()
    assert bool((P[:, :half] > 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_sample_probabilities_of_logits_far_smaller_than_the_greatest(dtype):
    """65 - x is 65 in fp32, 2^-18 off: as much as the weight is off then, relatively."""
    V = 1000
    x = torch.empty((2, V), device="cuda", dtype=dtype)
    x[:, ::2], x[:, 1::2] = 0.99 * 2.0 ** -18, -0.99 * 2.0 ** -18
    x[:, 3] = 65.0
    T, k, p, mp = [1.0] * 2, [0, 200], [1.0] * 2, [0.0] * 2
    P, tok, lp, cnt, st, noise = S._run(x, T, k, p, mp)
    assert st == 0
    for r in range(2):
        S._check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [300, 5003, 131072])
@pytest.mark.parametrize("top", [1e-9, -1e-9, 3e-3, -3e-3, 1e-30, 0.0])
def test_sample_rows_whose_greatest_logit_is_next_to_zero(top, V, dtype):
    R = len(S.SETTINGS)
    x = -S._logits("normal", R, V, V, torch.float32).abs()
    x[:, V // 3] = top
    x[:, V // 2] = top
    x[:, 5] = top - 1e-3
    x = x.clamp_(max=top).to(dtype)
    T, k, p, mp = map(list, zip(*S.SETTINGS))
    P, tok, lp, cnt, st, noise = S._run(x, T, k, p, mp)
    assert st == 0
    for r in range(R):
        S._check_row(V, x[r], T[r], k[r], p[r], mp[r], P[r], tok[r], lp[r], cnt[r], noise[r], True)
