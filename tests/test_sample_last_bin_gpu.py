"""rf_sample where a nucleus ends among a great many tokens some 32 octaves below the greatest, at the first of those whose
masses are summed as parts of 2^(-2047/64).

Such a mass is off by an SFU's 2^-22 and a rounding of 2^-23, relatively: with a million tokens of the kind that is
less than (2^-22 + 2^-23) 2^20 = 0.38 of a token in where the run ends, or one token in n_kept."""
import math

import numpy as np
import pytest
import torch

import test_sample_gpu as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("octaves", [31.93, 31.961, 31.969, 31.9745, 31.98, 31.9843, 31.985, 32.2])
def test_sample_nuclei_that_end_about_where_the_last_bin_begins(octaves, dtype):
    V, R = 1 << 20, 32
    half = V // 2
    x = torch.empty((R, V), device="cuda", dtype=dtype)
    x[:, :half], x[:, half:] = -16.0, -16.5
    x[:, 77] = 0.0
    T = float(np.float32(16.0 * math.log2(math.e) / octaves))
    a, b = math.exp(-16.0 / T), math.exp(-16.5 / T)
    total = 1.0 + (half - 1) * a + half * b
    p = np.array([(1.0 + (i + 0.5) / R * (half - 2) * a) / total for i in range(R)], dtype=np.float32)
    border = (p.astype(np.float64) * total - 1.0) / a
    assert border.min() > 0 and border.max() < half - 2
    P, _, _, cnt, st, _ = S._run(x, [T] * R, [0] * R, p.tolist(), [0.0] * R, draw=False)
    assert st == 0
    want = 1 + np.ceil(border)
    assert np.abs(cnt.cpu().numpy() - want).max() <= 1
    for r in (0, R - 1):                               # the run's tokens, the lowest ones first
        n = int(cnt[r])
        stays = torch.cat([torch.arange(n - 1, device="cuda") + (torch.arange(n - 1, device="cuda") >= 77),
                           torch.tensor([77], device="cuda")])
        assert int((P[r] > 0).sum()) == n and bool((P[r][stays] > 0).all())
