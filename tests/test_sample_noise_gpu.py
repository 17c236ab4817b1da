"""rf_sample with noise that is no number above 0: a token without a score is never drawn, and a row without any is
reported, whichever way its tokens are found."""
import math

import pytest
import torch

import ridge_map_kv_gb300 as rf
import test_sample_gpu as S

pytestmark = pytest.mark.gpu
SETTINGS = [(1.0, 20, 1.0, 0.0), (0.8, 20, 0.9, 0.0), (1.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 1000, 1.0, 0.0), (1.0, 0, 1.0, 0.05),
            (1.0, 1, 1.0, 0.0), (1.0, 0, 1e-9, 0.0)]


@pytest.mark.parametrize("V", [50, 5003, 131072])
@pytest.mark.parametrize("bad", [math.nan, -1.0, -0.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_rows_without_noise_of_use(dtype, bad, V):
    R = len(SETTINGS)
    x = S._logits("ranked", R, V, V, dtype)
    T, k, p, mp = map(list, zip(*SETTINGS))
    P, tok, lp, cnt, st, noise = S._run(x, T, k, p, mp)
    assert st == 0
    P2, tok2, lp2, cnt2, st, _ = S._run(x, T, k, p, mp, noise=torch.full_like(noise, bad))
    assert st == rf.RF_ERR_INVALID_ARG
    assert tok2.tolist() == [-1] * R and bool((lp2 == -math.inf).all())
    assert torch.equal(P, P2) and torch.equal(cnt, cnt2)
    # one token of those that stay has noise: it is drawn
    only = torch.full_like(noise, bad)
    last = torch.where(P > 0, P, math.inf).argmin(1)
    only[torch.arange(R, device="cuda"), last] = 1e3
    _, tok3, _, _, st, _ = S._run(x, T, k, p, mp, noise=only)
    assert st == 0 and torch.equal(tok3.long(), last)


def test_sample_noise_that_is_infinite_or_very_small():
    """Scores of 0 draw the lowest such token, scores beyond fp32 the lowest of those."""
    V = 3001
    x = torch.zeros((2, V), device="cuda")
    noise = torch.full((2, V), math.inf, device="cuda")
    noise[1, 7:] = 1e-42
    for k in (0, 40, 2000):
        _, tok, _, _, st, _ = S._run(x, k=[k] * 2, noise=noise)
        assert st == 0 and tok.tolist() == [0, 7]
