"""Channels that do not turn are each by itself: what is not finite in one of them reaches no other channel of the
rows, nor of the gains' gradients. Everything else has the bits that it has with a number in that place."""
import math

import pytest
import torch

import decoderef as R
import ridge_map_kv_gb300 as rf
import test_norm_rope_gpu as N

pytestmark = pytest.mark.gpu
CASES = [  # hd, rot, layout, dtype
    (128, 64, 0, 0), (128, 64, 0, 1), (128, 96, 1, 0), (64, 20, 1, 1), (64, 22, 1, 0), (64, 20, 0, 0), (40, 16, 0, 1), (256, 100, 1, 0),
    (256, 2, 1, 1), (80, 32, 0, 0)]


def _others(x, *at):
    """x with a 0 in one place, as bits."""
    x = x.clone()
    x[at] = 0.0
    return x.contiguous().view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("hd,rot,layout,dtype", CASES)
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_norm_rope_a_gain_that_is_not_finite(hd, rot, layout, dtype, value):
    rows, q, k = 7, 3, 2
    s = N._setup(rows, q, k, hd, rot, layout, dtype, 0, False, 0, 0)

    def call():
        y = torch.empty_like(s["x"])
        rf.rf_norm_rope(s["desc"], s["x"], s["gq"], s["gk"], y)
        return y.view(rows, q + k, hd)

    clean = call()
    for c in (rot, rot + 1, (rot + hd) // 2, hd - 1):
        kept = s["gq"][c].clone()
        s["gq"][c] = value
        y = call()
        s["gq"][c] = kept
        torch.cuda.synchronize()
        at = (slice(None), slice(0, q), c)
        assert not bool(torch.isfinite(y[at]).any())
        assert torch.equal(_others(y, *at), _others(clean, *at))


@pytest.mark.parametrize("hd,rot,layout,dtype", CASES)
@pytest.mark.parametrize("value", [-math.inf, math.nan])
def test_norm_rope_an_output_gradient_that_is_not_finite(hd, rot, layout, dtype, value):
    rows, q, k = 9, 2, 3
    s = N._setup(rows, q, k, hd, rot, layout, dtype, 0, False, 0, 0)
    dy = R.randn((rows, (q + k) * hd), 4, s["x"].dtype)
    clean = N._backward(s, dy)
    for c in (rot, rot + 1, (rot + hd) // 2, hd - 1):
        bad = dy.clone()
        bad.view(rows, q + k, hd)[5, q + 1, c] = value
        dx, dq, dk = N._backward(s, bad)
        assert torch.equal(dq, clean[1]) and not math.isfinite(float(dk[c]))
        assert torch.equal(_others(dk, c), _others(clean[2], c))
        at = (5, q + 1)                               # (the mean over that head's channels has it)
        assert torch.equal(_others(dx.view(rows, q + k, hd), *at), _others(clean[0].view(rows, q + k, hd), *at))
