"""rf_sample refuses probabilities that lie over its noise, which a row's CTAs read while others write: on the host,
before any launch. Pointers are aligned numbers that nothing dereferences."""
import os

import pytest

import ridge_map_kv_gb300 as rf

P, FAR = 256, 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(rf.LIB_PATH):
        from ridge_map_kv_gb300 import build
        build.build()
    rf.lib()


def _status(noise, probs, rows=3, ld_noise=100, ld_probs=100):
    d = rf.rf_sample_desc(n_rows=rows, vocab=100, ld_logits=100, ld_noise=ld_noise, ld_probs=ld_probs, dtype=rf.RF_BF16)
    with pytest.raises(rf.RFError) as ei:
        rf.rf_sample(d, P, noise=noise, probs=probs, token=P, stream=0)
    return ei.value.status, str(ei.value)


@pytest.mark.parametrize("shift", [0, 4, -4, 4 * 99, 4 * 100, 4 * 299, -4 * 299])
def test_sample_refuses_probabilities_over_the_noise(shift):
    status, text = _status(FAR, FAR + shift)
    assert status == rf.RF_ERR_INVALID_ARG and "noise" in text


@pytest.mark.parametrize("shift,ld_noise,ld_probs", [
    (4 * 99, 200, 200), (-4 * 99, 200, 200), (4 * 101, 200, 200), (4 * 301, 200, 200), (0, 100, 200), (4 * 150, 200, 300)])
def test_sample_refuses_probabilities_among_the_noise_rows(shift, ld_noise, ld_probs):
    status, text = _status(FAR, FAR + shift, ld_noise=ld_noise, ld_probs=ld_probs)
    assert status == rf.RF_ERR_INVALID_ARG and "noise" in text


@pytest.mark.parametrize("shift,ld", [(4 * 300, 100), (-4 * 300, 100), (4 * 100, 200), (-4 * 100, 200), (4 * 300, 200), (4 * 250, 350)])
def test_sample_takes_probabilities_beside_the_noise(shift, ld):
    """(Not refused for that: without a GPU the call ends at the device.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory")
    status, text = _status(FAR, FAR + shift, ld_noise=ld, ld_probs=ld)
    assert "noise" not in text
