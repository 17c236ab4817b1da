"""Kernels that are launched as dependents start while the kernel before them is still writing. Read-only loads are
defined only for data that nothing writes during the whole life of a kernel, so such kernels take plain ones."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ridge_map_kv_gb300", "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


DEPENDENT = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "pdl_wait()" in _code(f)]


def test_there_are_such_kernels():
    assert {"attn.cu", "attn_weights.cu", "evict.cu", "rope.cu", "verify.cu"} <= set(DEPENDENT)


@pytest.mark.parametrize("name", DEPENDENT)
def test_dependent_kernels_read_by_plain_loads(name):
    assert re.findall(r"__ldg|__restrict__|ld\.global\.nc|ld_global_nc\w*", _code(name)) == []


@pytest.mark.parametrize("name", DEPENDENT)
def test_every_dependent_kernel_waits_for_the_one_before_it(name):
    code = _code(name)
    bodies = code.split("__global__")[1:]
    kernels = [re.search(r"\b(k_\w+)\s*\(", b).group(1) for b in bodies]
    assert kernels and set(re.findall(r"launch_dependent\(\s*(k_\w+)", code)) <= set(kernels)
    for b in bodies:
        assert "pdl_wait()" in b
