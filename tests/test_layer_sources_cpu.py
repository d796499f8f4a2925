"""The sources of norm, routing and experts: no loads that may be served before the kernel before has ended.

The kernels start while the kernel before them may still write what they read, so nothing may be read through the
read-only path, which a compiler takes for __restrict__ pointers to const."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "bit_block_quantized_qm_gb300", "csrc")


@pytest.mark.parametrize("name", ["rmsnorm.cu", "route.cu", "experts.cu", "experts_mm.cu", "experts_few.cu", "experts.cuh"])
def test_plain_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__restrict__|__ldg\b|\.nc\b|ldg_nc", code)


@pytest.mark.parametrize("name", ["rmsnorm.cu", "route.cu", "experts.cu", "experts_mm.cu", "experts_few.cu"])
def test_every_kernel_waits(name):
    """Each kernel of a chain waits for the one before it: who waits for the last has waited for all."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    kernels = re.split(r"__global__", code)[1:]
    assert kernels and all("grid_dependency_wait()" in k for k in kernels)
