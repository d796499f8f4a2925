"""What the sources of the key/value cache's kernels may not say."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_block_quantized_qm_gb300", "csrc")


@pytest.mark.parametrize("name", ["kv_cache.cuh", "kv_cache.cu", "attn.cu", "attn_step.cu", "attn_prompt.cu",
                                  "attn_weights.cu", "tcgen05.cuh"])
def test_no_read_only_loads(name):
    """These kernels start (programmatic launches) while the one before them still writes
    lengths, cells or the workspace, so none of their loads may assume that memory stays
    as it is for the kernel's lifetime."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert not re.findall(r"__ldg\b|__restrict__|ld\.global\.nc|ld\.global\.[a-z:0-9_.]*\bnc\b", text)


def test_one_error_word_for_all_of_the_caches_kernels():
    """qm_device_status reads each word by a synchronous copy: what calls it after every
    step should not pay for a copy per file."""
    words = []
    for name in os.listdir(CSRC):
        if name.startswith(("kv_", "attn")):
            with open(os.path.join(CSRC, name)) as f:
                words += re.findall(r"__device__ unsigned int (g_\w+)", f.read())
    assert words == ["g_kv_error"]


@pytest.mark.parametrize("name", ["kv_cache.cu", "attn.cu", "attn_step.cu", "attn_prompt.cu", "attn_weights.cu"])
def test_the_number_of_sms_is_asked_for(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"\b152\b", code)
