"""The kernels' copies: each CTA loads into its own shared memory alone.

A copy that writes to several CTAs of a cluster is sound only for memory that is certain to be this GPU's own, and the
library takes managed memory and is loaded by processes that use several GPUs."""
import glob
import os

import pytest

ROOT = os.path.join(os.path.dirname(__file__), "..")
SOURCES = sorted(glob.glob(os.path.join(ROOT, "bit_block_quantized_qm_gb300", "csrc", "*")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_copies_to_one_cta(path):
    with open(path) as f:
        text = f.read().lower()
    assert "multi" + "cast" not in text


def test_there_are_sources():
    assert len(SOURCES) > 20
