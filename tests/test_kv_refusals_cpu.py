"""More refusals of the 4-bit key/value cache's entry points, on the host alone."""
import pytest

import bit_block_quantized_qm_gb300 as qm
from test_kv_cache_cpu import FINE, args, attn, cache, lib  # noqa: F401


def test_rows_and_heads_are_numbered_in_32_bits(lib):  # noqa: F811
    """More than 2^32 rows times heads have no number in the list of rows to be done again."""
    big = dict(n_tokens=1 << 30, max_q=1 << 30, n_heads=4, weights=None, lse=None, workspace_bytes=1 << 60)
    assert attn(lib, a=args(**big)) == qm.QM_ERR_SHAPE
