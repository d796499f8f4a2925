"""More refusals of the 4-bit key/value cache's entry points, on the host alone."""
import ctypes

import pytest

import bit_block_quantized_qm_gb300 as qm
from test_kv_cache_cpu import FINE, args, attn, cache, lib  # noqa: F401


def test_rows_and_heads_are_numbered_in_32_bits(lib):  # noqa: F811
    """More than 2^32 rows times heads have no number in the list of rows to be done again."""
    big = dict(n_tokens=1 << 30, max_q=1 << 30, n_heads=4, weights=None, lse=None, workspace_bytes=1 << 60)
    assert attn(lib, a=args(**big)) == qm.QM_ERR_SHAPE


def workspace(lib, c, heads, n, m, w, exact=False):  # noqa: F811
    f = lib.qm_attn_workspace_exact if exact else lib.qm_attn_workspace
    return f(ctypes.addressof(c), heads, n, m, w)


@pytest.mark.parametrize("dim", [64, 128, 96])
@pytest.mark.parametrize("seqs,kv,group", [(1, 8, 4), (64, 8, 4), (3, 1, 7), (2, 4, 1), (200, 2, 16), (1, 1, 64)])
def test_a_workspace_serves_every_smaller_call(lib, seqs, kv, group, dim):  # noqa: F811
    """qm_attn_workspace covers what each call of at most its sizes asks for, whichever kernel takes it."""
    c = cache(head_dim=dim, n_seqs=seqs, n_kv_heads=kv, table_stride=300, max_len=4800)
    sizes = [1, 2, 3, 5, 6, 7, 24, 25, 31, 32, 33, 63, 64, 65, 200, 256, 257, 700, 2048]
    most = {}
    for m in sizes:
        for n in (seqs, seqs * m, seqs * m + 5):
            for w in (0, 1):
                need = workspace(lib, c, kv * group, n, m, w)
                assert need >= 0
                most[n, min(m, n), w] = need
    for (n, m, w), need in most.items():
        for (n2, m2, w2) in most:
            if n2 <= n and m2 <= m and w2 <= w:
                assert most[n2, m2, w2] <= need
                assert workspace(lib, c, kv * group, n2, m2, w2, exact=True) <= need, (n, m, w, n2, m2, w2)


def test_a_prompts_workspace_runs_the_next_step(lib):  # noqa: F811
    """The example of the sizes of one long prompt, then a step."""
    c = cache(head_dim=128, n_seqs=1, n_kv_heads=8, n_pages=1000, table_stride=300, max_len=4800)
    need = workspace(lib, c, 32, 2048, 2048, 0)
    step = dict(n_heads=32, n_tokens=1, max_q=1, q_stride=4096, out_stride=4096, weights=None, workspace_bytes=need,
                workspace=1 << 40)
    assert attn(lib, c, args(**step)) in FINE
    assert workspace(lib, c, 32, 2048, 2048, 0, exact=True) < workspace(lib, c, 32, 1, 1, 0, exact=True) <= need
