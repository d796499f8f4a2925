"""GPU tests of the 4-bit key/value cache where what only the device sees is wrong, or
where calls meet: offsets that give a row to two sequences, workspaces that CUDA
graphs use.  Nothing here reaches past the buffers it is given.
"""
import ctypes

import numpy as np
import pytest

import kv_oracle as ko

torch = pytest.importorskip("torch")
from test_gpu_kv_cache import BF16, F32, check_attend, device, qm, to_dtype  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def sharp(n, new, group=4, seed=41, dim=128):
    """A cache and queries whose rows the prompt kernel lists to be done again, all of
    them: scores far apart, and a value channel that is always 0."""
    c = ko.Cache([n], 1, dim, 16, seed=seed)
    for t in range(n):
        row = c.cell(c.v, 0, 0, t)[:8 * dim].reshape(dim // 32, 16, 16)[:, t % 16]
        row[0, 5] = 0x88
    q = np.random.default_rng(seed + 1).standard_normal((new, group, dim)) * 20.0
    return c, q


@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_offsets_that_go_back(qm, dtype, weights):  # noqa: F811
    """Offsets 0, N, 0, N, 0, N: three sequences with the same N rows, so three times as
    many rows to be done again as the list has room for.  Reported; nothing past the
    workspace is written; the next call is as ever."""
    n, new, heads, dim = 300, 90, 4, 128
    c, q = sharp(n, new)
    one = device(qm, c)
    want = qm.qm_attn_q4_0(one, to_dtype(q, dtype))
    assert qm.qm_device_status(clear=True) == qm.QM_OK
    cache = qm.KVCache(one.k_pages, one.v_pages, one.page_table.repeat(5, 1).contiguous(),
                       torch.full((5,), n, dtype=torch.int32, device="cuda"), head_dim=dim, page_tokens=16)
    qd = to_dtype(q, dtype)
    need = qm.qm_attn_workspace(cache, heads, new, new, weights)
    guard = 1 << 16
    ws = torch.zeros(need + guard, dtype=torch.uint8, device="cuda")
    ws[need:] = 0xA5
    w = torch.zeros((5, 1, cache.max_len), device="cuda")
    out = torch.zeros_like(qd)
    lib = qm.load_library()

    def call(starts):
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        a = qm.QmAttnArgs(qd.data_ptr(), out.data_ptr(), None, w.data_ptr() if weights else None, s.data_ptr(), ws.data_ptr(),
                          need, new, new, heads * dim, heads * dim, cache.max_len, 0, 0, heads, dim ** -0.5,
                          qm.QM_F32 if dtype == F32 else qm.QM_BF16, 0)
        assert lib.qm_attn_q4_0(cache.ref, ctypes.addressof(a), None) == qm.QM_OK
        return qm.qm_device_status(clear=True)

    assert call([0, new, 0, new, 0, new]) == qm.QM_ERR_RANGE
    assert (ws[need:] == 0xA5).all()
    assert (ws[:4096] == 0).all()  # fit for the next call
    assert call([0, new, new, new, new, new]) == qm.QM_OK
    assert torch.equal(out, want)
    # (all rows were listed, so the call before listed each of them three times)
    assert torch.equal(ws[4096:4096 + 4 * new * heads].view(torch.int32).sort().values.cpu(),
                       torch.arange(new * heads, dtype=torch.int32))
    assert (ws[need:] == 0xA5).all()


def test_the_sharp_rows_are_right(qm):  # noqa: F811
    """What the test above runs, with offsets that are in order."""
    c, q = sharp(300, 90)
    for dtype in (F32, BF16):
        check_attend(qm, c, [90], 4, dtype, q=q)
