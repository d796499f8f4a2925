"""The 4-bit key/value cache without a GPU: refusals on the host (before any
CUDA call), the binding's checks, workspace sizes, and pins of the plain
implementation that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

import bit_block_quantized_qm_gb300 as qm
import kv_oracle as ko
from bit_block_quantized_qm_gb300 import build as qm_build


@pytest.fixture(scope="module")
def lib():
    qm_build.build()
    return qm.load_library()


K, V, T, L = 0x10000000, 0x40000000, 0x70000000, 0x71000000  # never dereferenced
Q, O, LSE, W, S, WS = 0x80000000, 0x90000000, 0xA0000000, 0xB0000000, 0xC0000000, 0xD0000000


def cache(**kw):
    d = dict(k_pages=K, v_pages=V, page_table=T, lengths=L, n_pages=10, table_stride=5, max_len=80, n_seqs=2,
             n_kv_heads=2, head_dim=64, page_tokens=16, reserved=0)
    d.update(kw)
    return qm.QmKVCache(*[d[f] for f, _ in qm.QmKVCache._fields_])


def args(**kw):
    d = dict(q=Q, out=O, lse=LSE, weights=W, q_starts=S, workspace=WS, workspace_bytes=1 << 28, n_tokens=6, max_q=3,
             q_stride=256, out_stride=256, weights_stride=80, window=0, sinks=0, n_heads=4, scale=0.125, dtype=0,
             reserved=0)
    d.update(kw)
    return qm.QmAttnArgs(*[d[f] for f, _ in qm.QmAttnArgs._fields_])


def attn(lib, c=None, a=None):
    c = cache() if c is None else c
    a = args() if a is None else a
    return lib.qm_attn_q4_0(ctypes.addressof(c), ctypes.addressof(a), None)


def append(lib, c=None, k=Q, v=O, dtype=0, n=6, ks=128, vs=128, starts=S):
    c = cache() if c is None else c
    return lib.qm_kv_append_q4_0(ctypes.addressof(c), k, v, dtype, n, ks, vs, starts, None)


def evict(lib, c=None, to=None, w=W, ws=80, budget=40, sinks=4, recent=8, kept=LSE, wo=O, os_=40):
    c = cache() if c is None else c
    to = cache(k_pages=K + (1 << 24), v_pages=V + (1 << 24), page_table=T + 4096, lengths=L + 4096) if to is None else to
    return lib.qm_kv_evict_q4_0(ctypes.addressof(c), ctypes.addressof(to), w, ws, budget, sinks, recent, kept, wo, os_,
                                None)


# What a call with nothing wrong answers here: there is no device, or the address is no device memory.
FINE = (qm.QM_ERR_CUDA, qm.QM_ERR_POINTER)


def test_struct_sizes_and_calls_that_pass_the_checks(lib):
    assert ctypes.sizeof(qm.QmKVCache) == 80 and ctypes.sizeof(qm.QmAttnArgs) == 136
    assert attn(lib) in FINE and append(lib) in FINE and evict(lib) in FINE
    c = cache()
    assert lib.qm_kv_read_q4_0(ctypes.addressof(c), Q, O, 6, S, None) in FINE


@pytest.mark.parametrize("bad", [dict(n_seqs=-1), dict(n_seqs=65536), dict(n_kv_heads=0), dict(n_kv_heads=40000),
                                 dict(head_dim=0), dict(head_dim=48), dict(head_dim=288), dict(page_tokens=8),
                                 dict(page_tokens=48), dict(page_tokens=1 << 17), dict(n_pages=-1),
                                 dict(n_pages=1 << 32), dict(table_stride=-1), dict(table_stride=1 << 32),
                                 dict(max_len=-1), dict(max_len=81), dict(max_len=1 << 31, table_stride=1 << 30),
                                 dict(reserved=1)], ids=str)
def test_cache_shapes_refused(lib, bad):
    c = cache(**bad)
    assert attn(lib, c) == qm.QM_ERR_SHAPE
    assert append(lib, c) == qm.QM_ERR_SHAPE
    assert lib.qm_kv_read_q4_0(ctypes.addressof(c), Q, O, 6, S, None) == qm.QM_ERR_SHAPE
    assert evict(lib, c) == qm.QM_ERR_SHAPE and evict(lib, to=c) == qm.QM_ERR_SHAPE
    assert lib.qm_attn_workspace(ctypes.addressof(c), 4, 6, 3, 0) == qm.QM_ERR_SHAPE


@pytest.mark.parametrize("bad,code", [
    (dict(k_pages=None), qm.QM_ERR_NULL), (dict(v_pages=None), qm.QM_ERR_NULL), (dict(page_table=None), qm.QM_ERR_NULL),
    (dict(lengths=None), qm.QM_ERR_NULL), (dict(k_pages=K + 8), qm.QM_ERR_ALIGN), (dict(v_pages=V + 4), qm.QM_ERR_ALIGN),
    (dict(page_table=T + 2), qm.QM_ERR_ALIGN), (dict(lengths=L + 1), qm.QM_ERR_ALIGN),
    (dict(v_pages=K + 64), qm.QM_ERR_ALIAS)], ids=str)
def test_cache_pointers_refused(lib, bad, code):
    c = cache(**bad)
    assert attn(lib, c) == code and append(lib, c) == code and evict(lib, c) == code


@pytest.mark.parametrize("bad,code", [
    (dict(n_heads=0), qm.QM_ERR_SHAPE), (dict(n_heads=3), qm.QM_ERR_SHAPE), (dict(n_heads=-2), qm.QM_ERR_SHAPE),
    (dict(n_tokens=-1), qm.QM_ERR_SHAPE), (dict(n_tokens=1 << 31), qm.QM_ERR_SHAPE), (dict(max_q=-1), qm.QM_ERR_SHAPE),
    (dict(n_tokens=7, q_starts=None), qm.QM_ERR_SHAPE), (dict(q_stride=252), qm.QM_ERR_SHAPE),
    (dict(q_stride=258), qm.QM_ERR_SHAPE), (dict(out_stride=128), qm.QM_ERR_SHAPE),
    (dict(weights_stride=79), qm.QM_ERR_SHAPE), (dict(window=-1), qm.QM_ERR_SHAPE), (dict(sinks=-1), qm.QM_ERR_SHAPE),
    (dict(scale=math.nan), qm.QM_ERR_SHAPE), (dict(scale=math.inf), qm.QM_ERR_SHAPE), (dict(dtype=2), qm.QM_ERR_SHAPE),
    (dict(reserved=1), qm.QM_ERR_SHAPE), (dict(q=None), qm.QM_ERR_NULL), (dict(out=None), qm.QM_ERR_NULL),
    (dict(q=Q + 4), qm.QM_ERR_ALIGN), (dict(out=O + 8), qm.QM_ERR_ALIGN), (dict(lse=LSE + 2), qm.QM_ERR_ALIGN),
    (dict(weights=W + 1), qm.QM_ERR_ALIGN), (dict(q_starts=S + 2), qm.QM_ERR_ALIGN),
    (dict(out=Q + 1024), qm.QM_ERR_ALIAS), (dict(out=K), qm.QM_ERR_ALIAS), (dict(lse=O), qm.QM_ERR_ALIAS),
    (dict(weights=O + 64), qm.QM_ERR_ALIAS), (dict(lse=T), qm.QM_ERR_ALIAS), (dict(weights=L - 16), qm.QM_ERR_ALIAS),
    (dict(out=S - 64), qm.QM_ERR_ALIAS)], ids=str)
def test_attention_arguments_refused(lib, bad, code):
    assert attn(lib, a=args(**bad)) == code


def test_attention_without_options_and_bf16(lib):
    assert attn(lib, a=args(lse=None, weights=None, q_starts=None)) in FINE
    assert attn(lib, a=args(dtype=1, q=Q + 8, out=O + 8)) in FINE
    assert attn(lib, a=args(dtype=1, q=Q + 4)) == qm.QM_ERR_ALIGN
    assert attn(lib, a=args(n_tokens=0, q=None, out=None)) == qm.QM_OK
    assert attn(lib, c=cache(n_seqs=0, k_pages=None, lengths=None)) == qm.QM_OK
    assert lib.qm_attn_q4_0(None, None, None) == qm.QM_ERR_NULL
    c = cache()
    assert lib.qm_attn_q4_0(ctypes.addressof(c), None, None) == qm.QM_ERR_NULL


def test_workspace(lib):
    c = cache()
    for heads, n, m, w in ((4, 6, 3, 1), (4, 2, 1, 1), (4, 2, 1, 0), (2, 400, 200, 1)):
        need = lib.qm_attn_workspace(ctypes.addressof(c), heads, n, m, w)
        assert need >= 0
        if need:
            a = dict(n_heads=heads, n_tokens=n, max_q=m, weights=W if w else None, q_stride=heads * 64,
                     out_stride=heads * 64)
            assert attn(lib, a=args(workspace_bytes=need, **a)) in FINE
            assert attn(lib, a=args(workspace_bytes=need - 1, **a)) == qm.QM_ERR_WORKSPACE
            assert attn(lib, a=args(workspace=None, **a)) == qm.QM_ERR_NULL
            assert attn(lib, a=args(workspace=WS + 8, **a)) == qm.QM_ERR_ALIGN
            assert attn(lib, a=args(workspace=Q, **a)) == qm.QM_ERR_ALIAS
    assert lib.qm_attn_workspace(ctypes.addressof(c), 3, 6, 3, 1) == qm.QM_ERR_SHAPE
    assert lib.qm_attn_workspace(ctypes.addressof(c), 4, -1, 3, 1) == qm.QM_ERR_SHAPE
    assert lib.qm_attn_workspace(None, 4, 6, 3, 1) == qm.QM_ERR_NULL


@pytest.mark.parametrize("bad,code", [
    (dict(k=None), qm.QM_ERR_NULL), (dict(v=None), qm.QM_ERR_NULL), (dict(n=-1), qm.QM_ERR_SHAPE),
    (dict(n=7, starts=None), qm.QM_ERR_SHAPE), (dict(ks=124), qm.QM_ERR_SHAPE), (dict(vs=130), qm.QM_ERR_SHAPE),
    (dict(dtype=-1), qm.QM_ERR_SHAPE), (dict(k=Q + 4), qm.QM_ERR_ALIGN), (dict(v=O + 8), qm.QM_ERR_ALIGN),
    (dict(starts=S + 1), qm.QM_ERR_ALIGN), (dict(k=K), qm.QM_ERR_ALIAS), (dict(v=K - 16), qm.QM_ERR_ALIAS)], ids=str)
def test_append_arguments_refused(lib, bad, code):
    assert append(lib, **bad) == code


def test_append_nothing(lib):
    assert append(lib, n=0, k=None, v=None) == qm.QM_OK
    assert append(lib, dtype=1, k=Q + 8) in FINE and append(lib, dtype=1, k=Q + 4) == qm.QM_ERR_ALIGN


def test_read_arguments_refused(lib):
    c = cache()

    def read(k=Q, v=O, n=6, starts=S):
        return lib.qm_kv_read_q4_0(ctypes.addressof(c), k, v, n, starts, None)

    assert read(k=None) == qm.QM_ERR_NULL and read(v=None) == qm.QM_ERR_NULL
    assert read(n=-1) == qm.QM_ERR_SHAPE and read(n=7, starts=None) == qm.QM_ERR_SHAPE
    assert read(k=Q + 8) == qm.QM_ERR_ALIGN and read(k=O) == qm.QM_ERR_ALIAS and read(v=V) == qm.QM_ERR_ALIAS
    assert read(n=0, k=None, v=None) == qm.QM_OK


@pytest.mark.parametrize("bad,code", [
    (dict(w=None), qm.QM_ERR_NULL), (dict(kept=None), qm.QM_ERR_NULL), (dict(wo=None), qm.QM_ERR_NULL),
    (dict(ws=79), qm.QM_ERR_SHAPE), (dict(os_=39), qm.QM_ERR_SHAPE), (dict(budget=-1), qm.QM_ERR_SHAPE),
    (dict(sinks=-1), qm.QM_ERR_SHAPE), (dict(recent=-1), qm.QM_ERR_SHAPE), (dict(recent=37), qm.QM_ERR_SHAPE),
    (dict(w=W + 2), qm.QM_ERR_ALIGN), (dict(kept=LSE + 1), qm.QM_ERR_ALIGN), (dict(wo=O + 2), qm.QM_ERR_ALIGN),
    (dict(wo=W + 64), qm.QM_ERR_ALIAS), (dict(wo=W, os_=40), qm.QM_ERR_ALIAS), (dict(kept=W), qm.QM_ERR_ALIAS),
    (dict(to=cache(n_seqs=3)), qm.QM_ERR_SHAPE), (dict(to=cache(head_dim=32)), qm.QM_ERR_SHAPE),
    (dict(to=cache(n_kv_heads=1)), qm.QM_ERR_SHAPE), (dict(to=cache(max_len=39)), qm.QM_ERR_SHAPE),
    (dict(to=cache(page_tokens=32)), qm.QM_ERR_SHAPE), (dict(to=cache(table_stride=6)), qm.QM_ERR_SHAPE),
    (dict(to=cache(k_pages=K + (1 << 24), v_pages=V + (1 << 24))), qm.QM_ERR_ALIAS),
    (dict(to=cache(k_pages=V, v_pages=K, page_table=T + 4096)), qm.QM_ERR_ALIAS)], ids=lambda x: str(x)[:40])
def test_evict_arguments_refused(lib, bad, code):
    assert evict(lib, **bad) == code


def test_evict_in_place_passes(lib):
    assert evict(lib, to=cache()) in FINE
    assert evict(lib, to=cache(), wo=W, os_=80) in FINE
    assert evict(lib, c=cache(n_seqs=0), to=cache(n_seqs=0), w=None) == qm.QM_OK


def test_the_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    pages = torch.zeros((4, 1, qm.kv_page_bytes(16, 64)), dtype=torch.uint8)
    with pytest.raises(ValueError):  # not CUDA tensors
        qm.KVCache(pages, pages.clone(), torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                   head_dim=64, page_tokens=16)
    with pytest.raises(TypeError):
        qm.KVCache(pages.float(), pages, torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                   head_dim=64, page_tokens=16)
    assert qm.kv_page_bytes(64, 128) == 4 * 9 * 128


# ---- pins of the plain implementation

def test_quantize_by_hand():
    x = np.zeros(32, np.float32)
    x[3], x[4], x[20] = -8.0, 8.0, 3.4
    q, d = ko.quantize(x)
    assert d == np.float16(1.0)  # -8 / -8: the first of the two sizes decides
    assert q[3] == 0 and q[4] == 15 and q[20] == 11 and q[0] == 8  # 8 clamps to 15: 7 steps
    x[3] = 0.0
    q, d = ko.quantize(x)
    assert d == np.float16(-1.0) and q[4] == 0 and q[20] == 5  # 3.4 / -1 + 8.5 = 5.1
    q, d = ko.quantize(np.full(32, np.nan, np.float32))
    assert (q == 8).all() and d == 0


def test_quantize_error_is_half_a_step():
    x = np.random.default_rng(0).standard_normal((500, 32)).astype(np.float32)
    q, d = ko.quantize(x)
    back = (q.astype(np.float64) - 8) * d.astype(np.float64)[:, None]
    step = np.abs(d.astype(np.float64))[:, None]
    # half a step, a whole one at the clamped end, and the scale's own rounding
    assert (np.abs(back - x) <= np.where(q == 15, 1.0, 0.5) * step + 8 * step * 2.0 ** -11 + 1e-6).all()


def test_attention_by_hand():
    c = ko.Cache([3], 1, 32, 16, seed=1)
    for t, (kv, vv) in enumerate(((1.0, 2.0), (2.0, -1.0), (0.0, 5.0))):
        ko.store(c, c.k, 0, 0, t, np.eye(32)[0] * kv)
        ko.store(c, c.v, 0, 0, t, np.ones(32) * vv)
    q = np.zeros((1, 1, 32))
    q[0, 0, 0] = math.log(2.0)
    out, lse, w, *_ = ko.attend(c, q, [0, 1], 1, 1.0)
    # scores log 2, 2 log 2, 0: weights 2, 4, 1 of 7
    np.testing.assert_allclose(out[0, 0], (2 * 2.0 - 4 + 5) / 7, rtol=1e-3)  # (binary16 scales)
    np.testing.assert_allclose(lse[0, 0], math.log(7), rtol=1e-3)
    np.testing.assert_allclose(w[0, 0], [2 / 7, 4 / 7, 1 / 7], rtol=2e-3)
    out, _, w, *_ = ko.attend(c, q, [0, 1], 1, 1.0, window=1, sinks=1)
    np.testing.assert_allclose(w[0, 0], [2 / 3, 0, 1 / 3], rtol=2e-3)


def test_visible_by_brute_force():
    for window in (0, 1, 3, 9):
        for sinks in (0, 2, 7):
            see = ko.visible(np.arange(-2, 6), 6, window, sinks)
            for i, p in enumerate(range(-2, 6)):
                for j in range(6):
                    want = j <= p and (window == 0 or p - j < window or j < sinks)
                    assert see[i, j] == want


def test_evict_by_hand():
    w = np.array([0.0, 5.0, 1.0, 5.0, np.nan, -1.0, 9.0, 0.5])
    assert ko.evict(w, 8, 4, 1, 1).tolist() == [0, 1, 6, 7]  # of the equal scores the lower position
    assert ko.evict(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]  # NaN goes first
    assert ko.evict(w, 3, 4, 1, 1).tolist() == [0, 1, 2]
