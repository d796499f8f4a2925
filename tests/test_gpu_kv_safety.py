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
    need = qm.qm_attn_workspace(cache, heads, new, new, weights, exact=True)
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


# ---- workspaces and CUDA graphs

def captured(cache, qm, q, side, **kw):  # noqa: F811
    """A graph of one call on `q` (captured on `side`), its output and its weights."""
    out = torch.empty_like(q)
    w = torch.zeros((cache.n_seqs, cache.n_kv_heads, cache.max_len), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qm.qm_attn_q4_0(cache, q, out=out, weights=w, **kw)
    return g, out, w


def replay(g, out, w):
    w.zero_()
    g.replay()
    torch.cuda.synchronize()
    return out.clone(), w.clone()


@pytest.mark.parametrize("new", [1, 3, 90], ids=["step", "draft", "prompt"])
def test_a_graph_keeps_its_workspace(qm, new):  # noqa: F811
    """Capture after a warm-up, then larger calls on the same stream and new tensors in
    whatever memory became free: replays write nothing but their outputs, and answer as before."""
    c = ko.Cache([900, 1200, 700], 2, 128, 64, seed=43)
    cache = device(qm, c)
    side = torch.cuda.Stream()
    q = torch.randn((3 * new, 8, 128), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = qm.qm_attn_q4_0(cache, q, weights=torch.zeros((3, 2, cache.max_len), device="cuda"))
    g, out, w = captured(cache, qm, q, side)
    first = replay(g, out, w)
    assert torch.equal(first[0], want)
    with torch.cuda.stream(side):  # needs more than the call that was captured
        qm.qm_attn_q4_0(cache, torch.randn((3 * 400, 8, 128), device="cuda"),
                        weights=torch.zeros((3, 2, cache.max_len), device="cuda"))
    torch.cuda.synchronize()
    others = []
    with torch.cuda.stream(side):
        for size in (1 << 12, 1 << 18, 1 << 21, 1 << 23) * 3:
            others.append(torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(3):
        again = replay(g, out, w)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        assert all(bool((x == 0x5A).all()) for x in others)


def test_captures_without_a_call_before_and_on_two_streams(qm):  # noqa: F811
    """Two graphs captured on one stream that has seen no call, replayed alone, in turn
    and at the same time on two streams, with eager calls between."""
    c = ko.Cache([5000, 3000], 2, 128, 64, seed=44)
    cache = device(qm, c)
    qs = [torch.randn((2 * n, 8, 128), device="cuda") for n in (1, 2)]
    side = torch.cuda.Stream()
    graphs = [captured(cache, qm, q, side) for q in qs]
    fresh = device(qm, c)
    want = []
    for q in qs:
        w = torch.zeros((2, 2, cache.max_len), device="cuda")
        want.append((qm.qm_attn_q4_0(fresh, q, weights=w), w))
    for order in ((1,), (0, 1), (1, 0, 0)):  # (the second graph first)
        for i in order:
            got = replay(*graphs[i])
            assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])
    with torch.cuda.stream(side):
        assert torch.equal(qm.qm_attn_q4_0(cache, qs[0]), want[0][0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for _, _, w in graphs:
            w.zero_()
        torch.cuda.synchronize()
        for s, (g, _, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i, (_, out, w) in enumerate(graphs):
            assert torch.equal(out, want[i][0]) and torch.equal(w, want[i][1])


def test_a_workspace_of_the_callers(qm):  # noqa: F811
    """One workspace for two caches, in eager and captured calls; too small or the wrong
    type is refused."""
    caches = [device(qm, ko.Cache([900, 1200], 2, 128, 64, seed=s)) for s in (45, 46)]
    q = torch.randn((2, 8, 128), device="cuda")
    p = torch.randn((160, 8, 128), device="cuda")
    want = [[qm.qm_attn_q4_0(x, y) for y in (q, p)] for x in caches]
    need = qm.qm_attn_workspace(caches[0], 8, 160, 80)  # for the steps too
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws[:qm.ATTN_WORKSPACE_ZEROED] = 0
    for x, (a, b) in zip(caches, want):
        for _ in range(2):
            assert torch.equal(qm.qm_attn_q4_0(x, q, workspace=ws), a)
            assert torch.equal(qm.qm_attn_q4_0(x, p, workspace=ws), b)
    assert (ws[:qm.ATTN_WORKSPACE_ZEROED] == 0).all()
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        qm.qm_attn_q4_0(caches[0], q, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0][0])
    with pytest.raises(qm.QMError) as e:
        qm.qm_attn_q4_0(caches[0], q, workspace=ws[:qm.qm_attn_workspace(caches[0], 8, 2, 1, exact=True) // 256 * 256 - 256])
    assert e.value.code == qm.QM_ERR_WORKSPACE
    with pytest.raises(TypeError):
        qm.qm_attn_q4_0(caches[0], q, workspace=ws.float())
    with pytest.raises(ValueError):
        qm.qm_attn_q4_0(caches[0], q, workspace=ws.cpu())
    # an explicit stream, eager and captured
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qm.qm_attn_q4_0(caches[1], q, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want[1][0])


# ---- calls that were refused though nothing is wrong with them

@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_rows_that_no_sequence_has_and_a_max_q_of_0(qm, dim, weights):  # noqa: F811
    """max_q = 0 says that no sequence has rows: nothing is touched, and one that has more
    than a row all the same is reported."""
    cache = device(qm, ko.Cache([40, 50], 1, dim, 16, seed=47))
    q = torch.randn((6, 2, dim), device="cuda")
    out = torch.full_like(q, 3.0)
    w = torch.full((2, 1, cache.max_len), 0.5, device="cuda") if weights else None
    kw = dict(out=out, max_q=0, weights=w)
    qm.qm_attn_q4_0(cache, q, q_starts=torch.zeros(3, dtype=torch.int32, device="cuda"), **kw)
    assert qm.qm_device_status(clear=True) == qm.QM_OK
    assert (out == 3.0).all() and (w is None or (w == 0.5).all())
    qm.qm_attn_q4_0(cache, q, q_starts=torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda"), **kw)
    assert qm.qm_device_status(clear=True) == qm.QM_ERR_RANGE


def test_evicting_caches_that_can_hold_nothing(qm):  # noqa: F811
    def empty():
        return qm.KVCache(torch.empty((0, 2, 576), dtype=torch.uint8, device="cuda"),
                          torch.empty((0, 2, 576), dtype=torch.uint8, device="cuda"),
                          torch.empty((3, 0), dtype=torch.int32, device="cuda"),
                          torch.zeros(3, dtype=torch.int32, device="cuda"), head_dim=64, page_tokens=16)

    a, b = empty(), empty()
    b.lengths += 7
    kept, w = qm.qm_kv_evict_q4_0(a, b, torch.empty((3, 2, 0), device="cuda"), 5, sinks=1, recent=2)
    assert (kept == -1).all() and (w == 0).all() and kept.shape == (3, 2, 5)
    assert b.lengths.tolist() == [0, 0, 0] and qm.qm_device_status(clear=True) == qm.QM_OK


def test_one_heads_stride_does_not_count(qm):  # noqa: F811
    """A single head's rows as a view whose head stride is anything."""
    c = ko.Cache([60], 1, 64, 16, seed=48)
    cache = device(qm, c)
    x = torch.randn((1, 5, 64), device="cuda")
    view = x.transpose(0, 1)  # [5, 1, 64], head stride 320
    assert view.stride() == (64, 320, 1)
    qm.qm_kv_append_q4_0(cache, view, view)
    k, v = qm.qm_kv_read_q4_0(cache, 5)
    qm.qm_kv_append_q4_0(cache, view.clone(memory_format=torch.contiguous_format), view.contiguous())
    again = qm.qm_kv_read_q4_0(cache, 5)
    assert torch.equal(k, again[0]) and torch.equal(v, again[1])
    out = torch.empty((1, 5, 64), device="cuda").transpose(0, 1)
    got = qm.qm_attn_q4_0(cache, view, out=out)
    assert torch.equal(got, qm.qm_attn_q4_0(cache, x[0].unsqueeze(1).contiguous()))
    with pytest.raises(ValueError):  # two heads that do not lie together
        qm.qm_attn_q4_0(cache, torch.randn((2, 5, 64), device="cuda").transpose(0, 1))
