"""GPU tests of the 4-bit key/value cache: append, read, attention, accumulated
weights and eviction, through the Python entry points, against the plain 64-bit
implementation in kv_oracle.

Bounds on the attention, element by element.  With u the error that a product
is allowed relative to its size, a score is off by at most ds = u * reach (reach
= scale * sum |q k|) plus f32 rounding of the logit, a probability by a factor
exp(2 ds), and the output by mass * (2 ds + u + rounding), mass = sum p |v|.
For f32 rows u = 2^-20 (products to 2^-21, as much again for the sums); for bf16
rows u = 2^-11 (keys, values and probabilities to 11 bits: 2^-12 each, two of
them in a product), and the output's own rounding of 2^-8 |out|.
"""
import numpy as np
import pytest

import kv_oracle as ko

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def qm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_block_quantized_qm_gb300 import build as qm_build
    qm_build.build()
    import bit_block_quantized_qm_gb300 as qm
    qm.load_library()
    torch.cuda.set_device(0)
    return qm


def device(qm, c, max_len=None):
    return qm.KVCache(torch.from_numpy(c.k.copy()).cuda(), torch.from_numpy(c.v.copy()).cuda(),
                      torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lengths.copy()).cuda(), head_dim=c.dim,
                      page_tokens=c.page, max_len=max_len)


def starts_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def to_dtype(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(dtype)


def bounds(got_dtype, out, lse, mass, reach):
    f32 = got_dtype == torch.float32
    u = 2.0 ** -20 if f32 else 2.0 ** -11
    ds = (u * reach + 2.0 ** -21 * np.where(np.isfinite(lse), np.abs(lse), 0) + 2.0 ** -20)[..., None]
    tol = mass * (2 * ds + u + 2.0 ** -20) + 1e-30
    if not f32:
        tol = tol + 2.0 ** -8 * np.abs(out)
    return tol, ds[..., 0]


def check_attend(qm, c, new, heads, dtype=torch.float32, window=0, sinks=0, scale=None, q_gain=1.5, weights=False,
                 seed=5, max_len=None, cache=None, q=None):
    g = np.random.default_rng(seed)
    rows = int(sum(new))
    starts = starts_of(new)
    if q is None:
        q = g.standard_normal((rows, heads, c.dim)) * q_gain
    qd = to_dtype(q, dtype)
    cache = device(qm, c, max_len) if cache is None else cache
    w0 = g.random((len(new), c.heads, cache.max_len)).astype(np.float32)
    w = torch.from_numpy(w0.copy()).cuda() if weights else None
    sc = c.dim ** -0.5 if scale is None else scale
    kw = dict(window=window, sinks=sinks, scale=scale, q_starts=torch.from_numpy(starts).cuda(),
              max_q=max(list(new) + [1]), return_lse=True)
    out, lse = qm.qm_attn_q4_0(cache, qd, weights=w, **kw)
    torch.cuda.synchronize()
    assert qm.qm_device_status(clear=True) == qm.QM_OK
    o, l, added, mass, reach = ko.attend(c, qd.float().cpu().numpy(), starts, heads, np.float32(sc), window, sinks)
    tol, ds = bounds(dtype, o, l, mass, reach)
    got, got_l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    empty = np.isinf(l)
    assert np.array_equal(np.isneginf(got_l), empty)
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], np.abs(got - o)[bad][:4], tol[bad][:4])
    assert (got[empty] == 0).all()
    bad = ~empty & ~(np.abs(got_l - np.where(empty, 0, l)) <= ds + 2.0 ** -20)
    assert not bad.any(), (np.argwhere(bad)[:4], got_l[bad][:4], l[bad][:4])
    if weights:
        got_w = w.cpu().numpy().astype(np.float64)
        n = added.shape[2]
        # each probability to exp(2 ds); sums of non-negative terms
        tol_w = added * (4 * ds.max(initial=0) + 2.0 ** -18) + 2.0 ** -22 * (w0[:, :, :n] + added) + 1e-7
        bad = ~(np.abs(got_w[:, :, :n] - (w0[:, :, :n] + added)) <= tol_w)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
        for b, length in enumerate(c.lengths):  # nothing past a sequence's length is touched
            assert np.array_equal(got_w[b, :, int(length):], w0[b, :, int(length):].astype(np.float64))
    again, lse2 = qm.qm_attn_q4_0(cache, qd, **kw)
    assert torch.equal(again.view(torch.int16 if dtype == torch.bfloat16 else torch.int32),
                       out.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)), "not deterministic"
    assert torch.equal(lse2, lse)
    return out, lse


F32, BF16 = torch.float32, torch.bfloat16

# lengths, new rows, kv heads, group, dim, page, window, sinks
STEPS = [
    ([1], [1], 1, 1, 128, 16, 0, 0),
    ([15, 16, 17], [1, 1, 1], 2, 4, 128, 16, 0, 0),
    ([63, 64, 65, 129], [1, 1, 1, 1], 2, 4, 128, 64, 0, 0),
    ([777], [1], 8, 4, 128, 16, 0, 0),
    ([1000, 1, 513, 0, 300], [1, 1, 1, 0, 1], 2, 3, 64, 32, 0, 0),
    ([2300, 700], [1, 1], 1, 8, 128, 256, 0, 0),
    ([900, 80], [1, 1], 2, 16, 64, 16, 0, 0),
    ([700, 701], [1, 1], 3, 7, 128, 32, 0, 0),
    ([2500, 40, 1200], [1, 1, 1], 2, 4, 128, 64, 1000, 4),
    ([2500, 40, 1200], [1, 1, 1], 2, 1, 64, 128, 33, 0),
    ([600, 601], [1, 1], 1, 2, 128, 16, 1, 0),
    ([600, 601], [1, 1], 1, 2, 128, 16, 1, 2),
    ([600, 100], [1, 1], 1, 4, 64, 16, 50, 400),
    ([300, 5, 33], [5, 5, 2], 2, 4, 128, 32, 0, 0),
    ([300, 5, 33], [7, 5, 3], 4, 1, 64, 16, 20, 3),
    ([300, 2, 33, 0], [7, 5, 3, 2], 2, 2, 128, 16, 0, 0),   # rows before the first token
    ([200, 64], [1, 1], 2, 4, 96, 16, 0, 0),
    ([200, 64], [3, 1], 2, 2, 32, 64, 100, 1),
    ([150, 70], [2, 2], 1, 4, 256, 16, 0, 0),
    ([5000], [1], 1, 4, 128, 64, 0, 0),
]
PROMPTS = [
    ([200], [200], 2, 4, 128, 64, 0, 0),
    ([129, 257, 40], [129, 100, 40], 2, 4, 128, 16, 0, 0),
    ([300, 190], [300, 190], 1, 1, 64, 32, 0, 0),
    ([300, 190], [150, 190], 1, 3, 128, 32, 60, 3),
    ([260, 100], [260, 33], 2, 2, 64, 16, 100, 4),
    ([450], [40], 1, 8, 128, 128, 0, 0),
    ([400], [400], 1, 2, 128, 256, 1, 0),
    ([100, 30], [140, 20], 1, 4, 128, 16, 0, 0),              # rows before the first token
    ([300], [300], 1, 7, 128, 16, 17, 40),
    ([130], [130], 2, 2, 96, 16, 0, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", STEPS + PROMPTS, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_attention(qm, case, dtype):
    lengths, new, kv, group, dim, page, window, sinks = case
    c = ko.Cache(lengths, kv, dim, page, seed=len(lengths) + page)
    check_attend(qm, c, new, kv * group, dtype, window, sinks, weights=True)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 90], ids=["step", "prompt"])
def test_attention_scale_and_sharp_scores(qm, dtype, new):
    c = ko.Cache([333, 95], 2, 128, 32, seed=3, scale=0.4)
    check_attend(qm, c, [new, min(new, 90)], 8, dtype, scale=0.21, q_gain=3.0, weights=True)
    check_attend(qm, c, [new, min(new, 90)], 8, dtype, scale=0.0)
    check_attend(qm, c, [new, min(new, 90)], 8, dtype, scale=-0.07)


# Between the two: more rows than a step's and few in all, and long prompts
# (more token tiles than any ring in the kernels has slots, windows that skip some).
BETWEEN = [
    ([1700], [50], 2, 4, 128, 16, 0, 0),
    ([900, 33, 400], [40, 33, 2], 1, 6, 64, 32, 0, 0),
    ([1500, 700], [25, 17], 2, 8, 128, 128, 300, 5),
    ([70], [63], 4, 4, 128, 64, 0, 0),
    ([1650, 1100], [90, 700], 1, 4, 128, 64, 0, 0),
    ([1650], [1650], 1, 2, 64, 16, 0, 0),
    ([2100, 300], [400, 300], 2, 2, 128, 32, 700, 150),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("case", BETWEEN, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_attention_between_and_long(qm, case, weights, dtype):
    lengths, new, kv, group, dim, page, window, sinks = case
    c = ko.Cache(lengths, kv, dim, page, seed=len(lengths) + page)
    check_attend(qm, c, new, kv * group, dtype, window, sinks, weights=weights)


def test_attention_calls_share_a_workspace(qm):
    """Steps, drafts, chunks and prompts in turn on one cache, with weights and without, twice over."""
    c = ko.Cache([640, 300], 2, 128, 32, seed=9)
    cache = device(qm, c)
    first = []
    for turn in range(2):
        for k, (new, weights) in enumerate([(1, True), (200, False), (1, False), (7, True), (130, True), (3, False), (60, False)]):
            out, lse = check_attend(qm, c, [new, new], 8, F32, weights=weights, cache=cache)
            if turn == 0:
                first.append((out.clone(), lse.clone()))
            assert torch.equal(out, first[k][0]) and torch.equal(lse, first[k][1])


@pytest.mark.parametrize("v_scale", [2.0 ** -13, 37.0, 6000.0])
@pytest.mark.parametrize("k_scale", [2.0 ** -12, 1.0, 7000.0])
@pytest.mark.parametrize("new", [1, 70], ids=["step", "prompt"])
def test_attention_scale_range(qm, new, k_scale, v_scale):
    """Scales over the range of binary16; queries sized so that scores stay ordinary."""
    c = ko.Cache([210], 1, 128, 16, seed=9)
    s = c.k[..., :].reshape(c.n_pages, 1, -1, 9 * 128)[..., 8 * 128:].view(np.float16)
    s[:] = (s.astype(np.float32) * (k_scale / 0.1)).astype(np.float16)
    s = c.v[..., :].reshape(c.n_pages, 1, -1, 9 * 128)[..., 8 * 128:].view(np.float16)
    s[:] = (s.astype(np.float32) * (v_scale / 0.1)).astype(np.float16)
    check_attend(qm, c, [new], 4, F32, q_gain=0.1 / k_scale)


@pytest.mark.parametrize("gain", [1e-20, 1e-6, 3e4, 1e12])
@pytest.mark.parametrize("new", [1, 70], ids=["step", "prompt"])
def test_attention_query_range(qm, new, gain):
    """Queries far from 1, brought back by the scale."""
    c = ko.Cache([210], 1, 128, 16, seed=10)
    check_attend(qm, c, [new], 4, F32, q_gain=gain, scale=float(np.float32(0.09 / gain)))


def poison(c, pool, b, h, t, value):
    c.scales(pool, b, h, t)[:] = value


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 3, 120], ids=["step", "draft", "prompt"])
def test_hidden_tokens_do_not_reach_a_row(qm, new, dtype, bad):
    """Non-finite scales in the unused places of the last cell, in the rest of
    the last page, and in tokens outside every row's window."""
    n, window, sinks = 400, 100, 3
    clean = ko.Cache([n], 2, 128, 64, seed=12)
    c = ko.Cache([n], 2, 128, 64, seed=12)
    for pool in (c.k, c.v):
        for h in range(2):
            for t in list(range(n, 448)) + list(range(sinks, n - new + 1 - window)):
                poison(c, pool, 0, h, t, bad)
    a, la = check_attend(qm, clean, [new], 8, dtype, window, sinks)
    cache = device(qm, c)
    q = np.random.default_rng(5).standard_normal((new, 8, 128)) * 1.5
    b, lb = qm.qm_attn_q4_0(cache, to_dtype(q, dtype), window=window, sinks=sinks, return_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert qm.qm_device_status(clear=True) == qm.QM_OK


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("new", [6, 150], ids=["draft", "prompt"])
def test_a_row_that_sees_a_non_finite_token(qm, new, which):
    """Token t is seen by the rows from its position on: those are non-finite where
    the formula is, and every row before it is as without it."""
    n = 300
    t = n - new // 2
    c = ko.Cache([n], 1, 128, 32, seed=13)
    poison(c, c.k if which == "k" else c.v, 0, 0, t, np.nan)
    clean = ko.Cache([n], 1, 128, 32, seed=13)
    q = np.random.default_rng(5).standard_normal((new, 4, 128)) * 1.5
    want, *_ = ko.attend(c, q.astype(np.float32), [0, new], 4, np.float32(128 ** -0.5))
    a = qm.qm_attn_q4_0(device(qm, clean), to_dtype(q, F32))
    b = qm.qm_attn_q4_0(device(qm, c), to_dtype(q, F32)).cpu().numpy()
    before = t - (n - new)
    assert np.isnan(b[np.isnan(want)]).all()
    assert np.isnan(want[before:]).all() and not np.isnan(want[:before]).any()
    # (K and V of token t differ only for rows that see it)
    np.testing.assert_allclose(b[:before], a.cpu().numpy()[:before], rtol=2e-5, atol=2e-6)


def test_non_finite_queries_stay_in_their_row(qm):
    for new in (1, 5, 80):
        c = ko.Cache([200], 1, 128, 16, seed=14)
        q = np.random.default_rng(5).standard_normal((new, 4, 128)).astype(np.float32)
        a = qm.qm_attn_q4_0(device(qm, c), to_dtype(q, F32)).cpu().numpy()
        q2 = q.copy()
        q2[new // 2, 1, 7] = np.nan
        q2[new // 2, 2, 9] = np.inf
        b = qm.qm_attn_q4_0(device(qm, c), to_dtype(q2, F32)).cpu().numpy()
        assert np.isnan(b[new // 2, 1]).all() and not np.isfinite(b[new // 2, 2]).any()
        keep = np.ones((new, 4), bool)
        keep[new // 2, 1:3] = False
        assert np.array_equal(a[keep], b[keep])


def test_strided_rows_uniform_rows_and_outputs_given(qm):
    c = ko.Cache([100, 120], 2, 128, 16, seed=15)
    cache = device(qm, c)
    for new in (1, 3, 60):
        qkv = torch.randn((2 * new, 4 + 4, 128), device="cuda")
        q = qkv[:, :4]
        buf = torch.full((2 * new, 6, 128), 7.0, device="cuda")
        lse = torch.empty((2 * new, 4), device="cuda")
        want = qm.qm_attn_q4_0(cache, q.contiguous(), q_starts=torch.tensor([0, new, 2 * new], dtype=torch.int32).cuda(),
                               max_q=new)
        got, _ = qm.qm_attn_q4_0(cache, q, out=buf[:, :4], lse=lse)
        assert torch.equal(got, want) and (buf[:, 4:] == 7.0).all() and torch.isfinite(lse).all()


def test_rows_of_no_sequence_are_left(qm):
    c = ko.Cache([100, 120], 1, 64, 16, seed=16)
    cache = device(qm, c)
    for new in (1, 40):
        q = torch.randn((2 * new + 5, 2, 64), device="cuda")
        out = torch.full_like(q, 3.0)
        s = torch.tensor([2, 2 + new, 2 + 2 * new], dtype=torch.int32).cuda()
        qm.qm_attn_q4_0(cache, q, out=out, q_starts=s, max_q=new)
        assert (out[:2] == 3.0).all() and (out[2 + 2 * new:] == 3.0).all()
        want = qm.qm_attn_q4_0(cache, q[2:2 + 2 * new].contiguous())
        assert torch.equal(out[2:2 + 2 * new], want)


def test_another_stream_and_calls_in_a_row(qm):
    c = ko.Cache([900, 1200], 2, 128, 64, seed=17)
    cache = device(qm, c)
    q = [torch.randn((2 * n, 8, 128), device="cuda") for n in (1, 64)]
    want = [qm.qm_attn_q4_0(cache, x) for x in q]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [qm.qm_attn_q4_0(cache, x) for _ in range(4) for x in q]
    here = [qm.qm_attn_q4_0(cache, x) for _ in range(4) for x in q]
    torch.cuda.synchronize()
    for i in range(8):
        assert torch.equal(got[i], want[i % 2]) and torch.equal(here[i], want[i % 2])


def test_attention_in_a_cuda_graph(qm):
    c = ko.Cache([900, 1200], 2, 128, 64, seed=18)
    cache = device(qm, c)
    q = torch.randn((2, 8, 128), device="cuda")
    out = torch.empty_like(q)
    w = torch.zeros((2, 2, cache.max_len), device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qm.qm_attn_q4_0(cache, q, out=out, weights=w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qm.qm_attn_q4_0(cache, q, out=out, weights=w)
    for n in (700, 901):
        cache.lengths.copy_(torch.tensor([n, n - 200], dtype=torch.int32))
        q.normal_()
        w.zero_()
        g.replay()
        torch.cuda.synchronize()
        got, gw = out.clone(), w.clone()
        w.zero_()
        want = qm.qm_attn_q4_0(cache, q, weights=w)
        assert torch.equal(got, want) and torch.equal(gw, w)
        assert abs(float(w[0].sum()) - 8.0) < 1e-3


def test_pools_past_four_gigabytes(qm):
    """Pages whose byte offsets do not fit 32 bits."""
    heads, dim, page, n = 8, 128, 256, 700
    per = heads * (page // 16) * 9 * dim
    n_pages = (1 << 32) // per + 8
    c = ko.Cache([n], heads, dim, page, seed=19, spare=0, table_extra=0)
    kp, vp = (torch.zeros((n_pages, heads, per // heads), dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = torch.tensor([n_pages - 1, 3, n_pages - 3], dtype=torch.int32)
    for i, p in enumerate(ids):
        kp[int(p)] = torch.from_numpy(c.k[c.table[0, i]]).cuda()
        vp[int(p)] = torch.from_numpy(c.v[c.table[0, i]]).cuda()
    cache = qm.KVCache(kp, vp, ids[None].cuda().contiguous(), torch.tensor([n], dtype=torch.int32).cuda(), head_dim=dim,
                       page_tokens=page)
    for new in (1, 64):
        check_attend(qm, c, [new], 16, F32, cache=cache, weights=True)
    # append, read and evict there too
    rows = torch.randn((3, 2, heads, dim), device="cuda")
    qm.qm_kv_append_q4_0(cache, rows[:, 0], rows[:, 1])
    k, v = qm.qm_kv_read_q4_0(cache, 3)
    for t in range(3):
        for h in range(heads):
            ko.store(c, c.k, 0, h, n - 3 + t, rows[t, 0, h].cpu().numpy())
            ko.store(c, c.v, 0, h, n - 3 + t, rows[t, 1, h].cpu().numpy())
    for h in range(heads):
        assert np.array_equal(k[:, h].cpu().numpy(), ko_f32(c.values(c.k, 0, h)[-3:]))
        assert np.array_equal(v[:, h].cpu().numpy(), ko_f32(c.values(c.v, 0, h)[-3:]))
    w = torch.rand((1, heads, cache.max_len), device="cuda")
    kept, _ = qm.qm_kv_evict_q4_0(cache, cache, w, 300, 4, 32)
    k, _ = qm.qm_kv_read_q4_0(cache, 300)
    for h in range(heads):
        assert np.array_equal(k[:, h].cpu().numpy(), ko_f32(c.values(c.k, 0, h)[kept[0, h].cpu().numpy()]))


def ko_f32(x):
    return np.asarray(x, np.float32)


@pytest.mark.parametrize("new", [1, 40], ids=["step", "prompt"])
def test_what_only_the_device_sees_is_checked(qm, new):
    """Missing or wild pages, wild lengths and offsets: reported, nothing faults."""
    c = ko.Cache([200, 180], 1, 128, 16, seed=20)
    q = torch.randn((2 * new, 2, 128), device="cuda")
    k = torch.randn((2 * new, 1, 128), device="cuda")
    starts = torch.tensor([0, new, 2 * new], dtype=torch.int32).cuda()

    def spoil(what):
        cache = device(qm, c)
        s = starts.clone()
        if what == "missing page":
            cache.page_table[0, 3] = -1
        elif what == "wild page":
            cache.page_table[1, 2] = 1 << 30
        elif what == "long":
            cache.lengths[0] = 1 << 30
        elif what == "negative":
            cache.lengths[1] = -5
        elif what == "offsets":
            s[1] = 1 << 30
        return cache, s

    for what in ("missing page", "wild page", "long", "negative", "offsets"):
        cache, s = spoil(what)
        out = qm.qm_attn_q4_0(cache, q, q_starts=s, max_q=new)
        assert qm.qm_device_status(clear=True) == qm.QM_ERR_RANGE, what
        assert qm.qm_device_status(clear=True) == qm.QM_OK
        if what in ("missing page", "long"):  # the other sequence is untouched by it
            good = qm.qm_attn_q4_0(device(qm, c), q, q_starts=starts, max_q=new)
            assert torch.equal(out[new:], good[new:])
    cache, s = spoil("long")
    qm.qm_kv_append_q4_0(cache, k, k, q_starts=s)
    assert qm.qm_device_status(clear=True) == qm.QM_ERR_RANGE
    cache, s = spoil("negative")
    qm.qm_kv_read_q4_0(cache, 2 * new, q_starts=s)
    assert qm.qm_device_status(clear=True) == qm.QM_ERR_RANGE


# ---- append and read

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [([1], [1], 1, 128, 16), ([40, 16, 0, 33], [40, 1, 0, 17], 3, 64, 16),
                                  ([300, 70], [300, 5], 2, 128, 64), ([31], [31], 1, 32, 16), ([50], [20], 2, 256, 32),
                                  ([50], [20], 2, 96, 32)],
                         ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_append_and_read(qm, case, dtype):
    lengths, new, heads, dim, page = case
    c = ko.Cache(lengths, heads, dim, page, seed=21)
    cache = device(qm, c)
    rows = int(sum(new))
    g = np.random.default_rng(22)
    kv = g.standard_normal((rows, 2, heads, dim)) * np.exp(g.standard_normal((rows, 2, heads, 1)) * 3)
    kv[0, 0, 0, :32] = 0.0
    kv[0, 1, 0, 3:5] = (-9.0, 9.0)  # two elements of the same size: the first one's sign counts
    kv = to_dtype(kv, dtype)
    starts = starts_of(new)
    qm.qm_kv_append_q4_0(cache, kv[:, 0], kv[:, 1], q_starts=torch.from_numpy(starts).cuda())
    k, v = qm.qm_kv_read_q4_0(cache, rows, q_starts=torch.from_numpy(starts).cuda())
    torch.cuda.synchronize()
    assert qm.qm_device_status(clear=True) == qm.QM_OK
    host = kv.float().cpu().numpy()
    for b, m in enumerate(new):
        for i in range(m):
            for h in range(heads):
                ko.store(c, c.k, b, h, lengths[b] - m + i, host[starts[b] + i, 0, h])
                ko.store(c, c.v, b, h, lengths[b] - m + i, host[starts[b] + i, 1, h])
    # every byte of the pools, those that were not written included
    assert np.array_equal(cache.k_pages.cpu().numpy(), c.k)
    assert np.array_equal(cache.v_pages.cpu().numpy(), c.v)
    for b, m in enumerate(new):
        for h in range(heads):
            sl = slice(starts[b], starts[b] + m)
            assert np.array_equal(k[sl, h].cpu().numpy(), ko_f32(c.values(c.k, b, h)[lengths[b] - m:]))
            assert np.array_equal(v[sl, h].cpu().numpy(), ko_f32(c.values(c.v, b, h)[lengths[b] - m:]))


def test_append_edge_values(qm):
    """Infinities, NaN, zeros of both signs, subnormals, values past binary16."""
    c = ko.Cache([8], 1, 64, 16, seed=23)
    cache = device(qm, c)
    x = np.random.default_rng(24).standard_normal((8, 1, 64)).astype(np.float32)
    x[0, 0, 5] = np.inf
    x[1, 0, 5] = np.nan
    x[2, 0, :32] = np.nan
    x[3, 0, :32] = -0.0
    x[4, 0, :32] = 1e-41
    x[5, 0, 40] = 6e5
    x[6, 0, 41] = -5.3e5
    x[7, 0, :32] *= 1e-7
    d = torch.from_numpy(x).cuda()
    qm.qm_kv_append_q4_0(cache, d, d)
    for t in range(8):
        ko.store(c, c.k, 0, 0, t, x[t, 0])
    got = cache.k_pages.cpu().numpy()
    page = int(c.table[0, 0])
    a, b = got[page, 0], c.k[page, 0]
    assert np.array_equal(a[:512], b[:512])
    sa, sb = a[512:].view(np.float16)[:16], b[512:].view(np.float16)[:16]
    assert np.array_equal(np.isnan(sa), np.isnan(sb)) and np.array_equal(sa[~np.isnan(sa)], sb[~np.isnan(sb)])


def test_append_reports_rows_without_a_place(qm):
    c = ko.Cache([2], 1, 64, 16, seed=25)
    cache = device(qm, c)
    x = torch.randn((5, 1, 64), device="cuda")
    qm.qm_kv_append_q4_0(cache, x, x)  # 5 rows, 2 tokens
    assert qm.qm_device_status(clear=True) == qm.QM_ERR_RANGE
    for t in range(2):
        ko.store(c, c.k, 0, 0, t, x[3 + t, 0].cpu().numpy())
    assert np.array_equal(cache.k_pages.cpu().numpy(), c.k)


# ---- eviction

EVICTS = [  # lengths, budget, sinks, recent, heads, dim, page
    ([100, 37, 0, 64], 64, 4, 16, 2, 128, 16),
    ([1500], 1024, 4, 128, 3, 64, 32),
    ([3000, 1200, 2049], 1000, 0, 0, 2, 128, 64),
    ([500, 33], 32, 8, 24, 1, 64, 16),       # nothing left to choose
    ([500, 33], 1, 0, 0, 1, 64, 16),
    ([40], 0, 0, 0, 1, 64, 16),
    ([70, 90], 200, 3, 5, 2, 32, 16),        # everything stays
    ([1025, 1024, 1026], 1025, 1, 1, 1, 96, 128),
    ([9000], 3001, 5, 100, 2, 64, 256),
]


def scores(kind, shape, g):
    if kind == "random":
        return np.exp(2 * g.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        return g.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    w = (g.standard_normal(shape) * 1e-3).astype(np.float32)  # close together, both signs
    w[g.random(shape) < 0.05] = np.nan
    w[g.random(shape) < 0.05] = np.inf
    w[g.random(shape) < 0.05] = -np.inf
    w[g.random(shape) < 0.1] = 0.0
    w[g.random(shape) < 0.1] = -0.0
    return w


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in place"])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "wild"])
@pytest.mark.parametrize("case", EVICTS, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_evict(qm, case, kind, in_place):
    lengths, budget, sinks, recent, heads, dim, page = case
    c = ko.Cache(lengths, heads, dim, page, seed=26)
    cache = device(qm, c)
    g = np.random.default_rng(27)
    w = scores(kind, (len(lengths), heads, cache.max_len), g)
    dw = torch.from_numpy(w.copy()).cuda()
    if in_place:
        to, to_host = cache, c
        if budget > cache.max_len:
            pytest.skip("a budget past the scores' stride has no place in them")
        kept, wo = qm.qm_kv_evict_q4_0(cache, to, dw, budget, sinks, recent, weights_out=dw)
    else:
        to_host = ko.Cache([min(n, budget) for n in lengths], heads, dim, 16 if page > 16 else 64, seed=28)
        to = device(qm, to_host)
        kept, wo = qm.qm_kv_evict_q4_0(cache, to, dw, budget, sinks, recent)
        assert np.array_equal(cache.k_pages.cpu().numpy(), c.k) and np.array_equal(dw.cpu().numpy(), w, equal_nan=True)
    torch.cuda.synchronize()
    assert qm.qm_device_status(clear=True) == qm.QM_OK
    assert to.lengths.tolist() == [min(n, budget) for n in lengths]
    kept, wo = kept.cpu().numpy(), wo.cpu().numpy()
    after = ko.Cache.__new__(ko.Cache)
    after.__dict__.update(to_host.__dict__)
    after.k, after.v = to.k_pages.cpu().numpy(), to.v_pages.cpu().numpy()
    for b, n in enumerate(lengths):
        for h in range(heads):
            want = ko.evict(w[b, h], n, budget, sinks, recent)
            m = len(want)
            assert np.array_equal(kept[b, h, :m], want)
            assert (kept[b, h, m:] == -1).all() and (wo[b, h, m:budget] == 0).all()
            assert np.array_equal(wo[b, h, :m], w[b, h][want], equal_nan=True)
            for pool, was in ((after.k, c.k), (after.v, c.v)):
                assert np.array_equal(after.values(pool, b, h, m), c.values(was, b, h)[want])


def test_evict_then_attend(qm):
    """A cut cache is a cache: attention over it is attention over the kept tokens."""
    c = ko.Cache([300, 150], 2, 128, 16, seed=29)
    cache = device(qm, c)
    w = torch.zeros((2, 2, cache.max_len), device="cuda")
    q = torch.randn((2, 8, 128), device="cuda")
    qm.qm_attn_q4_0(cache, q, weights=w)
    qm.qm_kv_evict_q4_0(cache, cache, w, 100, 4, 20, weights_out=w)
    c2 = ko.Cache([100, 100], 2, 128, 16, seed=29)
    c2.table, c2.n_pages = c.table, c.n_pages
    c2.k, c2.v = cache.k_pages.cpu().numpy(), cache.v_pages.cpu().numpy()
    check_attend(qm, c2, [1, 1], 8, cache=cache)


def test_empty_calls(qm):
    c = ko.Cache([10], 1, 64, 16, seed=30)
    cache = device(qm, c)
    e = torch.empty((0, 1, 64), device="cuda")
    qm.qm_kv_append_q4_0(cache, e, e)
    assert qm.qm_kv_read_q4_0(cache, 0)[0].shape == (0, 1, 64)
    assert qm.qm_attn_q4_0(cache, e).shape == (0, 1, 64)
    none = qm.KVCache(torch.empty((0, 1, 576), dtype=torch.uint8, device="cuda"),
                      torch.empty((0, 1, 576), dtype=torch.uint8, device="cuda"),
                      torch.empty((0, 1), dtype=torch.int32, device="cuda"),
                      torch.empty((0,), dtype=torch.int32, device="cuda"), head_dim=64, page_tokens=16)
    assert qm.qm_attn_q4_0(none, e).shape == (0, 1, 64)
