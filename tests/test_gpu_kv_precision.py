"""GPU tests of how many bits the attention over the 4-bit cache keeps where scales,
scores and sums are not ordinary.  Bounds as in test_gpu_kv_cache (mass = sum p |v|,
reach = scale * sum |q k|); where a test has its own, it says how it comes about.
"""
import numpy as np
import pytest

import kv_oracle as ko

torch = pytest.importorskip("torch")
from test_gpu_kv_cache import BF16, F32, check_attend, device, qm, starts_of, to_dtype  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def scales_of(c, pool):
    """All scales of a pool, f16 [pages][heads][cells][16 tokens][blocks] (a view)."""
    return pool.reshape(c.n_pages, c.heads, -1, 9 * c.dim)[..., 8 * c.dim:].view(np.float16).reshape(
        c.n_pages, c.heads, -1, 16, c.dim // 32)


def quants_of(c, b, h, t):
    """The quant bytes of a token's blocks (a view) [blocks][16]."""
    return lambda pool: c.cell(pool, b, h, t)[:8 * c.dim].reshape(c.dim // 32, 16, 16)[:, t % 16]


# ---- bf16 rows: lse and weights are f32 and keep f32's bits

@pytest.mark.parametrize("case", [([333, 95], [90, 90], 128, 0, 0), ([1300], [300], 64, 0, 0), ([700], [400], 128, 250, 5),
                                  ([333, 95], [1, 1], 128, 0, 0)], ids=["chunk", "64 wide", "window", "step"])
def test_statistics_of_bf16_rows(qm, case):  # noqa: F811
    """Only the output is rounded (its probabilities and values to 11 bits): a row's
    logarithm and the tokens' weights are as exact as an f32 call's, ds = 2^-20 of the reach."""
    lengths, new, dim, window, sinks = case
    c = ko.Cache(lengths, 2, dim, 32, seed=31, scale=0.4)
    g = np.random.default_rng(32)
    starts = starts_of(new)
    q = to_dtype(g.standard_normal((int(starts[-1]), 8, dim)) * 2.0, BF16)
    cache = device(qm, c)
    w = torch.zeros((len(new), 2, cache.max_len), device="cuda")
    _, lse = qm.qm_attn_q4_0(cache, q, window=window, sinks=sinks, q_starts=torch.from_numpy(starts).cuda(),
                             max_q=max(new), weights=w, return_lse=True)
    _, l, added, _, reach = ko.attend(c, q.float().cpu().numpy(), starts, 8, np.float32(dim ** -0.5), window, sinks)
    ds = 2.0 ** -20 * reach + 2.0 ** -21 * np.abs(l) + 2.0 ** -20
    off = np.abs(lse.cpu().numpy() - l)
    assert (off <= ds + 2.0 ** -20).all(), (off / (ds + 2.0 ** -20)).max()
    got = w.cpu().numpy().astype(np.float64)[:, :, :added.shape[2]]
    tol = added * (4 * ds.max() + 2.0 ** -18) + 2.0 ** -22 * added + 1e-7
    assert (np.abs(got - added) <= tol).all(), (np.abs(got - added) / tol).max()
    # every row has given 1 for each query head
    rows = np.asarray(new) * 8.0
    assert np.allclose(got.sum((1, 2)), rows, rtol=4 * ds.max() + 2.0 ** -18)


# ---- value scales anywhere in binary16's range, and mixed ones

def step_and_prompt(new):
    return pytest.mark.parametrize("new", new, ids=["step", "draft", "prompt"][:len(new)])


@pytest.mark.parametrize("v_scale", [2.0 ** -16, 2.0 ** -20, 2.0 ** -22])
@step_and_prompt([1, 3, 90])
def test_small_value_scales(qm, new, v_scale):  # noqa: F811
    """Scales that are small or subnormal in binary16."""
    for seed in (33, 34):
        c = ko.Cache([310], 1, 128, 16, seed=seed)
        s = scales_of(c, c.v)
        s[:] = (s.astype(np.float32) * (v_scale / 0.1)).astype(np.float16)
        check_attend(qm, c, [new], 4, F32)


@pytest.mark.parametrize("far", [8, 14, 20, 26])
@pytest.mark.parametrize("v_scale", [2.0 ** -13, 2.0 ** -6, 4.0])
@step_and_prompt([1, 3, 90])
def test_a_dominant_token_whose_value_is_nothing(qm, new, v_scale, far):  # noqa: F811
    """Token 40 outweighs every other by 2^far or so and its values are 0: the output is
    made of the others alone, and they keep their bits."""
    n, dim = 300, 128
    c = ko.Cache([n], 1, dim, 16, seed=35)
    s = scales_of(c, c.v)
    s[:] = (s.astype(np.float32) * (v_scale / 0.1)).astype(np.float16)
    t = 40
    quants_of(c, 0, 0, t)(c.v)[:] = 0x88
    for j in range(n):  # keys: 0 but for the first element, 1 for token 40
        quants_of(c, 0, 0, j)(c.k)[:] = 0x88
        c.scales(c.k, 0, 0, j)[:] = 0.125
    quants_of(c, 0, 0, t)(c.k)[0, 0] = 0x80  # element 0: -8
    q = np.zeros((new, 4, dim))
    q[..., 0] = -far * np.log(2.0)  # score of token 40 (scale 1): far bits
    q[..., 0] *= 1 + 0.01 * np.arange(4)
    check_attend(qm, c, [new], 4, F32, scale=1.0, q=q)


@pytest.mark.parametrize("big,small", [(4e4, 2e-3), (6e4, 3e-5), (500.0, 1e-4), (1.0, 1e-6), (60.0, 0.02)])
@pytest.mark.parametrize("other_block", [True, False], ids=["other block", "same block"])
@step_and_prompt([1, 3, 90])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_mixed_value_scales(qm, dtype, new, other_block, big, small):  # noqa: F811
    """One token with a large value scale, in one block of its head or in all of them
    but with values of 0 there, among tokens with small ones."""
    c = ko.Cache([200], 1, 128, 16, seed=36)
    s = scales_of(c, c.v)
    s[:] = (np.sign(s.astype(np.float32)) * small * np.random.default_rng(37).uniform(0.5, 1.5, s.shape)).astype(np.float16)
    t = 77
    if other_block:
        c.scales(c.v, 0, 0, t)[0] = big
    else:
        c.scales(c.v, 0, 0, t)[:] = big
        quants_of(c, 0, 0, t)(c.v)[:] = 0x88
    check_attend(qm, c, [new], 4, dtype)


# ---- long sums

@pytest.mark.parametrize("case", [(64, 16384, 8, 1, 128), (16, 24000, 8, 2, 64), (1, 120000, 1, 4, 128)],
                         ids=["64x16384", "16x24000", "1x120000"])
def test_long_sums_of_one_sign(qm, case):  # noqa: F811
    """Queries of 0 make every probability the same, so the output is the mean of the
    values; all positive, so every rounding that leans one way would show.  Products
    and sums in f32: 2^-21 for the products and as much for the sums, whose
    roundings are random (the values are): 2^-20 of the mean."""
    seqs, n, heads, group, dim = case
    gen = torch.Generator(device="cuda").manual_seed(38)
    page, pages = 256, -(-n // 256)
    shape = (seqs * pages, heads, 16)
    quants = torch.randint(9, 16, (*shape, 8 * dim, 2), dtype=torch.uint8, device="cuda", generator=gen)
    d = (0.05 + 0.1 * torch.rand((*shape, dim // 2), device="cuda", generator=gen)).half()
    pool = torch.cat([quants[..., 0] | (quants[..., 1] << 4), d.view(torch.uint8)], -1).reshape(seqs * pages, heads, -1)
    del quants
    table = torch.randperm(seqs * pages, generator=gen, device="cuda").to(torch.int32).reshape(seqs, pages)
    lengths = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    cache = qm.KVCache(pool.clone(), pool, table, lengths, head_dim=dim, page_tokens=page)
    q = torch.zeros((seqs, heads * group, dim), device="cuda")
    out, lse = qm.qm_attn_q4_0(cache, q, return_lse=True)
    assert qm.qm_device_status(clear=True) == qm.QM_OK
    # (the values read one sequence at a time, in f64)
    for b in range(0, seqs, max(1, seqs // 4)):
        one = qm.KVCache(cache.k_pages, cache.v_pages, table[b:b + 1].contiguous(), lengths[b:b + 1].contiguous(),
                         head_dim=dim, page_tokens=page)
        _, v = qm.qm_kv_read_q4_0(one, n)
        want = v.double().mean(0).repeat_interleave(group, 0)
        off = ((out[b].double() - want).abs() / want).max().item()
        assert off <= 2.0 ** -20, off * 2 ** 20
        assert (lse[b].double() - np.log(n)).abs().max().item() <= 2.0 ** -20 * (1 + np.log(n))


# ---- a bad row's weights

@pytest.mark.parametrize("dim", [128, 64, 96])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(300, 1, 0, 0), (300, 6, 0, 0), (300, 200, 0, 0), (420, 300, 60, 3)],
                         ids=["step", "draft", "prompt", "window"])
def test_a_bad_rows_weights_stay_with_the_tokens_it_sees(qm, case, dtype, dim):  # noqa: F811
    """A row whose query is not finite makes the weights of the tokens that it sees
    NaN; those that it does not see keep what the other rows give them."""
    n, new, window, sinks = case
    c = ko.Cache([n], 1, dim, 16, seed=39)
    q = np.random.default_rng(40).standard_normal((new, 4, dim)).astype(np.float32)
    bad = new // 2
    good = q.copy()
    good[bad, 1] = 0
    spoiled = good.copy()
    spoiled[bad, 1, 7] = np.nan
    cache = device(qm, c)
    ws = []
    for x in (good, spoiled):
        w = torch.full((1, 1, cache.max_len), 0.25, device="cuda")
        qm.qm_attn_q4_0(cache, to_dtype(x, dtype), window=window, sinks=sinks, weights=w)
        ws.append(w[0, 0].cpu().numpy())
    sees = ko.visible([n - new + bad], n, window, sinks)[0]
    assert np.isnan(ws[1][:n][sees]).all()
    assert np.array_equal(ws[1][:n][~sees], ws[0][:n][~sees])
    assert (ws[1][n:] == 0.25).all()
    assert qm.qm_device_status(clear=True) == qm.QM_OK
