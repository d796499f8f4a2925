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
