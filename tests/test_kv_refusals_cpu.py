"""More refusals of the 4-bit key/value cache's entry points, on the host alone."""
import ctypes

import pytest

import bit_block_quantized_qm_gb300 as qm
from test_kv_cache_cpu import FINE, K, L, O, Q, S, T, V, append, args, attn, cache, evict, lib  # noqa: F401


@pytest.mark.parametrize("n", [1 << 30, 1 << 29])
def test_rows_and_heads_are_numbered_in_an_int(lib, n):  # noqa: F811
    """2^31 and more rows times heads have no number in the kernels and their list of rows."""
    big = dict(n_tokens=n, max_q=n, n_heads=4, weights=None, lse=None, workspace_bytes=1 << 60)
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


# ---- what is written shares no bytes with what else is read or written

@pytest.mark.parametrize("kw,bad", [
    (dict(page_table=K + 64), {}), (dict(page_table=V + 11516), {}), (dict(lengths=K), {}), (dict(lengths=V - 4), {}),
    ({}, dict(starts=K + 128)), ({}, dict(starts=V - 8))], ids=str)
def test_append_writes_pools_alone(lib, kw, bad):  # noqa: F811
    assert append(lib, cache(**kw), **bad) == qm.QM_ERR_ALIAS


@pytest.mark.parametrize("bad", [dict(k=T), dict(v=T - 16), dict(k=L), dict(v=L - 3056), dict(starts=Q + 8),
                                 dict(starts=O + 3068), dict(k=T - 3056)], ids=str)
def test_read_writes_rows_alone(lib, bad):  # noqa: F811
    d = dict(k=Q, v=O, starts=S)
    d.update(bad)
    c = cache()
    assert lib.qm_kv_read_q4_0(ctypes.addressof(c), d["k"], d["v"], 6, d["starts"], None) == qm.QM_ERR_ALIAS


FAR = dict(k_pages=K + (1 << 24), v_pages=V + (1 << 24), page_table=T + 4096, lengths=L + 4096)


@pytest.mark.parametrize("bad", [
    dict(kept=K + 16), dict(kept=V - 4), dict(kept=K + (1 << 24)), dict(kept=V + (1 << 24) + 11516), dict(kept=T),
    dict(kept=T + 4096), dict(kept=L - 600), dict(kept=L + 4096), dict(wo=K), dict(wo=V + 64), dict(wo=K + (1 << 24)),
    dict(wo=T + 36), dict(wo=T + 4100), dict(wo=L + 4), dict(wo=L + 4100), dict(w=K + (1 << 24)), dict(w=L + 4096 - 1276),
    dict(w=V + (1 << 24)), dict(to=cache(**{**FAR, "lengths": L + 4})), dict(to=cache(**{**FAR, "lengths": L - 4})),
    dict(to=cache(**{**FAR, "lengths": T + 8})), dict(to=cache(**{**FAR, "lengths": K + 256})),
    dict(to=cache(**{**FAR, "page_table": K + (1 << 24) + 512})), dict(to=cache(**{**FAR, "k_pages": T - 64})),
    dict(to=cache(**{**FAR, "v_pages": L - 64}))], ids=lambda x: str(x)[:60])
def test_evict_writes_what_it_says_alone(lib, bad):  # noqa: F811
    assert evict(lib, **bad) == qm.QM_ERR_ALIAS


def test_evict_with_shared_lengths_and_shared_pools_passes(lib):  # noqa: F811
    assert evict(lib, to=cache(**{**FAR, "lengths": L})) in FINE
    assert evict(lib, to=cache(page_table=T + 4096, lengths=L + 4096)) in FINE  # the same pools, other pages
    assert evict(lib, to=cache(lengths=L + 4096)) in FINE  # in place, lengths apart
    assert evict(lib, to=cache(lengths=L + 8)) in FINE  # lengths side by side


def test_evicting_caches_that_can_hold_nothing_passes(lib):  # noqa: F811
    """With max_len 0 there are no weights to read, and an empty tensor has no address."""
    c = dict(max_len=0, k_pages=None, v_pages=None, page_table=None, n_pages=0, table_stride=0)
    assert evict(lib, cache(**c), to=cache(**{**c, "lengths": L + 4096}), w=None, ws=0, budget=12) in FINE
    assert evict(lib, cache(**c), to=cache(**{**c, "page_tokens": 64}), w=None, ws=0, budget=12) in FINE
    assert evict(lib, cache(**c), to=cache(**c), w=None, ws=8, budget=0, sinks=0, recent=0, kept=None, wo=None, os_=0) in FINE
    assert evict(lib, cache(**c), to=cache(**c), w=None, ws=0, budget=0, sinks=0, recent=0, kept=None, wo=None, os_=0) in FINE
    assert evict(lib, cache(**c), to=cache(**{**c, "lengths": L + 4096}), w=None, ws=0, budget=12, wo=None) == qm.QM_ERR_NULL


@pytest.mark.parametrize("bad", [dict(sinks=1 << 62, recent=1 << 62), dict(sinks=(1 << 63) - 1, recent=1),
                                 dict(sinks=1, recent=(1 << 63) - 1), dict(sinks=1 << 32), dict(recent=1 << 32)], ids=str)
def test_first_and_recent_tokens_that_do_not_add_up(lib, bad):  # noqa: F811
    """Their sum may pass 2^63."""
    assert evict(lib, **bad) == qm.QM_ERR_SHAPE
