"""A layer's norm, routing and experts without a GPU: refusals on the host (before any CUDA
call), the binding's checks, workspace sizes, and pins of the plain implementations that the GPU
tests compare with."""
import ctypes
import math

import pytest

import bit_block_quantized_qm_gb300 as qm
import layer_plain as lp
from bit_block_quantized_qm_gb300 import build as qm_build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    qm_build.build()
    return qm.load_library()


X, R, W, O, S, Q = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000  # never dereferenced
WG, WU, WD, WS = 0x100000000, 0x200000000, 0x300000000, 0x400000000
FINE = (qm.QM_ERR_CUDA, qm.QM_ERR_POINTER)


def norm(lib, **kw):
    d = dict(x=X, residual=R, weight=W, out=O, sum=S, q8=Q, n_rows=3, width=64, x_stride=64, residual_stride=64,
             out_stride=64, sum_stride=64, eps=1e-6, weight_offset=0.0, dtype=0, reserved=0)
    d.update(kw)
    a = qm.QmRmsnormArgs(*[d[f] for f, _ in qm.QmRmsnormArgs._fields_])
    return lib.qm_add_rmsnorm(ctypes.addressof(a), None)


def route(lib, **kw):
    d = dict(logits=X, bias=R, ids=O, weights=S, n_tokens=5, logits_stride=64, n_experts=64, top_k=8, n_groups=4,
             top_groups=2, group_top=2, scoring=0, renormalize=1, scale=1.0, dtype=0, reserved=0)
    d.update(kw)
    a = qm.QmRouteArgs(*[d[f] for f, _ in qm.QmRouteArgs._fields_])
    return lib.qm_route_experts(ctypes.addressof(a), None)


MATRIX = 256 * 512 // 32 * 18


def weights(**kw):
    d = dict(w_gate=WG, w_up=WU, w_down=WD, gate_stride=MATRIX, up_stride=MATRIX, down_stride=MATRIX, hidden=512, inner=256,
             n_experts=4, activation=1, reserved=(ctypes.c_int32 * 2)())
    d.update(kw)
    return qm.QmExperts(*[d[f] for f, _ in qm.QmExperts._fields_])


def experts(lib, e=None, **kw):
    d = dict(x=X, out=O, ids=R, weights=S, workspace=WS, workspace_bytes=1 << 40, n_tokens=6, x_stride=512, out_stride=512,
             top_k=2, dtype=0, reserved=(ctypes.c_int32 * 2)())
    d.update(kw)
    a = qm.QmExpertsArgs(*[d[f] for f, _ in qm.QmExpertsArgs._fields_])
    e = weights() if e is None else e
    return lib.qm_experts_q4_0(ctypes.addressof(e), ctypes.addressof(a), None)


def test_calls_that_pass_the_checks(lib):
    assert norm(lib) in FINE and route(lib) in FINE and experts(lib) in FINE
    assert norm(lib, residual=None, weight=None, q8=None) in FINE
    assert norm(lib, sum=X) in FINE and norm(lib, sum=R) in FINE
    assert norm(lib, n_rows=1, x_stride=0, out_stride=0, sum_stride=-5, residual_stride=1) in FINE
    assert experts(lib, weights(w_gate=None, gate_stride=-1)) in FINE
    assert experts(lib, weights(n_experts=1, up_stride=0, gate_stride=7, down_stride=0)) in FINE
    assert experts(lib, n_tokens=1, x_stride=3, out_stride=1) in FINE


def test_null_structs(lib):
    assert lib.qm_add_rmsnorm(None, None) == qm.QM_ERR_NULL
    assert lib.qm_route_experts(None, None) == qm.QM_ERR_NULL
    assert lib.qm_experts_q4_0(None, None, None) == qm.QM_ERR_NULL
    assert lib.qm_experts_q4_0(ctypes.addressof(weights()), None, None) == qm.QM_ERR_NULL
    assert lib.qm_experts_workspace(None, 1, 1) == qm.QM_ERR_NULL


@pytest.mark.parametrize("bad", [dict(n_rows=-1), dict(n_rows=1 << 31), dict(width=0), dict(width=-8), dict(width=(1 << 20) + 1),
                                 dict(x_stride=63), dict(residual_stride=0), dict(out_stride=-64), dict(sum_stride=60),
                                 dict(width=63, q8=Q), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf),
                                 dict(weight_offset=math.nan), dict(dtype=2), dict(dtype=-1), dict(reserved=1),
                                 dict(x_stride=1 << 62)], ids=str)
def test_norm_shapes_refused(lib, bad):
    assert norm(lib, **bad) == qm.QM_ERR_SHAPE


def test_norm_refusals(lib):
    assert norm(lib, x=None) == qm.QM_ERR_NULL
    assert norm(lib, n_rows=0, x=None, out=None) == qm.QM_OK
    assert norm(lib, out=None, sum=None, q8=None) == qm.QM_OK
    for bad in (dict(x=X + 2), dict(residual=R + 1), dict(out=O + 2), dict(sum=S + 3), dict(weight=W + 2), dict(q8=Q + 1),
                dict(dtype=1, x=X + 1)):
        assert norm(lib, **bad) == qm.QM_ERR_ALIGN
    assert norm(lib, dtype=1, x=X + 2, out=O + 2) in FINE
    for bad in (dict(out=X), dict(out=X + 64), dict(out=R), dict(out=W), dict(out=S), dict(q8=X + 700), dict(q8=O), dict(q8=S),
                dict(q8=W + 200), dict(sum=X + 256), dict(sum=R - 4), dict(sum=W), dict(sum=X, sum_stride=128),
                dict(sum=R, residual_stride=72), dict(sum=O + 4)):
        assert norm(lib, **bad) == qm.QM_ERR_ALIAS, bad


@pytest.mark.parametrize("bad", [dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(n_experts=0), dict(n_experts=1025),
                                 dict(logits_stride=63), dict(n_groups=0), dict(n_groups=65), dict(n_groups=3),
                                 dict(top_groups=0), dict(top_groups=5), dict(group_top=0), dict(group_top=3), dict(top_k=0),
                                 dict(top_k=33), dict(top_k=17, top_groups=1), dict(scoring=2), dict(scoring=-1),
                                 dict(renormalize=2), dict(scale=math.inf), dict(dtype=2), dict(reserved=1)], ids=str)
def test_route_shapes_refused(lib, bad):
    assert route(lib, **bad) == qm.QM_ERR_SHAPE


def test_route_refusals(lib):
    assert route(lib, n_tokens=0, logits=None) == qm.QM_OK
    for p in ("logits", "ids", "weights"):
        assert route(lib, **{p: None}) == qm.QM_ERR_NULL
    assert route(lib, bias=None) in FINE
    for bad in (dict(logits=X + 2), dict(bias=R + 2), dict(ids=O + 1), dict(weights=S + 2)):
        assert route(lib, **bad) == qm.QM_ERR_ALIGN
    for bad in (dict(ids=X), dict(ids=X + 5 * 256 - 4), dict(ids=R + 252), dict(weights=O + 156), dict(weights=X), dict(weights=R)):
        assert route(lib, **bad) == qm.QM_ERR_ALIAS


@pytest.mark.parametrize("bad", [dict(hidden=0), dict(hidden=48), dict(hidden=65568), dict(inner=16), dict(inner=100),
                                 dict(inner=-256), dict(n_experts=0), dict(n_experts=1025), dict(activation=3),
                                 dict(activation=-1), dict(up_stride=MATRIX - 16), dict(down_stride=MATRIX + 8),
                                 dict(gate_stride=0), dict(up_stride=1 << 62), dict(down_stride=1 << 40), dict(reserved=(ctypes.c_int32 * 2)(0, 1))],
                         ids=str)
def test_expert_shapes_refused(lib, bad):
    e = weights(**bad)
    assert experts(lib, e) == qm.QM_ERR_SHAPE
    assert lib.qm_experts_workspace(ctypes.addressof(e), 4, 2) == qm.QM_ERR_SHAPE


@pytest.mark.parametrize("bad", [dict(n_tokens=-1), dict(n_tokens=1 << 24), dict(n_tokens=1 << 23), dict(top_k=0),
                                 dict(top_k=1025), dict(x_stride=508), dict(out_stride=510), dict(x_stride=513), dict(dtype=2),
                                 dict(out_stride=1 << 61), dict(reserved=(ctypes.c_int32 * 2)(1, 0))], ids=str)
def test_expert_calls_refused(lib, bad):
    assert experts(lib, **bad) == qm.QM_ERR_SHAPE


def test_expert_refusals(lib):
    assert experts(lib, n_tokens=0, x=None) == qm.QM_OK
    for p in ("x", "out", "ids", "weights", "workspace"):
        assert experts(lib, **{p: None}) == qm.QM_ERR_NULL
    for p in ("w_up", "w_down"):
        assert experts(lib, weights(**{p: None})) == qm.QM_ERR_NULL
        assert experts(lib, weights(**{p: WD + 8})) == qm.QM_ERR_ALIGN
    for bad in (dict(x=X + 8), dict(out=O + 4), dict(ids=R + 2), dict(weights=S + 1), dict(workspace=WS + 8), dict(dtype=1, x=X + 4)):
        assert experts(lib, **bad) == qm.QM_ERR_ALIGN
    assert experts(lib, dtype=1, x=X + 8, out=O + 8) in FINE
    e = weights()
    need = lib.qm_experts_workspace(ctypes.addressof(e), 6, 2)
    assert need > 0
    assert experts(lib, workspace_bytes=need) in FINE and experts(lib, workspace_bytes=need - 1) == qm.QM_ERR_WORKSPACE
    row = 6 * 512 * 4
    for bad in (dict(out=X), dict(out=X + row - 16), dict(out=R), dict(out=S - row + 16), dict(out=WG), dict(out=WU + 4 * MATRIX - 16),
                dict(out=WD), dict(out=WS), dict(workspace=X - 16), dict(workspace=WG + 256), dict(workspace=WD - need // 256 * 256 + 256),
                dict(workspace=S), dict(workspace=R)):
        assert experts(lib, **bad) == qm.QM_ERR_ALIAS, bad


def test_workspace_serves_every_smaller_call(lib):
    for e in (weights(), weights(hidden=544, inner=96, w_gate=None, up_stride=1 << 20, down_stride=1 << 20)):
        size = {(t, k): lib.qm_experts_workspace(ctypes.addressof(e), t, k) for t in (1, 2, 7, 64, 65, 500, 5000) for k in (1, 2, 8, 33)}
        for (t, k), n in size.items():
            for (t2, k2), n2 in size.items():
                assert t2 > t or k2 > k or n2 <= n
    assert lib.qm_experts_workspace(ctypes.addressof(weights()), 0, 2) == 0


def test_binding_checks():
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        qm.qm_add_rmsnorm(x)  # not a CUDA tensor
    with pytest.raises(TypeError):
        qm.qm_add_rmsnorm(x.double())
    with pytest.raises(TypeError):
        qm.qm_route_experts([1.0], 1)
    with pytest.raises(ValueError):
        qm.qm_route_experts(x, 1)
    w = torch.zeros((2, 32, 36), dtype=torch.uint8)
    with pytest.raises(ValueError):
        qm.Experts(w, w, torch.zeros((2, 64, 18), dtype=torch.uint8))  # not CUDA tensors
    with pytest.raises(TypeError):
        qm.Experts(w.float(), w, w)


# ---- pins of the plain implementations

def test_plain_route_by_hand():
    logits = torch.tensor([[0.0, math.log(3), math.log(2), math.log(2)]])
    ids, w = lp.route(logits, 2, None, False, 1, 1, 2, False, 1.0)
    assert ids.tolist() == [[1, 2]] and torch.allclose(w, torch.tensor([[3 / 8, 2 / 8]], dtype=torch.float64))
    _, w = lp.route(logits, 2, None, False, 1, 1, 2, True, 2.0)
    assert torch.allclose(w, torch.tensor([[1.2, 0.8]], dtype=torch.float64))
    ids, w = lp.route(logits, 2, torch.tensor([0.6, 0.0, 0.0, 0.2]), False, 1, 1, 2, False, 1.0)
    assert ids.tolist() == [[0, 3]] and torch.allclose(w, torch.tensor([[1 / 8, 2 / 8]], dtype=torch.float64))
    # two groups {0, 1} and {2, 3}: sums 4 / 8 and 4 / 8 are equal, the first stays; by their largest, 3 / 8 and 2 / 8.
    ids, _ = lp.route(logits, 2, None, False, 2, 1, 2, True, 1.0)
    assert ids.tolist() == [[1, 0]]
    ids, _ = lp.route(logits[:, [2, 3, 0, 1]], 1, None, True, 2, 1, 1, True, 1.0)
    assert ids.tolist() == [[3]]


def test_plain_norm_by_hand():
    y, s = lp.norm(torch.tensor([[3.0, -4.0]]), torch.tensor([0.0, 1.0]), torch.tensor([[0.0, 8.0]]), 0.0, 1.0)
    r = 5 / math.sqrt(2)
    assert torch.allclose(y, torch.tensor([[3 / r, 8 / r]], dtype=torch.float64)) and s.tolist() == [[3.0, 4.0]]


def test_plain_experts_by_hand():
    """One expert whose matrices are 32 times one block row; ones in, so products are sums of quants."""
    row = torch.zeros(18, dtype=torch.uint8)
    row[:2] = torch.tensor([0.5]).half().view(torch.uint8)
    row[2:] = 0x88
    row[2] = 0x9F  # elements 0 and 16: (15 - 8) / 2 and (9 - 8) / 2
    w = row.repeat(1, 32, 1)
    assert lp.q4_values(w)[0, 3].nonzero().flatten().tolist() == [0, 16]
    out, bound = lp.experts(w, w, w, torch.ones((1, 32)), torch.zeros((1, 1), dtype=torch.int32), torch.tensor([[2.0]]), 0)
    assert torch.allclose(out, torch.full((1, 32), 2.0 * 16 * 4, dtype=torch.float64)) and (bound > 0).all()
    out, _ = lp.experts(None, w, w, -torch.ones((1, 32)), torch.zeros((1, 1), dtype=torch.int32), torch.tensor([[1.0]]), 1)
    assert torch.allclose(out, torch.full((1, 32), -4 / (1 + math.exp(4)) * 4, dtype=torch.float64))
    out, _ = lp.experts(None, w, w, torch.ones((1, 32)), torch.full((1, 1), -1, dtype=torch.int32), torch.tensor([[1.0]]), 1)
    assert (out == 0).all()
