"""GPU tests of a layer's norm, routing and experts at sizes past those of the other tests: rows for several rounds of
the kernels' grids, the longest rows, the most experts, and memory past 32 bits' reach."""
import math

import pytest

import layer_plain as lp
from test_gpu_layer import Block, check_route, generator, near, qm, rows  # noqa: F401 (a fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# ---- the norm

@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,width", [(5003, 8), (5003, 128), (5003, 264), (5003, 512), (2501, 1032), (2501, 2056), (2501, 4096),
                                     (1301, 8200), (611, 16384), (3001, 97), (2501, 4097), (701, 16383), (501, 16385)])
def test_norm_of_many_rows(qm, n, width, dtype, residual):  # noqa: F811
    """More rows than thread blocks are resident, no multiple of them; in place as well."""
    gen = generator(n + width)
    x = rows(n, width, dtype, gen)
    r = rows(n, width, dtype, gen) if residual else None
    w = torch.randn(width, generator=gen).cuda()
    want, s = lp.norm(x, w, r, 1e-5, 1.0)
    bounds = lp.norm_bounds(want, s, dtype, width // 256 + 50)
    out, total, _ = qm.qm_add_rmsnorm(x, w, residual=r, eps=1e-5, weight_offset=1.0)
    near(out, want, bounds[0])
    if not residual:
        return
    near(total, s, bounds[1])
    for into in (x.clone(), r.clone()):
        a, b = (into, r) if torch.equal(into, x) else (x, into)
        again, same, _ = qm.qm_add_rmsnorm(a, w, residual=b, eps=1e-5, weight_offset=1.0, sum_out=into)
        assert same is into and torch.equal(into, total) and torch.equal(again, out)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,width", [(5003, 128), (5003, 288), (2501, 4096), (701, 8224), (501, 16416)])
def test_norm_of_many_rows_to_8_bits(qm, n, width, dtype):  # noqa: F811
    gen = generator(n + width)
    x, r = rows(n, width, dtype, gen), rows(n, width, dtype, gen)
    w = torch.randn(width, generator=gen).cuda()
    out, _, q8 = qm.qm_add_rmsnorm(x, w, residual=r, want_q8=True)
    as_f32, _, _ = qm.qm_add_rmsnorm(x.float(), w, residual=r.float())
    assert torch.equal(q8.view(-1), qm.qm_quantize_q8_0(as_f32))
    assert torch.equal(out, as_f32.to(dtype))
    want, s = lp.norm(x, w, r, 1e-6, 0.0)
    near(out, want, lp.norm_bounds(want, s, dtype, width // 256 + 50)[0])


# ---- experts

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,hidden,inner,tokens,top_k", [
    (4, 7168, 256, 150, 2),    # rows' pieces in a launch of their own, longer than its registers hold
    (2, 20480, 64, 5, 2),      # rows and inner activations longer than 512 threads' registers hold
    (2, 64, 20480, 200, 2),
    (2, 65536, 32, 3, 2), (2, 32, 65536, 3, 2), (2, 65536, 32, 90, 1), (2, 32, 65536, 90, 1),  # the longest
    (8, 64, 96, 5000, 1), (5, 96, 64, 9001, 3),     # more tokens than a grid of the sums has
    (1024, 32, 64, 5000, 3),                        # the most experts, with tiles
    (3, 256, 128, 3, 1024), (3, 64, 64, 40, 300)])  # tokens of many experts, each many times
def test_experts_of_sizes(qm, n, hidden, inner, tokens, top_k, dtype):  # noqa: F811
    b = Block(qm, n, hidden, inner, seed=n + hidden + tokens)
    g = b.gen
    x = torch.randn((tokens, hidden), generator=g).to(dtype).cuda()
    ids = torch.randint(0, n, (tokens, top_k), generator=g, dtype=torch.int32).cuda()
    weights = torch.softmax(torch.randn((tokens, top_k), generator=g), -1).cuda()
    b.check(x, ids, weights)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [7, 40, 300])
def test_experts_of_padded_batches(qm, tokens, dtype):  # noqa: F811
    """What lies in rows without experts, and in weights without one, reaches nothing."""
    b = Block(qm, 4, 256, 288, seed=50)
    x, ids, weights = b.rows(tokens, 2, dtype)
    ids[1::3] = -1
    ids[2::3, 1] = -5
    clean = b.check(x, ids, weights)
    x2, w2 = x.clone(), weights.clone()
    x2[1::3] = torch.tensor([math.nan, math.inf, -math.inf, 3e38]).repeat(64).to(dtype).cuda()
    w2[ids < 0] = math.nan
    out = torch.full_like(x, math.nan)
    assert torch.equal(qm.qm_experts_q4_0(b.handle, x2, ids, w2, out=out), clean)
    assert (out[1::3] == 0).all()


# ---- memory past 32 bits' reach

def test_rows_far_apart(qm):  # noqa: F811
    """Rows 2^31 elements (and 2^32 bytes) apart, of the norm, of logits and of tokens."""
    far, out = (torch.as_strided(torch.zeros(2 ** 31 + 4096, dtype=BF16, device="cuda"), (2, 4096), (2 ** 31, 1)) for _ in range(2))
    gen = generator(51)
    x = torch.randn((2, 4096), generator=gen).to(BF16).cuda()
    far.copy_(x)
    qm.qm_add_rmsnorm(far, out=out)
    assert torch.equal(out, qm.qm_add_rmsnorm(x)[0])
    for a, b in zip(qm.qm_route_experts(far[:, :256], 8), qm.qm_route_experts(x[:, :256].contiguous(), 8)):
        assert torch.equal(a, b)
    blk = Block(qm, 3, 256, 96, seed=52)
    ids, weights = torch.tensor([[0, 2], [1, 2]], dtype=torch.int32, device="cuda"), torch.rand((2, 2), generator=gen).cuda()
    want = blk.check(x[:, :256].contiguous(), ids, weights)
    qm.qm_experts_q4_0(blk.handle, far[:, :256], ids, weights, out=out[:, :256])
    assert torch.equal(out[:, :256], want)


@pytest.mark.parametrize("tokens", [2, 30, 120])
def test_experts_far_apart(qm, tokens):  # noqa: F811
    """Experts' matrices more than 2^32 bytes apart."""
    blk = Block(qm, 2, 256, 96, seed=53)
    apart = 2 ** 32 + 4096
    buf = torch.zeros(apart + 3 * 65536, dtype=torch.uint8, device="cuda")
    far = []
    for i, w in enumerate((blk.gate, blk.up, blk.down)):
        t = torch.as_strided(buf, w.shape, (apart, w.shape[2], 1), 65536 * i)
        t.copy_(w)
        far.append(t)
    other = qm.Experts(*far)
    for dtype in (F32, BF16):
        x, ids, weights = blk.rows(tokens, 2, dtype)
        assert torch.equal(qm.qm_experts_q4_0(other, x, ids, weights), blk.check(x, ids, weights))
        x[0, 7] = math.inf  # (taken again element by element)
        a, b = qm.qm_experts_q4_0(other, x, ids, weights), qm.qm_experts_q4_0(blk.handle, x, ids, weights)
        assert torch.equal(a.nan_to_num(7.0, 8.0, 9.0), b.nan_to_num(7.0, 8.0, 9.0))
