"""GPU tests of a layer's norm, routing and experts against plain implementations in
f64, at the sizes and inputs where they can go wrong."""
import math

import pytest

import layer_plain as lp

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_block_quantized_qm_gb300 import build as qm_build
    qm_build.build()
    import bit_block_quantized_qm_gb300 as m
    torch.cuda.set_device(0)
    assert m.qm_device_status(clear=True) == m.QM_OK
    yield m
    assert m.qm_device_status(clear=True) == m.QM_OK


def near(got, want, bound):
    off = (got.double().cpu() - want.double().cpu()).abs()
    bad = ~(off <= bound.cpu())
    assert not bad.any(), (int(bad.sum()), bad.numel(), float((off / bound.cpu()).nan_to_num(math.inf).max()))


def generator(seed):
    return torch.Generator().manual_seed(seed)


# ---- the norm

def rows(n, width, dtype, gen, pad=0, shift=0):
    """[n, width] on the GPU with rows `pad` elements longer apart, `shift` elements into their memory."""
    x = torch.randn((n, width), generator=gen) * torch.exp(torch.randn((n, 1), generator=gen))
    buf = torch.zeros(n * (width + pad) + shift + 8, dtype=dtype, device="cuda")
    view = buf[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    view.copy_(x)
    return view


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,width,pad,shift", [
    (1, 4096, 0, 0), (3, 8, 0, 0), (5, 7, 0, 0), (2, 1, 0, 0), (4, 264, 24, 0), (3, 4096, 0, 1), (2, 4104, 8, 0),
    (7, 8200, 0, 0), (2, 16384, 0, 0), (2, 16392, 0, 0), (3, 20001, 3, 0), (65, 512, 0, 0), (2, 4095, 0, 0)])
@pytest.mark.parametrize("residual,weight,offset", [(True, True, 0.0), (False, True, 1.0), (True, False, 0.0)])
def test_norm(qm, n, width, pad, shift, dtype, residual, weight, offset):
    gen = generator(n * 31 + width)
    x = rows(n, width, dtype, gen, pad, shift)
    r = rows(n, width, dtype, gen, pad, shift) if residual else None
    w = torch.randn(width, generator=gen).cuda() if weight else None
    out, total, q8 = qm.qm_add_rmsnorm(x, w, residual=r, eps=1e-5, weight_offset=offset)
    want, s = lp.norm(x, w, r, 1e-5, offset)
    b_out, b_sum = lp.norm_bounds(want, s, dtype, width // 512 + 50)
    near(out, want, b_out)
    assert q8 is None and (total is not None) == residual
    if residual:
        near(total, s, b_sum)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("width", [33, 255, 257, 1023, 4097, 8191, 8193, 16383, 16385])
def test_norm_of_odd_widths(qm, width, dtype):
    gen = generator(width)
    x, r = rows(5, width, dtype, gen), rows(5, width, dtype, gen)
    w = torch.randn(width, generator=gen).cuda()
    want, s = lp.norm(x, w, r, 1e-5, 1.0)
    bounds = lp.norm_bounds(want, s, dtype, width // 512 + 50)
    out, total, _ = qm.qm_add_rmsnorm(x, w, residual=r, eps=1e-5, weight_offset=1.0)
    near(out, want, bounds[0])
    near(total, s, bounds[1])
    again, same, _ = qm.qm_add_rmsnorm(x, w, residual=r, eps=1e-5, weight_offset=1.0, sum_out=r)
    assert same is r and torch.equal(r, total) and torch.equal(again, out)


@pytest.mark.parametrize("width", [32, 96, 4096, 8224, 16416])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_norm_to_8_bits(qm, width, dtype):
    """Of f32 rows the blocks are what qm_quantize_q8_0 makes of the f32 output; of bf16 rows those of the
    same numbers held as f32."""
    gen = generator(width)
    x, r = rows(9, width, dtype, gen), rows(9, width, dtype, gen)
    x[4] = 0
    r[4] = 0  # blocks of zeros
    w = torch.randn(width, generator=gen).cuda()
    out, total, q8 = qm.qm_add_rmsnorm(x, w, residual=r, want_q8=True)
    as_f32, _, _ = qm.qm_add_rmsnorm(x.float(), w, residual=r.float())
    assert torch.equal(q8.view(-1), qm.qm_quantize_q8_0(as_f32))
    assert torch.equal(out, as_f32.to(dtype))
    none, _, alone = qm.qm_add_rmsnorm(x, w, residual=r, want_q8=True, want_out=False)
    assert none is None and torch.equal(alone, q8)


@pytest.mark.parametrize("shift", [0, 1])
def test_norm_in_place(qm, shift):
    """The sum in the residual's place, or in x's: the residual stream of a decoder."""
    gen = generator(5)
    for dtype in (F32, BF16):
        x, r = rows(6, 520, dtype, gen, shift=shift), rows(6, 520, dtype, gen, shift=shift)
        out, total, _ = qm.qm_add_rmsnorm(x, None, residual=r)
        for into in (x.clone(), r.clone()):
            a, b = (into, r) if torch.equal(into, x) else (x, into)
            out2, total2, _ = qm.qm_add_rmsnorm(a, None, residual=b, sum_out=into)
            assert total2 is into and torch.equal(total2, total) and torch.equal(out2, out)


def test_norm_leaves_the_rest_alone(qm):
    buf = torch.full((4, 80), 7.0, device="cuda")
    qm.qm_add_rmsnorm(torch.ones((4, 64), device="cuda"), out=buf[:, 8:72])
    assert (buf[:, :8] == 7).all() and (buf[:, 72:] == 7).all()
    near(buf[:, 8:72], torch.ones(4, 64), torch.full((4, 64), 1e-5))


def test_norm_of_infinities(qm):
    x = torch.ones((3, 64), device="cuda")
    x[0, 3] = math.inf
    x[1, 5] = math.nan
    out, _, q8 = qm.qm_add_rmsnorm(x, want_q8=True)
    assert out[0, 3].isnan() and (out[0, :3] == 0).all() and out[1].isnan().all() and (out[2] - 1).abs().max() < 1e-5
    assert torch.equal(q8.view(-1), qm.qm_quantize_q8_0(out))


# ---- routing

def check_route(qm, logits, top_k, **kw):
    d = dict(bias=None, sigmoid=False, groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0)
    d.update(kw)
    ids, weights = qm.qm_route_experts(logits, top_k, bias=d["bias"],
                                       scoring=qm.QM_SCORE_SIGMOID if d["sigmoid"] else qm.QM_SCORE_SOFTMAX,
                                       n_groups=d["groups"], top_groups=d["top_groups"], group_top=d["group_top"],
                                       renormalize=d["renormalize"], scale=d["scale"])
    want_ids, want = lp.route(logits, top_k, d["bias"], d["sigmoid"], d["groups"], d["top_groups"], d["group_top"],
                              d["renormalize"], d["scale"])
    assert torch.equal(ids.cpu(), want_ids), (ids.cpu() != want_ids).nonzero()[:5]
    # A score exp(d) / sum: d = l - max is rounded once (2^-24 |d| of the score), exp by 2 units, the sum by 37 of
    # terms below it, reciprocal, product, the division by the chosen scores' sum and the scale: |d| + 64 units.
    x = logits.double().cpu()
    dist = (x - x.amax(-1, keepdim=True)).abs().nan_to_num(0.0, 0.0).gather(1, want_ids.long()).amax(-1, keepdim=True)
    near(weights, want, (dist + 64) * 2.0 ** -24 * want.abs() * 2 + 1e-37)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 2), (8, 2), (31, 5), (33, 32), (60, 4), (64, 8), (128, 8), (160, 6),
                                           (256, 8), (300, 10), (512, 9), (1000, 32), (1024, 1)])
@pytest.mark.parametrize("sigmoid,bias", [(False, False), (True, False), (False, True), (True, True)])
def test_route(qm, experts, top_k, dtype, sigmoid, bias):
    gen = generator(experts + 7 * top_k)
    logits = (2 * torch.randn((37, experts), generator=gen)).to(dtype).cuda()
    b = (0.1 * torch.randn(experts, generator=gen)).cuda() if bias else None
    check_route(qm, logits, top_k, sigmoid=sigmoid, bias=b, renormalize=top_k % 2 == 0, scale=1.0 if bias else 2.5)


@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(256, 8, 4, 8), (64, 2, 1, 6), (64, 64, 5, 5), (96, 4, 3, 7),
                                                             (40, 8, 8, 10), (1024, 64, 33, 32), (33, 11, 2, 6), (6, 2, 1, 3)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("bias", [False, True])
def test_route_in_groups(qm, experts, groups, top_groups, top_k, group_top, bias):
    gen = generator(experts + groups)
    logits = (2 * torch.randn((29, experts), generator=gen)).cuda()
    b = (0.1 * torch.randn(experts, generator=gen)).cuda() if bias else None
    for sigmoid in (False, True):
        check_route(qm, logits, top_k, sigmoid=sigmoid, bias=b, groups=groups, top_groups=top_groups, group_top=group_top)


def test_route_many_rows(qm):
    """Enough rows that some choices lie next to each other: their order is that of the formula."""
    gen = generator(1)
    logits = (1.5 * torch.randn((3000, 256), generator=gen)).cuda()
    bias = (0.1 * torch.randn(256, generator=gen)).cuda()
    check_route(qm, logits, 8, sigmoid=True, bias=bias, groups=8, top_groups=4)


def test_route_close_choices(qm):
    """Choices that f32 cannot tell apart, and equal ones."""
    gen = generator(2)
    base = torch.randn((64, 32), generator=gen)
    base = torch.cat([base, base + torch.randint(-3, 4, base.shape, generator=gen) * 2.0 ** -23], 1)
    bias = (0.01 * torch.randn(32, generator=gen)).repeat(2).cuda()
    for sigmoid in (False, True):
        check_route(qm, base.cuda(), 10, sigmoid=sigmoid, bias=bias)
        check_route(qm, base.cuda(), 10, sigmoid=sigmoid, bias=bias, groups=4, top_groups=2)
        check_route(qm, base.cuda(), 10, sigmoid=sigmoid, groups=2, top_groups=1)
    same = torch.zeros((5, 40), device="cuda")
    check_route(qm, same, 9)
    check_route(qm, same, 9, bias=torch.zeros(40, device="cuda"), groups=4, top_groups=2)
    check_route(qm, torch.randint(-1, 2, (200, 64), generator=gen).float().cuda(), 20, sigmoid=True)


@pytest.mark.parametrize("low", [-math.inf, torch.finfo(F32).min])
def test_route_masked(qm, low):
    """Experts masked by their logit or by their bias, until none are left."""
    gen = generator(3)
    logits = torch.randn((20, 48), generator=gen)
    for i in range(20):
        logits[i, torch.randperm(48, generator=gen)[:min(48, 3 * i)]] = low
    check_route(qm, logits.cuda(), 6)
    check_route(qm, logits.cuda(), 6, groups=4, top_groups=2)
    check_route(qm, logits.cuda(), 6, sigmoid=True, renormalize=False)
    bias = torch.zeros(48)
    bias[::2] = low
    check_route(qm, torch.randn((20, 48), generator=gen).cuda(), 6, bias=bias.cuda())
    check_route(qm, torch.randn((20, 48), generator=gen).cuda(), 30, bias=bias.cuda(), sigmoid=True)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_of_nothing_by_close_biases(qm, sigmoid):
    """Rows whose mask leaves nothing: the biases choose, next to each other as they are."""
    gen = generator(4)
    bias = 1 + torch.randperm(40, generator=gen).float() * 2.0 ** -23
    logits = torch.full((5, 40), -math.inf)
    logits[0] = 0
    logits[1, 7] = 3
    ids, weights = qm.qm_route_experts(logits.cuda(), 6, bias=bias.cuda(),
                                       scoring=qm.QM_SCORE_SIGMOID if sigmoid else qm.QM_SCORE_SOFTMAX)
    order = torch.argsort(bias, descending=True)
    assert torch.equal(ids[2:].long().cpu(), order[:6].expand(3, 6)) and (weights[2:] == 0).all()
    assert torch.equal(ids[0].long().cpu(), order[:6])
    assert ids[1, 0] == 7 and torch.equal(ids[1, 1:].long().cpu(), order[order != 7][:5])


def test_route_bad_rows(qm):
    """NaN and infinities: the ids are experts, each once; other rows are as ever."""
    gen = generator(4)
    logits = torch.randn((6, 64), generator=gen).cuda()
    want = qm.qm_route_experts(logits, 8, bias=torch.zeros(64, device="cuda"))
    bad = logits.clone()
    bad[0, 3], bad[1, 60], bad[2] = math.nan, math.inf, math.nan
    for kw in ({}, dict(bias=torch.zeros(64, device="cuda")), dict(n_groups=4, top_groups=1), dict(scoring=qm.QM_SCORE_SIGMOID)):
        ids, weights = qm.qm_route_experts(bad, 8, **kw)
        assert ((ids >= 0) & (ids < 64)).all()
        assert all(len(set(r)) == 8 for r in ids.tolist())
        if kw.get("scoring") is None:
            assert weights[:3].isnan().all()
    ids, weights = qm.qm_route_experts(bad, 8, bias=torch.zeros(64, device="cuda"))
    assert torch.equal(ids[3:], want[0][3:]) and torch.equal(weights[3:], want[1][3:])


def test_route_strided_rows(qm):
    gen = generator(6)
    wide = torch.randn((11, 100), generator=gen).cuda()
    check_route(qm, wide[:, 3:67], 8)


# ---- experts

class Block:
    """Random experts of a size, on the GPU."""

    def __init__(self, qm, n, hidden, inner, gated=True, kind=1, seed=0, size=0.2, fused=False):
        gen = generator(seed)
        w = [lp.q4_random((n, r), k, gen, size).cuda() for r, k in ((inner, hidden), (inner, hidden), (hidden, inner))]
        if fused:  # gate and up as halves of one tensor
            both = torch.cat(w[:2], 1)
            w[:2] = both[:, :inner], both[:, inner:]
        self.gate, self.up, self.down = w if gated else (None, *w[1:])
        self.hidden, self.n, self.kind, self.qm, self.gen = hidden, n, kind, qm, gen
        self.handle = qm.Experts(self.gate, self.up, self.down, activation=kind)

    def rows(self, tokens, top_k, dtype, skew=0.0, idle=0.0):
        g = self.gen
        x = torch.randn((tokens, self.hidden), generator=g).to(dtype).cuda()
        top = torch.topk(torch.randn((tokens, self.n), generator=g) + skew * torch.randn(self.n, generator=g), top_k, -1)
        ids = top.indices.to(torch.int32)
        ids[torch.rand(ids.shape, generator=g) < idle] = -1
        return x, ids.cuda(), torch.softmax(top.values, -1).cuda()

    def check(self, x, ids, weights, out=None):
        out = self.qm.qm_experts_q4_0(self.handle, x, ids, weights, out=out)
        want, bound = lp.experts(self.gate, self.up, self.down, x, ids, weights, self.kind)
        near(out, want, bound)
        return out


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,hidden,inner,tokens,top_k", [
    (1, 32, 32, 1, 1), (3, 64, 96, 5, 2), (8, 256, 256, 1, 2), (8, 512, 1024, 7, 3), (4, 256, 288, 200, 2), (5, 544, 352, 33, 5),
    (16, 768, 512, 64, 4), (2, 256, 1408, 300, 1), (64, 512, 128, 3, 8), (3, 1024, 256, 500, 2), (130, 256, 256, 40, 6)])
def test_experts(qm, n, hidden, inner, tokens, top_k, dtype):
    b = Block(qm, n, hidden, inner, seed=n + hidden)
    x, ids, weights = b.rows(tokens, top_k, dtype, skew=1.0)
    b.check(x, ids, weights)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,hidden,inner,tokens,top_k", [
    (40, 288, 320, 40, 4), (16, 64, 640, 16, 8), (9, 2048, 32, 12, 6), (1024, 96, 64, 70, 3), (24, 1280, 800, 6, 24),
    (12, 352, 544, 24, 4), (4, 4096, 1408, 1, 4), (2, 4096, 4096, 3, 2),  # up to 8 rows an expert
    (4, 352, 288, 25, 2), (3, 1024, 544, 40, 1), (20, 64, 512, 60, 5)])  # 8 to 16
def test_experts_with_few_rows(qm, n, hidden, inner, tokens, top_k, dtype):
    """Few rows an expert on average, some with many and some with none; lengths that are odd multiples of a block."""
    b = Block(qm, n, hidden, inner, seed=n + inner)
    b.check(*b.rows(tokens, top_k, dtype, skew=2.0))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,hidden,inner,tokens,top_k", [
    (2, 4096, 512, 24, 1), (2, 4384, 512, 150, 1), (2, 512, 4096, 150, 2), (3, 288, 4704, 20, 2), (5, 4384, 4704, 9, 2)])
def test_experts_of_long_rows(qm, n, hidden, inner, tokens, top_k, dtype):
    """Few tiles of many units, which several thread blocks share."""
    b = Block(qm, n, hidden, inner, seed=n * hidden)
    x, ids, weights = b.rows(tokens, top_k, dtype, skew=1.0)
    out = b.check(x, ids, weights)
    assert torch.equal(qm.qm_experts_q4_0(b.handle, x, ids, weights), out)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 100])
def test_experts_rows_in_one_of_many(qm, rows, dtype):
    """All rows to the last of many experts: around the sizes of its tiles, and several of them."""
    b = Block(qm, 33, 512, 288, seed=rows)
    x, ids, weights = b.rows(rows, 2, dtype)
    ids[:, 0], ids[:, 1] = 32, -1
    b.check(x, ids, weights)
    ids[:, 1] = 32  # the same expert twice
    b.check(x, ids, weights)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens", [2, 90])
def test_experts_activations(qm, kind, gated, tokens):
    b = Block(qm, 4, 512, 320, gated=gated, kind=kind, seed=kind)
    for dtype in (F32, BF16):
        b.check(*b.rows(tokens, 2, dtype))


@pytest.mark.parametrize("tokens,count", [(1, 0), (9, 3), (130, 77), (300, 0), (257, 1)])
def test_experts_without_rows(qm, tokens, count):
    """Pairs without an expert, tokens without any, experts without rows, all rows to one expert."""
    b = Block(qm, 6, 256, 256, seed=11)
    x, ids, weights = b.rows(tokens, 3, F32)
    ids[:] = -1
    ids[:count] = torch.tensor([4, -7, 4], dtype=torch.int32, device="cuda")
    out = b.check(x, ids, weights)
    assert (out[count:] == 0).all()
    ids[:count, 1] = torch.arange(count, dtype=torch.int32, device="cuda") % 6
    b.check(x, ids, weights)


def test_experts_ids_out_of_range(qm):
    b = Block(qm, 4, 256, 256, seed=12)
    x, ids, weights = b.rows(20, 2, F32)
    ids[3, 1], ids[17, 0] = 4, 2 ** 31 - 1
    got = qm.qm_experts_q4_0(b.handle, x, ids, weights)
    assert qm.qm_device_status(clear=True) == qm.QM_ERR_RANGE
    ids[3, 1], ids[17, 0] = -1, -1
    assert torch.equal(got, b.check(x, ids, weights))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_experts_strides(qm, dtype):
    """Rows of x and out inside wider ones, experts whose gate and up share a tensor."""
    b = Block(qm, 5, 256, 320, seed=13, fused=True)
    x, ids, weights = b.rows(40, 2, dtype)
    wide = torch.randn((40, 272), generator=b.gen).to(dtype).cuda()
    wide[:, 8:264] = x
    out = torch.full((40, 300), 5.0, dtype=dtype, device="cuda")
    b.check(wide[:, 8:264], ids, weights, out=out[:, 4:260] if dtype == F32 else out[:, 8:264])
    assert (out[:, :4] == 5).all() and (out[:, 264:] == 5).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e4, 1e25])
def test_experts_sizes_of_numbers(qm, scale, dtype):
    """Rows of very small and very large numbers, and rows of both."""
    b = Block(qm, 3, 512, 256, kind=0, gated=False, seed=14)
    x, ids, weights = b.rows(50, 2, dtype)
    x[::2] *= scale
    x[5, ::3] *= scale
    b.check(x, ids, weights)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [3, 150])
def test_experts_scales_of_blocks(qm, tokens, dtype):
    """Block scales over all of binary16: 0, subnormal, very large; and a few that are infinite or NaN, which
    reach the rows that use them alone."""
    b = Block(qm, 3, 512, 256, kind=0, gated=False, seed=15)
    gen = generator(16)
    for w in (b.up, b.down):
        blocks = w.view(*w.shape[:-1], -1, 18)
        d = torch.exp(torch.rand(blocks.shape[:-1], generator=gen) * 22 - 18).half()  # 1.5e-8 .. 55
        d[torch.rand(d.shape, generator=gen) < 0.05] = 0
        blocks[..., :2] = d.unsqueeze(-1).contiguous().view(torch.uint8).cuda()
    x, ids, weights = b.rows(tokens, 2, dtype)
    ids[0] = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    ids[1:] = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    clean = b.check(x, ids, weights)
    big = b.up.view(3, 256, 16, 18)
    big[0, 5, 3, :2] = torch.tensor([6e4]).half().view(torch.uint8).cuda()
    b.check(x, ids, weights)
    big[0, 7, 2, :2] = torch.tensor([math.inf]).half().view(torch.uint8).cuda()
    big[0, 7, 2, 2:] = 0x99
    got = qm.qm_experts_q4_0(b.handle, x, ids, weights)
    assert not got[0].isfinite().any() and torch.equal(got[1:], clean[1:])


def test_experts_bad_rows(qm):
    """A row with NaN or an infinity gives what the formula does; the other rows are as without it."""
    for tokens in (5, 140):
        for dtype in (F32, BF16):
            b = Block(qm, 2, 256, 256, kind=0, gated=False, seed=17)
            x, ids, weights = b.rows(tokens, 1, dtype)
            clean = b.check(x, ids, weights)
            x2 = x.clone()
            x2[1, 7], x2[3, 200] = math.nan, math.inf
            got = qm.qm_experts_q4_0(b.handle, x2, ids, weights)
            rest = torch.ones(tokens, dtype=torch.bool)
            rest[[1, 3]] = False
            assert torch.equal(got[rest.cuda()], clean[rest.cuda()])
            assert got[1].isnan().all() and not got[3].isfinite().any()


def test_experts_one_dense_block(qm):
    """One expert and ids of 0: an ordinary feed-forward block, the product of the framework's own."""
    b = Block(qm, 1, 512, 768, seed=18)
    x = torch.randn((70, 512), generator=b.gen).cuda()
    ids = torch.zeros((70, 1), dtype=torch.int32, device="cuda")
    got = b.check(x, ids, torch.ones((70, 1), device="cuda"))
    g, u = (qm.qm_matmul_q4_0(x, w.reshape(-1), 768) for w in (b.gate, b.up))
    want = qm.qm_matmul_q4_0((torch.nn.functional.silu(g) * u).contiguous(), b.down.reshape(-1), 512)
    assert (got - want).abs().max() <= 1e-4 * want.abs().max()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 6, 400])
def test_experts_same_again(qm, tokens, dtype):
    """The same call gives the same bits, whatever the workspace held, on another stream, and in a graph whose
    inputs change between replays."""
    b = Block(qm, 8, 1024, 512, seed=19)
    x, ids, weights = b.rows(tokens, 2, dtype, skew=1.0)
    want = b.check(x, ids, weights)
    ws = torch.full((qm.qm_experts_workspace(b.handle, tokens, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(qm.qm_experts_q4_0(b.handle, x, ids, weights, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = qm.qm_experts_q4_0(b.handle, x, ids, weights, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(x)
    with torch.cuda.graph(graph):
        qm.qm_experts_q4_0(b.handle, x, ids, weights, out=out)
    x2, ids2, weights2 = b.rows(tokens, 2, dtype, idle=0.3)
    old = x.clone(), ids.clone(), weights.clone()
    for a, bb, c in ((x2, ids2, weights2), old):
        x.copy_(a), ids.copy_(bb), weights.copy_(c)
        graph.replay()
        assert torch.equal(out, qm.qm_experts_q4_0(b.handle, x, ids, weights))
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_experts_two_streams_at_once(qm, dtype):
    """Calls of all sizes on two streams at once, while a captured one is replayed on a third: each has its own
    workspace."""
    b = Block(qm, 8, 1024, 512, seed=22)
    calls = [b.rows(tokens, 2, dtype, skew=1.0) for tokens in (1, 20, 70, 300)]
    want = [qm.qm_experts_q4_0(b.handle, *c) for c in calls]
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want[1])
    with torch.cuda.graph(graph):
        qm.qm_experts_q4_0(b.handle, *calls[1], out=out)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        got += [(j, qm.qm_experts_q4_0(b.handle, *calls[j], stream=streams[s])) for s, j in enumerate((i % 4, (i + i // 4) % 4))]
        with torch.cuda.stream(streams[2]):
            graph.replay()
    torch.cuda.synchronize()
    for j, g in got:
        assert torch.equal(g, want[j])
    assert torch.equal(out, want[1])


@pytest.mark.parametrize("tokens", [1, 20, 60, 200])
def test_experts_of_zeros(qm, tokens):
    """Weights that are all 0 (quants of 8) give exactly 0, whatever their scales and the rows."""
    b = Block(qm, 4, 512, 320, seed=23)
    for w in (b.up, b.down):
        w.view(*w.shape[:-1], -1, 18)[..., 2:] = 0x88
    for dtype in (F32, BF16):
        x, ids, weights = b.rows(tokens, 2, dtype)
        assert (qm.qm_experts_q4_0(b.handle, 100 * x, ids, weights) == 0).all()


def test_experts_one_token_is_a_row_of_many(qm):
    """What a token gets hardly depends on who is with it: within the tolerance, by whichever path."""
    b = Block(qm, 8, 1024, 512, seed=20)
    x, ids, weights = b.rows(600, 2, F32)
    many = b.check(x, ids, weights)
    for i in (0, 299, 599):
        one = qm.qm_experts_q4_0(b.handle, x[i:i + 1], ids[i:i + 1], weights[i:i + 1])
        assert (one[0] - many[i]).abs().max() <= 2e-5 * many[i].abs().max()


def test_a_layer(qm):
    """Norm, logits, routing, experts and the next norm, one after the other, in a graph, against f64."""
    hidden, inner, n, k, tokens = 512, 256, 16, 4, 75
    b = Block(qm, n, hidden, inner, seed=21)
    gen = b.gen
    w_norm, w_next = (1 + 0.1 * torch.randn(hidden, generator=gen)).cuda(), (1 + 0.1 * torch.randn(hidden, generator=gen)).cuda()
    w_route = lp.q4_random((n,), hidden, gen, 1.0).cuda()
    bias = (0.05 * torch.randn(n, generator=gen)).cuda()
    attn, stream = torch.randn((tokens, hidden), generator=gen).cuda(), torch.randn((tokens, hidden), generator=gen).cuda()

    def layer(attn, stream):
        y, s, _ = qm.qm_add_rmsnorm(attn, w_norm, residual=stream)
        ids, weights = qm.qm_route_experts(qm.qm_matmul_q4_0(y, w_route.reshape(-1), n), k, bias=bias,
                                           scoring=qm.QM_SCORE_SIGMOID, n_groups=4, top_groups=3, scale=1.5)
        f = qm.qm_experts_q4_0(b.handle, y, ids, weights)
        out, s2, _ = qm.qm_add_rmsnorm(f, w_next, residual=s)
        return y, ids, weights, out, s2

    layer(attn, stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ids, weights, out, s2 = layer(attn, stream)
    attn.copy_(torch.randn((tokens, hidden), generator=gen))
    graph.replay()
    for a, c in zip((y, ids, weights, out, s2), layer(attn, stream)):
        assert torch.equal(a, c)
    # Every step against f64 on what the step before it gave.
    want, s = lp.norm(attn, w_norm, stream, 1e-6, 0.0)
    near(y, want, lp.norm_bounds(want, s, F32, 60)[0])
    f, bound = lp.experts(b.gate, b.up, b.down, y, ids, weights, 1)
    total = f + s
    near(s2, total, bound + 2.0 ** -23 * (total.abs() + bound) + 2.0 ** -24 * s.abs())
    assert (out.double() - lp.norm(s2, w_next, None, 1e-6, 0.0)[0]).abs().max() < 1e-5
