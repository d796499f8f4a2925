"""GPU tests of a layer's norm, routing and experts: calls that the header allows and that lie off the usual ones."""
import math

import pytest

import layer_plain as lp
from test_gpu_layer import Block, check_route, generator, near, qm  # noqa: F401 (a fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# ---- experts

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("tokens", [3, 40, 170])  # few rows an expert, up to 24, more
def test_experts_whose_gate_is_up(qm, tokens, kind, dtype):  # noqa: F811
    """One tensor as gate and as up: act(W x) * (W x), not act(W x)."""
    b = Block(qm, 4, 512, 320, kind=kind, seed=kind + 30)
    b.gate = b.up
    b.handle = qm.Experts(b.up, b.up, b.down, activation=kind)
    b.check(*b.rows(tokens, 2, dtype))


# ---- routing

@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("size", [5.0, 300.0, 3e4])
def test_route_groups_of_large_biases(qm, size, sigmoid):  # noqa: F811
    """Groups whose two choices are far larger than their sum: f32 loses of the choices what tells the sums apart.
    All experts of the groups that stay are chosen."""
    gen = generator(31)
    logits = torch.randn((300, 128), generator=gen)
    bias = torch.tensor([size, -size]).repeat(64).cuda()
    check_route(qm, logits.cuda(), 32, bias=bias, sigmoid=sigmoid, groups=64, top_groups=16)
    check_route(qm, logits.cuda(), 32, bias=bias, sigmoid=sigmoid, groups=64, top_groups=16, group_top=1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(F32).min, -3e38, 3e38])
def test_route_groups_of_extreme_biases(qm, low, sigmoid):  # noqa: F811
    """Groups masked in part or whole by biases whose sums f32 holds, loses everything in, or cannot hold."""
    gen = generator(32)
    logits = torch.randn((40, 64), generator=gen)
    bias = torch.zeros((16, 4))
    bias[::3] = low
    bias[1::3, 1:] = low
    bias = bias.reshape(-1).cuda()
    for top_groups in (2, 8, 13):
        for group_top in (1, 2):
            check_route(qm, logits.cuda(), 4, bias=bias, sigmoid=sigmoid, groups=16, top_groups=top_groups, group_top=group_top)


def test_route_weights_of_small_scores(qm):  # noqa: F811
    """Scores below f32's range have weights all the same where they are divided by their sum."""
    gen = generator(33)
    logits = torch.randn((50, 40), generator=gen)
    for at in (-60.0, -85.0, -88.0, -95.0, -110.0, -300.0, -600.0):
        check_route(qm, (logits + at).cuda(), 5, sigmoid=True, scale=2.5)
        check_route(qm, (logits + at).cuda(), 5, sigmoid=True, groups=4, top_groups=2)
    # Experts that their biases choose, far below the largest.
    for at in (-60.0, -100.0, -300.0):
        for sigmoid in (False, True):
            far = logits.clone()
            far[:, 10:] += at
            bias = torch.zeros(40)
            bias[10:20] = 4 + torch.randperm(10, generator=gen).float()
            check_route(qm, far.cuda(), 5, bias=bias.cuda(), sigmoid=sigmoid)
    # Below f64's, and masked: 0 (the formula's sum is).
    for at in (-1e4, -math.inf):
        _, weights = qm.qm_route_experts(torch.full((3, 40), at, device="cuda"), 5, scoring=qm.QM_SCORE_SIGMOID)
        assert (weights == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_experts_of_threads_on_one_stream(qm, dtype):  # noqa: F811
    """Threads that call the same experts on the same stream, each with rows of its own."""
    import threading
    b = Block(qm, 8, 512, 320, seed=40)
    calls = [b.rows(tokens, 2, dtype, skew=1.0) for tokens in (1, 30, 64, 300)]
    want = [qm.qm_experts_q4_0(b.handle, *c) for c in calls]
    torch.cuda.synchronize()
    wrong = [0] * len(calls)
    stream = torch.cuda.current_stream()

    def work(i):
        for _ in range(60):
            wrong[i] += not torch.equal(qm.qm_experts_q4_0(b.handle, *calls[i], stream=stream), want[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0] * len(calls)


# ---- the key/value cache

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_attention_of_threads_on_one_stream(qm, dtype):  # noqa: F811
    """Threads that attend to the same cache on the same stream: single tokens and prompts whose rows are done again,
    with weights and without."""
    import threading

    from test_gpu_kv_cache import device, to_dtype
    from test_gpu_kv_safety import sharp
    c, q = sharp(300, 90)
    cache = device(qm, c)
    qs = [to_dtype(q[-new:], dtype) for new in (1, 90, 1, 40)]

    def attend(i, stream=None):
        w = torch.zeros((1, 1, cache.max_len), device="cuda") if i > 1 else None
        out = qm.qm_attn_q4_0(cache, qs[i], weights=w, stream=stream)
        return (out,) if w is None else (out, w)
    want = [attend(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = [0] * 4
    stream = torch.cuda.current_stream()

    def work(i):
        for _ in range(60):
            wrong[i] += not all(torch.equal(a, b) for a, b in zip(attend(i, stream), want[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0] * 4


@pytest.mark.parametrize("at", [-20.0, -65.0, -80.0, -95.0])
def test_route_weights_of_scores_far_apart(qm, at):  # noqa: F811
    """Chosen scores of which some are below f32's range and their sum is not.  The bound is check_route's, and 2^-102:
    a score of f32 is off by 2^-128 at most (1 / (1 + exp(88.8)) comes out 0), divided by a sum of 2^-26 and more."""
    logits = (at + 12 * torch.randn((60, 40), generator=generator(34))).cuda()
    ids, weights = qm.qm_route_experts(logits, 32, scoring=qm.QM_SCORE_SIGMOID)
    want_ids, want = lp.route(logits, 32, None, True, 1, 1, 2, True, 1.0)
    assert torch.equal(ids.cpu(), want_ids)
    x = logits.double().cpu()
    dist = (x - x.amax(-1, keepdim=True)).abs().gather(1, want_ids.long()).amax(-1, keepdim=True)
    near(weights, want, (dist + 64) * 2.0 ** -24 * want.abs() * 2 + 2.0 ** -102)


@pytest.mark.parametrize("at", [-86.0, -88.5, -91.0, -103.0])
def test_route_groups_of_small_scores(qm, at):  # noqa: F811
    """Groups whose scores are near the end of f32's range, or below it."""
    gen = generator(35)
    for dtype in (F32, BF16):
        logits = (at + torch.randn((200, 64), generator=gen)).to(dtype).cuda()
        for group_top in (1, 2):
            check_route(qm, logits, 9, sigmoid=True, groups=16, top_groups=5, group_top=group_top)
            check_route(qm, logits, 9, sigmoid=True, groups=16, top_groups=5, group_top=group_top, bias=torch.zeros(64, device="cuda"))
    far = torch.zeros((200, 64))
    far[:, 1:] = at + torch.randn((200, 63), generator=gen)
    check_route(qm, far.cuda(), 9, groups=16, top_groups=5, renormalize=False)
    check_route(qm, far.cuda(), 9, renormalize=False, bias=torch.zeros(64, device="cuda"))
