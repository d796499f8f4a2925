"""GPU test of the example that runs the cache's operators together: prompts, steps
and an eviction against plain torch on what the cache holds."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_block_quantized_qm_gb300 import build as qm_build
    qm_build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import attention_block
    torch.cuda.set_device(0)
    return attention_block


def plain(block, x, new):
    """The block on the cache's own values, in f64."""
    import bit_block_quantized_qm_gb300 as qm
    wq, _, _, wo = block.w
    d = block.dim
    lengths = block.cache.lengths.tolist()
    out, first = [], 0
    q = (x.double() @ qm.qm_dequant_q4_0(wq).view(block.heads * d, -1).double().T).view(-1, block.heads, d)
    everything = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    k_all, v_all = qm.qm_kv_read_q4_0(block.cache, int(everything[-1]), q_starts=everything)
    for b, (m, n) in enumerate(zip(new, lengths)):
        k, v = (t[int(everything[b]):int(everything[b + 1])].double().repeat_interleave(block.heads // block.kv_heads, 1)
                for t in (k_all, v_all))
        s = torch.einsum("qhd,khd->hqk", q[first:first + m], k) / d ** 0.5
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        s.masked_fill_(torch.arange(n, device="cuda")[None, :] > pos, float("-inf"))
        out.append(torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v))
        first += m
    o = torch.cat(out).reshape(-1, block.heads * d)
    return o @ qm.qm_dequant_q4_0(wo).view(block.hidden, -1).double().T


def test_prompts_steps_and_eviction(example):
    hidden, heads, kv_heads, dim, n_seqs = 512, 8, 2, 64, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = [example.random_q4_0(n, k, gen) for n, k in ((heads * dim, hidden), (kv_heads * dim, hidden),
                                                     (kv_heads * dim, hidden), (hidden, heads * dim))]
    block = example.AttentionBlock(*w, hidden, heads, kv_heads, dim, n_seqs, capacity=300, page_tokens=32)

    def check(new):
        x = torch.randn((sum(new), hidden), device="cuda", generator=gen)
        got = block.forward(x, new).double()
        want = plain(block, x, new)
        # f32 products and sums throughout, queries taken in f32: 2^-17 per product of
        # the projections at most, on two of them and the scores between.
        assert float((got - want).norm() / want.norm()) < 1e-4

    check([200, 17, 90])
    for _ in range(3):
        check([1, 1, 1])
    total = block.weights.sum((1, 2))  # every row of every head has given 1
    rows = torch.tensor([203, 20, 93], device="cuda") * heads
    assert torch.allclose(total, rows.float(), rtol=1e-5)
    kept = block.evict(budget=64, recent=16)
    assert block.cache.lengths.tolist() == [64, 20, 64]
    assert (kept[0, :, :4] == torch.arange(4, device="cuda")).all() and (kept[1, :, 20:] == -1).all()
    check([1, 1, 1])
    check([5, 2, 40])


def test_the_example_runs(example, capsys):
    example.main()
    assert "after 200 steps" in capsys.readouterr().out
