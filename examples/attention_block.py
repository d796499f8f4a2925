"""One attention block of a decoder over the 4-bit key/value cache: prompts,
single-token steps, accumulated weights and eviction, with Q4_0 projections.

    python examples/attention_block.py

A batch of requests goes through the block: their prompts in one call, then
steps of one token each; every token's accumulated attention weight is kept, and
when a request's cache reaches its capacity all caches are cut back to a budget
(first tokens, recent tokens, and those that were looked at most).
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_block_quantized_qm_gb300 as qm


class AttentionBlock:
    """Q4_0 projections around attention over a cache of `n_seqs` requests.
    The weights are uint8 Q4_0 block streams (rows of hidden / 32 blocks)."""

    def __init__(self, wq, wk, wv, wo, hidden, heads, kv_heads, dim, n_seqs, capacity, page_tokens=64, window=0, sinks=4):
        self.w = (wq, wk, wv, wo)
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.window, self.sinks = window, sinks
        pages = -(-capacity // page_tokens)
        pool = (n_seqs * pages, kv_heads, qm.kv_page_bytes(page_tokens, dim))
        dev = wq.device
        table = torch.arange(n_seqs * pages, dtype=torch.int32, device=dev).reshape(n_seqs, pages)
        self.cache = qm.KVCache(torch.empty(pool, dtype=torch.uint8, device=dev),
                                torch.empty(pool, dtype=torch.uint8, device=dev), table,
                                torch.zeros(n_seqs, dtype=torch.int32, device=dev), head_dim=dim, page_tokens=page_tokens)
        # What every cached token has collected; a token's count starts at 0.
        self.weights = torch.zeros((n_seqs, kv_heads, self.cache.max_len), device=dev)
        self.longest = 0  # the host's own count of the longest cache

    def forward(self, x, new):
        """x f32 [sum(new)][hidden]: `new` tokens of each request, in a row."""
        starts = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32, device=x.device)
        n = x.shape[0]
        wq, wk, wv, wo = self.w
        q = qm.qm_matmul_q4_0(x, wq, self.heads * self.dim).view(n, self.heads, self.dim)
        k = qm.qm_matmul_q4_0(x, wk, self.kv_heads * self.dim).view(n, self.kv_heads, self.dim)
        v = qm.qm_matmul_q4_0(x, wv, self.kv_heads * self.dim).view(n, self.kv_heads, self.dim)
        self.cache.lengths += starts[1:] - starts[:-1]
        self.longest += max(new)
        qm.qm_kv_append_q4_0(self.cache, k, v, q_starts=starts)
        o = qm.qm_attn_q4_0(self.cache, q, window=self.window, sinks=self.sinks, q_starts=starts, max_q=max(new),
                            weights=self.weights)
        return qm.qm_matmul_q4_0(o.view(n, self.heads * self.dim), wo, self.hidden)

    def evict(self, budget, recent):
        """Cut every request's cache back to `budget` tokens, in place."""
        kept, _ = qm.qm_kv_evict_q4_0(self.cache, self.cache, self.weights, budget, sinks=self.sinks, recent=recent,
                                      weights_out=self.weights)
        self.weights[..., budget:] = 0
        self.longest = min(self.longest, budget)
        return kept


def random_q4_0(n, k, gen):
    """A random Q4_0 weight of n rows: 18-byte blocks with scales that keep activations near 1."""
    blocks = torch.randint(0, 256, (n, k // 32, 18), dtype=torch.uint8, device="cuda", generator=gen)
    d = (torch.rand((n, k // 32, 1), device="cuda", generator=gen) + 0.5) * (0.2 / k ** 0.5)
    blocks[..., :2] = d.half().view(torch.uint8)
    return blocks.reshape(-1)


def main():
    hidden, heads, kv_heads, dim, n_seqs, capacity = 4096, 32, 8, 128, 4, 640
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = [random_q4_0(n, k, gen) for n, k in ((heads * dim, hidden), (kv_heads * dim, hidden), (kv_heads * dim, hidden),
                                             (hidden, heads * dim))]
    block = AttentionBlock(*w, hidden, heads, kv_heads, dim, n_seqs, capacity)
    prompts = [500, 37, 256, 300]
    y = block.forward(torch.randn((sum(prompts), hidden), device="cuda", generator=gen), prompts)
    print("prompts", prompts, "-> output", tuple(y.shape), "rms %.3f" % y.square().mean().sqrt())
    x = torch.randn((n_seqs, hidden), device="cuda", generator=gen)
    for step in range(200):
        if block.longest == capacity:
            block.evict(budget=384, recent=128)
            print("step", step, "evicted; lengths", block.cache.lengths.tolist())
        x = block.forward(x, [1] * n_seqs)
        x = x / x.square().mean(-1, keepdim=True).sqrt()
    print("after 200 steps: lengths", block.cache.lengths.tolist(), "weight collected per head %.1f"
          % block.weights[0, 0].sum())
    if qm.qm_device_status() != qm.QM_OK:
        raise SystemExit("a kernel reported an error")


if __name__ == "__main__":
    main()
