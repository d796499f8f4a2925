"""A plain 64-bit implementation of the 4-bit key/value cache and its operators
in numpy, for the tests: layout, quantization, attention, accumulated weights
and eviction, written from the definitions in include/qm.h."""
import math

import numpy as np


def cell_bytes(dim):
    return 9 * dim


class Cache:
    """Host copy of a cache: pools as uint8 arrays, table, lengths."""

    def __init__(self, lengths, heads, dim, page, seed, spare=2, scale=0.1, table_extra=1):
        g = np.random.default_rng(seed)
        self.lengths = np.asarray(lengths, np.int32)
        self.heads, self.dim, self.page = heads, dim, page
        per = [-(-max(int(n), 0) // page) for n in lengths]
        self.n_pages = sum(per) + spare
        order = g.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(per), max(per + [1]) + table_extra), -1, np.int32)
        at = 0
        for i, n in enumerate(per):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.k = self._pool(g, scale)
        self.v = self._pool(g, scale)

    def _pool(self, g, scale):
        cells, nb = self.page // 16, self.dim // 32
        shape = (self.n_pages, self.heads, cells)
        q = g.integers(0, 256, (*shape, 256 * nb), dtype=np.uint8)
        d = (scale * (0.5 + np.abs(g.standard_normal((*shape, 16 * nb)))) * g.choice([-1.0, 1.0], (*shape, 16 * nb)))
        return np.concatenate([q, d.astype(np.float16).view(np.uint8)], -1).reshape(self.n_pages, self.heads, -1)

    def cell(self, pool, b, h, t):
        """The bytes of the cell that holds token t (a view)."""
        page = pool[self.table[b, t // self.page], h]
        i = t % self.page // 16
        return page[i * cell_bytes(self.dim):(i + 1) * cell_bytes(self.dim)]

    def scales(self, pool, b, h, t):
        """The token's scales (a writable float16 view)."""
        c = self.cell(pool, b, h, t)[8 * self.dim:].view(np.float16).reshape(16, -1)
        return c[t % 16]

    def values(self, pool, b, h, n=None):
        """f64 [n][dim] values of the first n tokens (default: all)."""
        n = int(self.lengths[b]) if n is None else n
        nb = self.dim // 32
        out = np.zeros((n, self.dim))
        for t0 in range(0, n, 16):
            c = self.cell(pool, b, h, t0)
            m = min(16, n - t0)
            q = c[:256 * nb].reshape(nb, 16, 16)[:, :m].astype(np.int64)
            d = c[256 * nb:].view(np.float16).astype(np.float64).reshape(16, nb)[:m]
            both = np.concatenate([q & 15, q >> 4], -1) - 8  # [nb][m][32]
            with np.errstate(invalid="ignore"):
                out[t0:t0 + m] = (both.transpose(1, 0, 2) * d[:, :, None]).reshape(m, self.dim)
        return out


def quantize(x):
    """Q4_0 quants [.., 32] and binary16 scales of f32 blocks [.., 32]."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        a = np.where(np.isnan(x), np.float32(0), np.abs(x))
        top = a.max(-1, keepdims=True)
        first = np.argmax(np.abs(x) == top, -1)[..., None]
        m = np.where(top == 0, np.float32(0), np.take_along_axis(x, first, -1))
        d = (m / np.float32(-8)).astype(np.float32)
        r = np.where(d == 0, np.float32(0), np.float32(1) / d).astype(np.float32)
        t = np.floor((x * r).astype(np.float32) + np.float32(8.5))
        q = np.where(np.isnan(t), 8, np.clip(t, 0, 15)).astype(np.uint8)
        return q, d[..., 0].astype(np.float16)


def store(cache, pool, b, h, t, row):
    """Quantize one row of f32 into its place."""
    nb = cache.dim // 32
    q, d = quantize(np.asarray(row, np.float32).reshape(nb, 32))
    c = cache.cell(pool, b, h, t)
    c[:256 * nb].reshape(nb, 16, 16)[:, t % 16] = q[:, :16] | (q[:, 16:] << 4)
    cache.scales(pool, b, h, t)[:] = d


def visible(pos, n, window, sinks):
    """bool [len(pos)][n]: which tokens rows at these positions see."""
    j = np.arange(n)[None, :]
    p = np.asarray(pos)[:, None]
    see = j <= p
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return see


def attend(cache, q, starts, n_heads, scale, window=0, sinks=0):
    """f64 (out, lse, added weights) and, for error bounds, per row and head:
    (mass [..][dim] = sum_j p_j |v_j|, reach = scale max_j sum |q k_j| over seen j)."""
    q = np.asarray(q, np.float64)
    n_seqs = len(cache.lengths)
    out = np.zeros(q.shape)
    mass = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -math.inf)
    reach = np.zeros(q.shape[:2])
    added = np.zeros((n_seqs, cache.heads, int(max(cache.lengths.max(initial=0), 1))))
    group = n_heads // cache.heads
    for b in range(n_seqs):
        first, count = int(starts[b]), int(starts[b + 1] - starts[b])
        n = int(cache.lengths[b])
        if count == 0 or n == 0:
            continue
        see = visible(np.arange(n - count, n), n, window, sinks)
        for h in range(cache.heads):
            k, v = cache.values(cache.k, b, h), cache.values(cache.v, b, h)
            for head in range(h * group, (h + 1) * group):
                x = q[first:first + count, head]
                for i in range(count):
                    s = see[i]
                    if not s.any():
                        continue
                    kk, vv = k[s], v[s]
                    with np.errstate(all="ignore"):
                        y = scale * (kk @ x[i])
                        top = y.max()
                        e = np.exp(y - top)
                        z = e.sum()
                        p = e / z
                        out[first + i, head] = p @ vv
                        mass[first + i, head] = p @ np.abs(vv)
                        lse[first + i, head] = top + np.log(z)
                        reach[first + i, head] = abs(scale) * (np.abs(kk) @ np.abs(x[i])).max()
                    added[b, h, np.nonzero(s)[0]] += p
    return out, lse, added, mass, reach


def evict(weights, length, budget, sinks, recent):
    """Kept positions (ascending) of one list of scores."""
    if length <= budget:
        return np.arange(length)
    w = np.asarray(weights[:length], np.float64)
    key = np.where(np.isnan(w), -math.inf, w)
    rank_nan = np.isnan(w)
    middle = [j for j in range(sinks, length - recent)]
    middle.sort(key=lambda j: (rank_nan[j], -key[j], j))
    keep = list(range(sinks)) + middle[:budget - sinks - recent] + list(range(length - recent, length))
    return np.asarray(sorted(keep), np.int64)
