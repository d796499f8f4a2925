"""GPU tests of how the step kernel cuts its work: batches whose tile lists lie
end to end (an equal stretch for each CTA, lists cut wherever a stretch ends) and
warps that go through more tiles than their rings hold, against the plain
implementation.  The rule that cuts is replayed here, and each case says which of
its two forms it reaches and how many tiles a warp has to take.
"""
import numpy as np
import pytest

import kv_oracle as ko

pytest.importorskip("torch")
from test_gpu_kv_cache import BF16, F32, check_attend, qm  # noqa: E402,F401

TILE, WARPS = 64, 4


def tile_count(length, count, window, sinks):
    """Tiles of 64 tokens that a list of a sequence with `count` rows goes through."""
    if count == 0:
        return 0
    total = -(-length // TILE)
    n = total
    if window > 0:
        lo = max(0, max(length - count, 0) - window + 1)
        n1 = min(-(-min(sinks, lo) // TILE), total)
        n = n1 + max(0, total - max(n1, lo // TILE))
    return max(n, 1)


def split(lengths, new, kv, group, max_len, window, sinks):
    """(form, tiles per CTA at most, tiles of the longest list) for the grid of a GPU with 152 SMs."""
    rows = max(new) * group
    rows_cta = 4 if rows <= 4 else 8
    groups = -(-rows // rows_cta)
    lists = kv * groups
    tiles = [tile_count(n, m, window, sinks) for n, m in zip(lengths, new)]
    n_lists = len(lengths) * lists
    most = max(1, -(-max_len // TILE)) * n_lists
    grid = min(456, 152 * (3 if rows_cta == 4 else 2), max(-(-most // WARPS), n_lists))
    total = sum(tiles) * lists
    per = max(WARPS, -(-(-(-total // grid)) // WARPS) * WARPS)
    p = per
    while p <= max(per + per // 4, 2 * WARPS):
        if sum(-(-t // p) for t in tiles) * lists <= grid:
            return "ranges", p, max(tiles)
        p += WARPS
    return "stretches", per, max(tiles)


def ragged(n, lo, hi, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi + 1, n)]


# lengths, new rows, kv heads, group, dim, page, window, sinks, form, tiles of a warp at least
CASES = [
    (ragged(64, 300, 3000, 1), [1] * 64, 8, 4, 128, 64, 0, 0, "stretches", 7),
    (ragged(48, 300, 3000, 2), [1, 1, 0] * 16, 8, 1, 64, 16, 0, 0, "stretches", 3),
    (ragged(40, 1, 2500, 3), [1] * 40, 8, 3, 128, 16, 0, 0, "stretches", 3),
    (ragged(64, 700, 2600, 4), [1] * 64, 4, 8, 128, 64, 0, 0, "stretches", 4),      # CTAs of 8 rows
    (ragged(40, 20, 1500, 5), ([5, 1, 0, 3] * 10), 4, 4, 64, 32, 0, 0, "stretches", 4),  # drafts
    (ragged(64, 300, 3000, 6), [1] * 64, 8, 4, 128, 32, 700, 70, "stretches", 3),
    (ragged(30, 100, 1800, 7), [3] * 30, 8, 2, 128, 128, 900, 5, "stretches", 3),
    ([9000], [1], 8, 4, 128, 64, 0, 0, "ranges", 1),
    (ragged(64, 300, 3000, 8), [1] * 64, 16, 2, 64, 16, 0, 0, "stretches", 11),
    ([4200, 4100], [1, 1], 200, 1, 64, 16, 0, 0, "ranges", 16),  # a CTA per list
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join([str(len(c[0])), *(str(x) for x in c[2:9])]))
def test_split(case):
    """The rule's replay, so that the cases below reach what they are there for."""
    lengths, new, kv, group, dim, page, window, sinks, form, least = case
    per_seq = -(-max(lengths) // page) + 1
    got, per, longest = split(lengths, new, kv, group, per_seq * page, window, sinks)
    assert got == form
    assert min(per, longest) // WARPS >= least, (per, longest)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("weights", [False, True], ids=["", "weights"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join([str(len(c[0])), *(str(x) for x in c[2:9])]))
def test_step(qm, case, weights, dtype):  # noqa: F811
    lengths, new, kv, group, dim, page, window, sinks, _, _ = case
    c = ko.Cache(lengths, kv, dim, page, seed=len(lengths) + page)
    check_attend(qm, c, new, kv * group, dtype, window, sinks, weights=weights)
