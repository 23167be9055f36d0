"""The chunk kernels' ranges with the start weights that each kernel takes, as they stand in the
sources: over ragged batches every key tile is covered once and every cut unit is merged
whole."""
import os
import random
import re

import pytest

from tests.test_chunk_plan_host import Plan, check

HEADER = os.path.join(os.path.dirname(__file__), "..", "ragged_softmax_attention_gb300", "csrc", "fw_internal.h")


def constant(name):
    with open(HEADER) as f:
        return int(re.search(rf"constexpr int {name} = (\d+);", f.read()).group(1))


SPAN = constant("kChunkMinSpan")
# start weight, row tiles of a unit, workers: one row tile over BF16, one over FP8, two, two on pairs of CTAs
KERNELS = {"one": (constant("kChunkPieceCostOne"), 1, 152), "one FP8": (constant("kChunkPieceCost"), 1, 152),
           "two": (constant("kChunkPieceCost"), 2, 152), "pairs": (constant("kChunkPieceCostPair"), 2, 76)}


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("seed", range(25))
def test_ragged_batches_by_kernel(kernel, seed):
    cost, NT, workers = KERNELS[kernel]
    r = random.Random(5000 + seed)
    long = r.choice([1, 3, 60, 400, 2500])
    d = [r.choice([0, 1, 1, r.randint(0, long)]) for _ in range(r.choice([1, 2, 5, 17, 48]))]
    n = [r.choice([0, x, x + r.randint(0, 9000), r.randint(0, 300), x + r.randint(0, 130)]) for x in d]
    G, Hkv = r.choice([(5, 8), (4, 8), (1, 16), (4, 2), (7, 4), (32, 1), (160, 1), (300, 2), (128, 1)])
    for grid in (workers, r.choice([1, 2, 3, 7, 16])):
        for window in (-1, r.choice([0, 1, 127, 1023])):
            check(Plan(d, n, G, Hkv, NT, grid, r.random() < 0.7, window, cost, SPAN))
