"""A workspace of the gather products made for the most rows holds every smaller call."""
import random

import pytest

from combine_moe_route_topk_amd import _lib

SIZES = [_lib.lib.moe_gather_gemm_int4_workspace_bytes, _lib.lib.moe_gather_gemm_mxfp4_workspace_bytes]


@pytest.mark.parametrize("size", SIZES)
def test_sizes_grow_with_rows_and_experts(size):
    # around every length at which the grouping takes larger chunks of rows
    rows = sorted({max(0, m * 16384 + d) for m in range(70) for d in (-1, 0, 1, 2)} |
                  {m << 20 for m in range(1, 2048, 97)} | {1, 64, 65, 255, 256, 257, 2**20 + 1, 2**31 - 1})
    for e in (1, 8, 300, 1024):
        sizes = [size(n, e) for n in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0, e
    for n in (0, 64, 16384, 16385, 2**20, 2**20 + 1, 2**31 - 1):
        sizes = [size(n, e) for e in range(1, 1025)]
        assert sizes == sorted(sizes), n


@pytest.mark.parametrize("size", SIZES)
def test_smaller_calls_fit(size):
    rng = random.Random(0)
    for _ in range(20000):
        n, e = int(2 ** rng.uniform(0, 31)), int(2 ** rng.uniform(0, 10))
        assert size(rng.randint(0, n - 1), rng.randint(1, e)) <= size(n - 1, e), (n, e)
