"""A workspace of moe_balance_loss made for the largest batch holds every smaller one."""
import random

from combine_moe_route_topk_amd import _lib

size = _lib.lib.moe_balance_loss_workspace_bytes


def test_sizes_grow_with_tokens():
    # around every border of the chunk length: 16 k tokens per workgroup, and the mean sequence
    borders = sorted({max(0, m * 16384 + d) for m in range(6) for d in (-1, 0, 1, 2)} |
                     {m * b + d for b in (1, 3, 4, 37, 2048) for m in (1, 2, 3, 15, 16, 17) for d in (-1, 0, 1)} |
                     {2**20, 2**20 + 1, 2**31 - 2, 2**31 - 1})
    for e in (8, 256, 1024):
        for b in (1, 3, 4, 37, 2048, 20000, 1 << 20):
            sizes = [size(n, e, b) for n in borders]
            assert sizes == sorted(sizes) and sizes[0] > 0, (e, b)


def test_sizes_grow_with_sequences_and_experts():
    for n in (0, 1, 16, 63, 64, 65, 4095, 4096, 16384, 16385, 32768, 2**31 - 1):
        for e in (7, 256, 1024):
            sizes = [size(n, e, b) for b in (1, 2, 3, 4, 5, 16, 37, 255, 2047, 2048, 4096, 20000, 32768, 1 << 20)]
            assert sizes == sorted(sizes), (n, e)
        sizes = [size(n, e, 37) for e in range(1, 1025)]
        assert sizes == sorted(sizes), n


def test_smaller_batches_fit():
    rng = random.Random(0)
    for _ in range(20000):
        n, e, b = (int(2 ** rng.uniform(0, top)) for top in (31, 10, 20))
        assert size(rng.randint(0, n - 1), rng.randint(1, e), rng.randint(1, b)) <= size(n - 1, e, b), (n, e, b)
