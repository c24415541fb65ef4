"""Pins of the MXFP4 oracle."""
from fractions import Fraction

import numpy as np

from oracle.mxfp4 import dequantize, product, quantize, scale_values, values

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def test_code_values_written_out():
    packed = np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], np.uint8)
    assert values(packed).tolist() == GRID + [-v for v in GRID]
    assert scale_values([0, 1, 127, 254]).tolist() == [2.0 ** -127, 2.0 ** -126, 1.0, 2.0 ** 127]
    assert np.isnan(scale_values([255])[0])


def _block(first, x):
    """Quantised value of x in a block whose largest magnitude is `first`."""
    b = np.zeros((1, 32), np.float32)
    b[0, 0], b[0, 1] = first, x
    c, s = quantize(b)
    return dequantize(c, s)[0, 1], int(s[0, 0])


def test_midpoints_go_to_the_even_code_and_neighbours_to_the_nearer_one():
    for i in range(7):
        lo, hi = GRID[i], GRID[i + 1]
        mid = np.float32((lo + hi) / 2)
        assert _block(6.0, mid)[0] == (lo if i % 2 == 0 else hi)
        assert _block(6.0, np.nextafter(mid, np.float32(0)))[0] == lo
        assert _block(6.0, np.nextafter(mid, np.float32(9)))[0] == hi
        assert _block(6.0, -np.nextafter(mid, np.float32(9)))[0] == -hi


def test_scales_of_powers_of_two_and_the_ends_of_the_range():
    for p in (-120, -3, 0, 1, 2, 60, 127):
        assert _block(2.0 ** p, 0)[1] == p - 2 + 127
        assert _block(np.nextafter(np.float32(2.0 ** p), np.float32(0)), 0)[1] == p - 3 + 127
    assert _block(0.0, 0.0)[1] == 0 and _block(2.0 ** -149, 0)[1] == 0
    assert _block(2.0 ** -126, 0)[1] == 0 and _block(2.0 ** -125, 0)[1] == 0
    assert _block(2.0 ** -124, 0)[1] == 1
    assert _block(7.9, 7.9)[0] == 6.0                       # beyond the grid saturates
    for bad in (np.inf, -np.inf, np.nan):
        v, s = _block(bad, 1.0)
        assert s == 255 and np.isnan(v)


def test_product_against_fractions():
    rng = np.random.default_rng(0)
    r, n, k, e = 3, 4, 64, 2
    rows, w = (rng.integers(0, 256, s, dtype=np.uint8) for s in ((r, k // 2), (e, n, k // 2)))
    rs = rng.integers(120, 134, (r, k // 32), dtype=np.uint8)
    ws = rng.integers(120, 134, (e, n, k // 32), dtype=np.uint8)
    experts = np.array([1, 0, 1])
    y, mag = product(rows, rs, experts, w, ws)
    for p in range(r):
        for c in range(n):
            acc, ab = Fraction(0), Fraction(0)
            for i in range(k):
                nib = lambda q, i: GRID[(int(q[i // 2]) >> (4 * (i % 2))) & 7] * (-1) ** ((int(q[i // 2]) >> (4 * (i % 2) + 3)) & 1)
                t = (Fraction(nib(rows[p], i)) * Fraction(nib(w[experts[p], c], i)) *
                     Fraction(2) ** (int(rs[p, i // 32]) + int(ws[experts[p], c, i // 32]) - 254))
                acc += t
                ab += abs(t)
            assert float(acc) == y[p, c] and float(ab) == mag[p, c]


def test_product_of_constants():
    k, n = 256, 3
    rows = np.full((2, k // 2), 0x44, np.uint8)              # 2.0
    w = np.full((1, n, k // 2), 0xBB, np.uint8)              # -1.5
    rs = np.full((2, k // 32), 128, np.uint8)
    ws = np.full((1, n, k // 32), 126, np.uint8)
    ws[0, 2, 0] = 127                                        # one block twice as large
    y, mag = product(rows, rs, [0, 0], w, ws)
    assert (y[:, :2] == -3.0 * k).all() and (y[:, 2] == -3.0 * (k + 32)).all() and (mag == -y).all()
