"""Pins of the 4-bit integer oracle."""
from fractions import Fraction

import numpy as np
import pytest

from oracle.int4 import dequantize, pack, product, quantize, unpack


def test_codes_written_out():
    packed = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2], np.uint8)
    assert unpack(packed)[0].tolist() == list(range(16)) * 2
    assert np.array_equal(pack(unpack(packed)), packed)
    assert dequantize(packed, np.array([[0.5]]))[0, :16].tolist() == [(q - 8) * 0.5 for q in range(16)]
    assert dequantize(packed, np.array([[0.5]]), np.array([[3.0]]))[0, :16].tolist() == [q * 0.5 + 3 for q in range(16)]


def _codes(x, affine=False, bf16=False, group=32):
    c, s, b = quantize(x, group, affine, bf16)
    return unpack(c), s, b


def test_ties_go_to_even_and_neighbours_to_the_nearer():
    third = np.float32(1) / np.float32(7)
    for half in (0.5, 1.5, 2.5, 5.5, -0.5, -3.5):
        for step, want in ((0, round(half)), (1, int(np.floor(half)) + 1), (-1, int(np.floor(half)))):
            x = np.zeros((1, 32), np.float32)
            x[0, 0] = 7.0
            assert np.float32(7.0) * third == 1.0            # s = 1
            v = np.float32(half)
            x[0, 1] = np.nextafter(v, np.float32(99 * step)) if step else v
            q, s, _ = _codes(x)
            assert s[0, 0] == 1.0 and q[0, 1] - 8 == want, (half, step)


def test_affine_of_a_ramp_and_constants():
    x = np.tile(np.arange(16, dtype=np.float32) * 0.25 - 3.0, 2)[None]
    q, s, b = _codes(x, affine=True)
    assert s[0, 0] == 0.25 and b[0, 0] == -3.0 and q[0].tolist() == list(range(16)) * 2
    q, s, b = _codes(np.full((1, 32), 5.5, np.float32), affine=True)
    assert s[0, 0] == 0 and b[0, 0] == 5.5 and (q == 0).all()
    q, s, _ = _codes(np.zeros((1, 32), np.float32))
    assert s[0, 0] == 0 and (q == 8).all()


def test_groups_that_are_not_finite():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 64), np.float32)
        x[0, 40] = bad
        q, s, _ = _codes(x)
        assert np.isfinite(s[0, 0]) and np.isnan(s[0, 1]) and (q[0, 32:] == 8).all()
        q, s, b = _codes(x, affine=True)
        assert b[0, 0] == 1.0 and np.isnan(s[0, 1]) and np.isnan(b[0, 1]) and (q[0, 32:] == 0).all()
    x = np.zeros((1, 32), np.float32)
    x[0, 0], x[0, 1] = 3e38, -3e38
    assert np.isnan(_codes(x, affine=True)[1][0, 0]) and np.isfinite(_codes(x)[1][0, 0])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_values_are_within_half_a_step(affine, bf16):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 256)).astype(np.float32)
    c, s, b = quantize(x, 64, affine, bf16)
    step = np.repeat(s.astype(np.float64), 64, 1)
    # a bf16 bias or scale may move the ends of the range by 2^-9 of themselves
    slack = 2.0 ** -8 * np.abs(x).max() if bf16 else 2.0 ** -20
    assert (np.abs(dequantize(c, s, b) - x) <= 0.5 * step + slack).all()


@pytest.mark.parametrize("affine", [False, True])
def test_product_against_fractions(affine):
    rng = np.random.default_rng(0)
    r, n, k, e, g = 3, 4, 64, 2, 32
    x = rng.integers(-64, 64, (r, k)) / 16.0
    w = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    s = rng.integers(1, 64, (e, n, k // g)) / 256.0
    b = rng.integers(-64, 64, (e, n, k // g)) / 32.0 if affine else None
    experts = np.array([1, 0, 1])
    y, bound = product(x, experts, w, s, b)
    for p in range(r):
        for c in range(n):
            acc, top = Fraction(0), Fraction(0)
            for i in range(k):
                q = (int(w[experts[p], c, i // 2]) >> (4 * (i % 2))) & 15
                sc = Fraction(s[experts[p], c, i // g])
                bi = Fraction(b[experts[p], c, i // g]) if affine else -8 * sc
                acc += Fraction(x[p, i]) * (sc * q + bi)
                top += abs(Fraction(x[p, i])) * (23 * sc + (abs(bi) if affine else 0))
            assert float(acc) == pytest.approx(y[p, c], rel=1e-15) and float(top) == pytest.approx(bound[p, c], rel=1e-15)
