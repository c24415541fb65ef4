"""MXFP4 quantisation and expert products (test infrastructure only).

The OCP microscaling format: E2M1 codes (bits s ee m; value (-1)^s * m/2 for
ee = 0, (-1)^s * (1 + m/2) * 2^(ee-1) otherwise), two per byte with the even
element in the low nibble, and one E8M0 scale byte X = 2^(X-127) per 32
elements, 255 meaning NaN.

Quantisation of a block with largest magnitude m: X = max(E - 2, 0), E the
exponent field of m as a float32 (so 2^(X-127) = 2^(floor(log2 m) - 2) for
normal m above 2^-125); the code of an element is the grid value nearest to
x / 2^(X-127), a tie going to the even code, beyond 6 to 6, the sign bit kept.
A block with a NaN or an infinity: X = 255, codes 0.

Products: y[p, n] = sum_b 2^(sx + sw - 254) sum_{k in b} q(x) q(w), in float64:
a block's sum is an integer multiple of 1/4 below 2^11 and exact, the scaled sum
over blocks is float64.  With an up projection, silu(g) * u.

Pins (tests/test_oracle_mxfp4.py): the sixteen code values written out; every
midpoint and its neighbours; powers of two as block maxima; Fraction brute
force of a small product; constant codes in closed form.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def _e2m1_values() -> np.ndarray:
    out = np.empty(16)
    for c in range(16):
        ee, m = (c >> 1) & 3, c & 1
        v = 0.5 * m if ee == 0 else (1 + 0.5 * m) * 2.0 ** (ee - 1)
        out[c] = -v if c & 8 else v
    return out


_VALUES = _e2m1_values()


def values(codes: np.ndarray) -> np.ndarray:
    """Packed codes [..., K/2] -> float64 element values [..., K] (unscaled)."""
    codes = np.asarray(codes, np.uint8)
    out = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    out[..., 0::2] = _VALUES[codes & 15]
    out[..., 1::2] = _VALUES[codes >> 4]
    return out


def scale_values(scales: np.ndarray) -> np.ndarray:
    s = np.asarray(scales, np.int64)
    return np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))


def dequantize(codes, scales) -> np.ndarray:
    """float64 [..., K]."""
    return values(codes) * np.repeat(scale_values(scales), BLOCK, axis=-1)


def quantize(x: np.ndarray):
    """x float32 [R, K] -> (codes uint8 [R, K/2], scales uint8 [R, K/32])."""
    x = np.ascontiguousarray(x, np.float32)
    r, k = x.shape
    b = x.reshape(r, k // BLOCK, BLOCK)
    bits = np.abs(b).view(np.uint32)
    e = (bits.max(axis=2) >> 23).astype(np.int64)          # NaN and inf sort above all
    bad = e == 255
    byte = np.where(bad, 255, np.maximum(e - 2, 0))
    v = np.abs(b.astype(np.float64)) / np.ldexp(1.0, np.where(bad, 0, byte) - 127)[:, :, None]
    v = np.where(bad[:, :, None], 0.0, v)
    # distance to each of the 8 magnitudes; the even code wins a tie, so look at
    # the even codes first
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    mag = order[np.argmin(np.abs(v[..., None] - _VALUES[order]), axis=-1)]
    code = np.where(bad[:, :, None], 0, mag | (np.signbit(b).astype(np.int64) << 3))
    code = code.reshape(r, k).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte.astype(np.uint8)


def product(rows, row_scales, experts, w, w_scales):
    """-> (y float64 [R, N], sum of the terms' absolute values [R, N]); row i
    takes expert experts[i]."""
    x = dequantize(rows, row_scales)
    experts = np.asarray(experts, np.int64)
    y = np.zeros((x.shape[0], w.shape[1]))
    mag = np.zeros_like(y)
    for e in np.unique(experts):
        sel = np.nonzero(experts == e)[0]
        we = dequantize(w[e], w_scales[e])
        y[sel] = x[sel] @ we.T
        mag[sel] = np.abs(x[sel]) @ np.abs(we).T
    return y, mag


def silu(g):
    return g / (1.0 + np.exp(-g))
