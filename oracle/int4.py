"""4-bit integer weights with group scales and their products (test
infrastructure only).

Codes 0 .. 15, two per byte with the even element in the low nibble; per group of
32, 64 or 128 elements one scale s and, in the affine form, one bias b:
    w = s (q - 8)    or    w = s q + b.
Quantisation: T rounds to the scales' type, the difference, the constants and the
products before it are float32; the quotients are rounded from float64, ties to
even:
    symmetric:  s = T(max |x| * (1/7)),   q = clamp(rne(x / s) + 8, 0, 15)
    affine:     s = T((max - min) * (1/15)), b = T(min), q = clamp(rne((x - b) / s), 0, 15)
s = 0: q = 8 (affine 0).  A group with a NaN or an infinity, or whose range or
rounded bias is infinite: s (and b) NaN, q = 8 (affine 0).

(A float32 quotient is a half integer exactly or 2^-26 away from one, relative to
a step, so float64 decides as exact arithmetic does; x - b is exact in float64
where the exponents are within 29 of each other.)

Pins (tests/test_oracle_int4.py): codes written out, ties and their neighbours,
Fractions for a small product.
"""
from __future__ import annotations

import numpy as np

from . import codecs


def _round(v, bf16):
    v = np.asarray(v, np.float32)
    return codecs.bf16_bits_to_f32(codecs.f32_to_bf16_bits(v)) if bf16 else v


def unpack(codes):
    codes = np.asarray(codes, np.uint8)
    out = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), np.int64)
    out[..., 0::2] = codes & 15
    out[..., 1::2] = codes >> 4
    return out


def pack(q):
    q = np.asarray(q, np.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def quantize(x, group, affine, bf16_scales):
    """x float32 [R, K] -> codes [R, K/2], scales [R, K/group] float32, biases or None."""
    x = np.ascontiguousarray(x, np.float32)
    r, k = x.shape
    g = x.reshape(r, k // group, group)
    bad = ~np.isfinite(g).all(axis=2)
    with np.errstate(all="ignore"):
        if affine:
            lo, hi = g.min(axis=2), g.max(axis=2)
            span = (hi - lo).astype(np.float32)
            s = _round(span * (np.float32(1) / np.float32(15)), bf16_scales)
            b = _round(lo, bf16_scales)
            bad |= ~np.isfinite(span) | ~np.isfinite(b)
        else:
            s = _round(np.abs(g).max(axis=2) * (np.float32(1) / np.float32(7)), bf16_scales)
            b = np.zeros_like(s)
        off = g.astype(np.float64) - b.astype(np.float64)[:, :, None]
        v = off / np.where(s == 0, np.inf, s.astype(np.float64))[:, :, None]
        q = np.rint(v) + (0 if affine else 8)
    q = np.where(bad[:, :, None], 0 if affine else 8, np.clip(np.nan_to_num(q), 0, 15))
    s, b = np.where(bad, np.float32(np.nan), s), np.where(bad, np.float32(np.nan), b)
    return pack(q.reshape(r, k)), s, b if affine else None


def dequantize(codes, scales, biases=None):
    """float64 [..., K]."""
    q = unpack(codes)
    group = q.shape[-1] // scales.shape[-1]
    s = np.repeat(np.asarray(scales, np.float64), group, axis=-1)
    if biases is None:
        return s * (q - 8)
    return s * q + np.repeat(np.asarray(biases, np.float64), group, axis=-1)


def product(x, experts, w, scales, biases=None):
    """x float [R, K], row i taking expert experts[i] -> (y float64 [R, N], bound
    [R, N]): the bound is the sum over groups of (23 s + |b|) sum |x|, more than
    any partial sum of s (-8 X + sum q x) + ... can reach."""
    x = np.asarray(x, np.float64)
    experts = np.asarray(experts, np.int64)
    y = np.zeros((x.shape[0], w.shape[1]))
    bound = np.zeros_like(y)
    group = 2 * w.shape[-1] // scales.shape[-1]
    mag = np.abs(x).reshape(x.shape[0], -1, group).sum(2)
    for e in np.unique(experts):
        sel = np.nonzero(experts == e)[0]
        y[sel] = x[sel] @ dequantize(w[e], scales[e], None if biases is None else biases[e]).T
        top = 23.0 * np.abs(np.asarray(scales[e], np.float64))
        if biases is not None:
            top = top + np.abs(np.asarray(biases[e], np.float64))
        bound[sel] = mag[sel] @ top.T
    return y, bound


def silu(g):
    return g / (1.0 + np.exp(-g))
