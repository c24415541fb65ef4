"""Helpers of the 4-bit integer product tests: which kernel a size takes, and inputs
whose products are exact in fp32.

``form_of`` repeats the rule of csrc/gemm_int4.hip (shape_of) with the constants read
from there, so a test can state the form that it is about and fails when a size no
longer takes it."""
import os
import re

import numpy as np

from oracle import codecs

SOURCE = os.path.join(os.path.dirname(__file__), "..", "combine_moe_route_topk_amd", "csrc")


def _constant(name, file="gemm_int4.hip"):
    with open(os.path.join(SOURCE, file)) as fh:
        return int(re.search(rf"\b{name} = (\d+)\b", fh.read())[1])


def form_of(r, e, k, n, group, scale_bytes, glu, aligned=True):
    """-> (form, rows of a tile, whether the product's launch groups the rows itself),
    form "wide", "deep" (K over 8 waves) or "split" (over 4)."""
    narrow, few, many = (_constant(c) for c in ("kNarrowRows", "kFewBlocks", "kManyBlocks"))
    wide_t, unit, direct_rows = _constant("kWideT"), _constant("kUnit"), _constant("kDirectRows", "expert_tiles.hpp")

    def groups(kt, waves):
        return -(-n // ((8 if glu else 16) * kt * waves))

    def tiles(height):
        return min(-(-r // height) + e, r)
    nb = 1 if r < narrow * e or tiles(32) * groups(wide_t, 4) < many else 2
    whole = aligned and k % unit == 0 and k // group * scale_bytes % 16 == 0
    t = tiles(16 * nb)
    if whole and t * groups(wide_t, 4) >= many:
        form = "wide"
    else:
        form = "deep" if nb == 1 and t * groups(4, 1) <= few else "split"
    return form, 16 * nb, nb == 1 and r <= direct_rows


def bf16(v):
    return codecs.bf16_bits_to_f32(codecs.f32_to_bf16_bits(np.ascontiguousarray(v, np.float32)))


def three_terms(x, group, terms):
    """The first ``terms`` bf16 terms of the sum of each group of x, float64 [R, K / group]."""
    left = np.asarray(x, np.float64).reshape(x.shape[0], -1, group).sum(2)
    total = np.zeros_like(left)
    for _ in range(terms):
        t = bf16(left).astype(np.float64)
        total, left = total + t, left - t
    return total


def exact_case(r, e, k, n, group, affine, glu=False, seed=0, experts=None):
    """x, experts, w, up whose every partial sum is a multiple of 1/2 below 2^23, an fp32
    number, in any order.  One group of each row has a sum of 18 bits: an element of up to
    255 2^10, one of up to 255 2^2 and small ones; with codes up to 15, scales 1/2 and 1 and
    biases up to 8 it adds at most (15 + 8) (2^18 + 2^10 + 3 * 128), below 2^22.6, and the
    others (15 + 8) 3 K, which K < 2^13 keeps below 2^19.2."""
    assert k < 2 ** 13
    rng = np.random.default_rng(seed + r + e + k + n)
    x = rng.integers(-3, 4, (r, k)).astype(np.float32)
    at = rng.integers(0, k // group, r) * group
    first = rng.integers(0, group, r)
    second = (first + 1 + rng.integers(0, group - 1, r)) % group
    odd = lambda: 2 * rng.integers(64, 128, r) + 1                 # 129 .. 255
    x[np.arange(r), at + first] = odd() * 2.0 ** 10 * rng.choice([-1, 1], r)
    x[np.arange(r), at + second] = odd() * 2.0 ** 2 * rng.choice([-1, 1], r)
    ex = rng.integers(0, e, r).astype(np.int32) if experts is None else np.asarray(experts, np.int32)

    def weights():
        codes = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
        s = np.where(rng.random((e, n, k // group)) < 0.5, 0.5, 1.0).astype(np.float32)
        b = rng.integers(-8, 9, s.shape).astype(np.float32) if affine else None
        return codes, s, b
    return x, ex, weights(), weights() if glu else None
