"""The MXFP4 products element by element: the gate's activation over its whole
range, and every block's own scales.

silu(a) = a / (1 + e^-a) is formed from the exponential and reciprocal
instructions.  The exponent a * -log2(e) is rounded once, and its constant is
2^-26.1 off: |a| (2^-24 + 2^-26.1) relative in e^-a, which counts where a < 0.
The two instructions (1 ulp each), the sum and two products add less than 2^-21.
Down to a = -87 the result is within 2^-21 + |a| 2^-23.6 of silu(a) * u, then
rounded to bf16 (2^-8, or half its smallest subnormal, 2^-134).  Below, the
reciprocal's subnormals are lost: the result lies between 0 and the value.

Block scales: where a gate is 128 or more, silu(a) = a to 2^-180, so both
factors are sums of ones scaled by powers of two, exact in fp32, and only
roundings are left: 2^-8 + 2^-21.  A block with scale 2^0 is 1 part in K / 32 of
its sum, which is 2^-7.1 or more up to K = 4224, and a raised one 8 times that,
so no missing or misplaced block passes.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle import codecs
from oracle.mxfp4 import product, silu
from tests.gpu_util import as_f32, to_dev, to_np

pytestmark = pytest.mark.gpu


def _call(kind, rows, rs, ids, w, up=None):
    args = [to_dev(rows), to_dev(rs)]
    kw = {} if up is None else dict(w_up=to_dev(up[0]), w_up_scales=to_dev(up[1]))
    if kind == "gather":
        y = moe.moe_gather_gemm_mxfp4(*args, to_dev(ids), to_dev(w[0]), to_dev(w[1]), **kw)
    else:
        offs = np.searchsorted(ids, np.arange(w[0].shape[0] + 1)).astype(np.int32)
        y = moe.moe_grouped_gemm_mxfp4(*args, to_dev(offs), to_dev(w[0]), to_dev(w[1]), **kw)
    return as_f32(to_np(y)).astype(np.float64)


@pytest.mark.parametrize("r", [3, 100])                              # streamed weights, tiles
@pytest.mark.parametrize("p", [0, 40, 100])
def test_silu_over_its_range(r, p):
    """Gates -128, -127.5, ..., 128 exactly, times u = 2^p."""
    a = np.arange(-256, 257) / 2.0
    n, k = a.size, 128
    codes = np.zeros((n, k), np.uint8)
    for i, v in enumerate(np.abs(a)):
        codes[i, :int(v)] = 2                                        # ones, and a half
        if v % 1:
            codes[i, int(v)] = 1
    codes |= np.where(a < 0, 8, 0).astype(np.uint8)[:, None]
    up = np.zeros((n, k), np.uint8)
    up[:, 5] = 2
    pack = lambda c: (c[:, 0::2] | (c[:, 1::2] << 4))[None]
    one = lambda *s: np.full(s, 127, np.uint8)
    got = _call("grouped", np.full((r, k // 2), 0x22, np.uint8), one(r, k // 32), np.zeros(r, np.int32),
                (pack(codes), one(1, n, k // 32)), (pack(up), one(1, n, k // 32) + np.uint8(p)))
    want = silu(a) * 2.0 ** p
    assert (got == got[0]).all()
    near = a >= -87
    bound = (2.0 ** -8 + 2.0 ** -21 + np.abs(a) * 2.0 ** -23.6) * np.abs(want) + 2.0 ** -134
    assert (np.abs(got[0] - want) <= bound)[near].all()
    assert ((got[0] <= 0) & (got[0] >= want - bound))[~near].all()


def _raised(rng, codes_shape, k):
    """Scales 2^0 with each block raised to 2^3 in one place."""
    s = np.full(codes_shape[:-1] + (k // 32,), 127, np.uint8)
    flat = s.reshape(-1, k // 32)
    flat[rng.permutation(np.arange(k // 32) % flat.shape[0]), np.arange(k // 32)] += 3
    return s


# 16-row tiles (grouped inside the launch for rows in any order), 32- and 64-row
# tiles, and the tile kernel; K of whole and of partial stages
@pytest.mark.parametrize("kind", ["grouped", "gather"])
@pytest.mark.parametrize("r", [12, 40, 70, 300])
@pytest.mark.parametrize("k", [384, 2048, 2688, 4224])
@pytest.mark.parametrize("glu", [False, True])
def test_each_block_takes_its_own_scales(kind, r, k, glu):
    rng = np.random.default_rng(r + k)
    e, n = 2, 48
    rows, w = np.full((r, k // 2), 0x22, np.uint8), np.full((e, n, k // 2), 0x22, np.uint8)
    rs, ws, us = (_raised(rng, s, k) for s in ((r, 1), (e, n, 1), (e, n, 1)))
    ids = np.sort(np.arange(r) % e).astype(np.int32)
    if kind == "gather":
        ids = rng.permutation(ids)
    got = _call(kind, rows, rs, ids, (w, ws), (w, us) if glu else None)
    g, _ = product(rows, rs, ids, w, ws)
    if not glu:
        assert np.array_equal(got, as_f32(codecs.f64_to_bf16_bits(g)))
        return
    assert g.min() >= 128
    u, _ = product(rows, rs, ids, w, us)
    assert (np.abs(got - g * u) <= (2.0 ** -8 + 2.0 ** -21) * g * u).all()
