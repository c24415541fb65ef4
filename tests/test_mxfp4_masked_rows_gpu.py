"""moe_gather_gemm_mxfp4 with many rows whose id lies outside [0, E), as the rank
of an expert-parallel layer passes them for the rows of other ranks.

The tile kernel halves its columns where the tiles that really exist are few;
with many such rows they are fewer than the row count suggests, and every
column of every valid row still has to be written.  Tolerance as for the other
products: half a step of bf16 (2^-8) of the result plus 2^-11 of the terms'
magnitude for the fp32 accumulation on the matrix cores; with SwiGLU the same
through |silu'| <= 1.1.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle import codecs
from oracle.mxfp4 import product, silu
from tests.gpu_util import DEV, as_f32, to_dev, to_np

pytestmark = pytest.mark.gpu


def _operand(rng, *shape, low=121):
    k = shape[-1]
    return (rng.integers(0, 256, shape[:-1] + (k // 2,), dtype=np.uint8),
            rng.integers(low, low + 13, shape[:-1] + (k // 32,), dtype=np.uint8))


# rows of each expert, rows without one, N, SwiGLU: between what the row count
# and what the valid rows say about the number of tiles; at its ends; none valid
CASES = [([400] * 4, 800, 4096, False), ([384] * 4, 1024, 2048, True), ([512] * 8, 256, 2048, False),
         ([512] * 8, 256, 1024, True), ([716], 308, 8448, False), ([32768], 256, 256, False),
         ([1, 0, 130, 300], 4000, 4200, False), ([256], 5000, 4200, True), ([0, 0], 3000, 2100, False),
         ([0, 700, 0, 1], 3500, 1050, True)]


@pytest.mark.parametrize("counts,gone,n,glu", CASES)
def test_every_column_of_every_valid_row(counts, gone, n, glu):
    e, r, k = len(counts), sum(counts) + gone, 256
    rng = np.random.default_rng(r + n)
    ids = np.concatenate([np.repeat(np.arange(e), counts), np.tile([-1, e, 2**31 - 1, -2**31], gone)[:gone]])
    ids = rng.permutation(ids).astype(np.int32)
    low = 117 if glu else 121                                        # gates of moderate size
    rows, rs = _operand(rng, r, k, low=low)
    w = _operand(rng, e, n, k, low=low)
    up = _operand(rng, e, n, k) if glu else None
    y = torch.full((r, n), 7.0, dtype=torch.bfloat16, device=DEV)
    kw = dict(w_up=to_dev(up[0]), w_up_scales=to_dev(up[1])) if glu else {}
    moe.moe_gather_gemm_mxfp4(to_dev(rows), to_dev(rs), to_dev(ids), to_dev(w[0]), to_dev(w[1]), y=y, **kw)
    good = (ids >= 0) & (ids < e)
    bits = to_np(y)
    assert (as_f32(bits[~good]) == 7).all()
    got = as_f32(bits[good]).astype(np.float64)
    g, mg = product(rows[good], rs[good], ids[good], *w)
    want, bound = g, 2.0 ** -8 * np.abs(g) + 2.0 ** -11 * mg
    if glu:
        u, mu = product(rows[good], rs[good], ids[good], *up)
        with np.errstate(over="ignore"):
            s = silu(g)
        want = s * u
        bound = ((2.0 ** -8 + 2.0 ** -20) * np.abs(want) +
                 2.0 ** -11 * (1.1 * mg * np.abs(u) + mu * np.abs(s)) + 2.0 ** -22 * mg * mu)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside the bound"
