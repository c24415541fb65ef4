"""Products with 4-bit integer weights where there are many tiles, so that the waves
of a workgroup split the columns: each form against float64.

Tolerance, as for the other forms: (528 + 2 groups + 6) 2^-24 of the sum of magnitudes.
Here a group's sum rounds at most 128 times and once per group when scaled; X, the sum
of x over a group, at most 12 times and once in its three bf16 terms; their products
with the biases are exact and added in at most 3 roundings a group: 141 + 4 groups,
which is less for up to 193 groups.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from tests.gpu_util import DEV, to_dev, to_np
from tests.test_int4_gpu import BF16, F32, FORMS, _bits, _call, _case, _check, _dev

pytestmark = pytest.mark.gpu

# whole rows of scales in both types, and the last 16 groups half there
K = {32: 1280, 64: 2560, 128: 5120}


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("r,e,n", [(160, 150, 140), (320, 30, 1001)])
def test_many_tiles(r, e, n, glu, group, affine, scale_dtype):
    # one expert of several tiles, one of a full one, one of a single row
    rng = np.random.default_rng(n)
    ex = rng.integers(3, e, r)
    ex[rng.permutation(r)[:70]] = 0
    ex[rng.permutation(np.nonzero(ex)[0])[:17]] = [1] * 16 + [2]
    case = _case(r, e, K[group], n, group, affine, scale_dtype, glu, experts=ex)
    out_dtype = BF16 if glu else F32
    y = _call(case, scale_dtype, out_dtype)
    _check(y, case, out_dtype)
    assert np.array_equal(to_np(y), to_np(_call(case, scale_dtype, out_dtype)))


@pytest.mark.parametrize("units", [1, 2, 3, 4, 5])
def test_many_tiles_short_rows(units):
    for group in (32, 64, 128):
        if units * 256 % (8 * group):
            continue
        case = _case(160, 150, units * 256, 140, group, True, BF16)
        _check(_call(case, BF16, F32), case, F32)


@pytest.mark.parametrize("k", [160, 256, 416, 1056])
def test_many_rows_and_ends_inside_a_unit(k):
    for affine, scale_dtype, glu in ((False, BF16, True), (True, F32, False)):
        case = _case(320, 30, k, 1001, 32, affine, scale_dtype, glu)
        _check(_call(case, scale_dtype, F32), case, F32)


@pytest.mark.parametrize("affine", [False, True])
def test_scales_that_begin_at_4_bytes(affine):
    """Scales that are no whole 16 bytes from a line take another form; the same product."""
    x, ex, w, _ = case = _case(160, 150, 1280, 140, 32, affine, BF16)
    want = _call(case, BF16, F32)

    def moved(t):
        if t is None:
            return None
        buf = torch.empty(t.numel() + 2, dtype=t.dtype, device=t.device)
        buf[2:] = t.reshape(-1)
        return buf[2:].view(t.shape)
    codes, s, b = _dev(w, BF16)
    got = moe.moe_gather_gemm_int4(to_dev(_bits(x)), to_dev(ex), codes, moved(s), moved(b), out_dtype=F32)
    _check(got, case, F32)
    _check(want, case, F32)


@pytest.mark.parametrize("affine", [False, True])
def test_one_element_reaches_every_column_once(affine):
    """x is 1 in one place: the result is that weight, exactly (no other term is not 0)."""
    r, e, k, n = 160, 150, 1280, 140
    x, ex, w, _ = _case(r, e, k, n, 32, affine, F32 if not affine else BF16)
    at = (np.arange(r) * 37) % k
    x = np.zeros((r, k), np.float32)
    x[np.arange(r), at] = 1.0
    scale = F32 if not affine else BF16
    if affine:                                   # both terms and their sum are bf16 numbers times powers of 2
        w = (w[0], np.full_like(w[1], 0.5), np.round(w[2] * 64) / 4)
    y = to_np(_call((x, ex, w, None), scale, F32))
    byte = w[0][ex, :, at // 2]
    q = np.where((at % 2 == 1)[:, None], byte >> 4, byte & 15).astype(np.float64)
    s = w[1][ex, :, at // 32].astype(np.float64)
    want = s * (q - 8) if not affine else s * q + w[2][ex, :, at // 32]
    if affine:
        assert np.array_equal(y, want)
    else:                                        # s (-8) and s q in one fp32 product of exact sums
        assert np.array_equal(y, (s * (q - 8)).astype(np.float32))


@pytest.mark.parametrize("r,e,n", [(160, 150, 140), (320, 30, 1001)])
def test_many_tiles_rows_without_an_expert_stay(r, e, n):
    ex = np.arange(r) % e
    ex[::4], ex[1::5], ex[2::7] = -1, e, -2**31
    case = _case(r, e, 1280, n, 32, True, BF16, experts=ex)
    y = torch.full((r, n), 7.0, dtype=F32, device=DEV)
    _call(case, BF16, F32, y=y)
    _check(y, case, F32)
    assert (y[to_dev((ex < 0) | (ex >= e))] == 7).all()


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("r,e,n", [(160, 150, 140), (320, 30, 1001)])
def test_many_tiles_nan_and_infinity_stay(r, e, n, affine):
    case = _case(r, e, 1280, n, 32, affine, BF16, experts=np.arange(r) % e)
    clean = _call(case, BF16, F32)
    x = case[0].copy()
    x[2, 3], x[5, 1279] = np.nan, np.inf
    got = _call((x, *case[1:]), BF16, F32)
    rows = torch.ones(r, dtype=torch.bool, device=DEV)
    rows[[2, 5]] = False
    assert not torch.isfinite(got[~rows]).any() and torch.equal(got[rows], clean[rows])
    hit = torch.zeros((r, n), dtype=torch.bool, device=DEV)
    hit[to_dev(case[1] == 0), 7] = True
    for part in (1, 2) if affine else (1,):            # a scale, a bias
        w = [v if v is None else v.copy() for v in case[2]]
        w[part][0, 7, -1] = np.nan
        got = _call((case[0], case[1], tuple(w), None), BF16, F32)
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


def test_many_tiles_replayed():
    """Two captured products, of 16- and 32-row tiles, that share a workspace."""
    ws = torch.empty(max(moe.moe_gather_gemm_int4_workspace_bytes(r, e) for r, e in ((160, 150), (320, 30))),
                     dtype=torch.uint8, device=DEV)
    steps = []
    for r, e, n in ((160, 150, 140), (320, 30, 1001)):
        case = _case(r, e, 1280, n, 32, True, BF16)
        w, x, ex = _dev(case[2], BF16), to_dev(_bits(case[0])), to_dev(case[1])
        y = torch.empty((r, n), dtype=BF16, device=DEV)

        def step(x=x, ex=ex, w=w, y=y):
            moe.moe_gather_gemm_int4(x, ex, *w, y=y, workspace=ws)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        steps.append((x, ex, e, y, step, g))
    for rep in range(4):
        for x, ex, e, y, step, g in steps:
            x.copy_(torch.roll(x, 1, 0))
            ex.copy_((ex + 1) % e)
            y.fill_(7)
            ws.fill_(255)
            g.replay()
            got = y.clone()
            torch.cuda.synchronize()
            step()
            assert torch.equal(got, y), rep
