"""Products with 4-bit integer weights in each form that a size can take (form_of): against
float64, exactly where every partial sum is an fp32 number, and by the mean square error of
random inputs.

Mean square, u = 2^-24.  For inputs of independent signs the mean square of any partial sum
is at most the sum of the squares of all terms in it.  A group's sum is 33 additions in each
of up to 2 G / 32 matrix instructions (half of them for the constant or X), each off by at
most a step, 2 u of the partial sum; the root mean squares of all these errors add at most
linearly:
    2 u 33 (G / 16) sum_groups s sqrt(sum (q^2 + 64) x^2)     (64: the constant -8)
for codes and constant; with the biases 2 u 33 (G / 32) (s sqrt(sum q^2 x^2) + |b| sqrt(sum
x^2)) a group.  Adding the groups, scaled, takes 2 roundings a group and 8 parts of K 14 more,
each at most u of a sum with mean square sum (s q + b)^2 x^2 <= 2 sum (s^2 q^2 + b^2) x^2.
Biases multiplied by the matrix cores are three products for 16 groups, 3 * 17 additions off
by 2 u of such a sum: below 8 u more a group.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle.int4 import product, unpack
from tests.gpu_util import DEV, to_dev, to_np
from tests.int4_forms import exact_case, form_of
from tests.test_int4_gpu import BF16, F32, FORMS, U, _bits, _call, _case, _check, _dev

pytestmark = pytest.mark.gpu

WHOLE = {32: 768, 64: 1536, 128: 1024}       # whole 256s and whole 16 bytes of scales
LONG = {32: 2048, 64: 2048, 128: 2048}       # two units for each of four waves
RAGGED = {32: 2080, 64: 2240, 128: 2176}     # and a part of one more
# rows, experts, K, columns (with SwiGLU), and the form
SHAPES = {
    "wide, rows found in the launch": (64, 64, WHOLE, 600, 260, ("wide", 16, True)),
    "wide, 16 rows": (160, 150, WHOLE, 140, 70, ("wide", 16, False)),
    "wide, 32 rows": (320, 30, WHOLE, 1001, 501, ("wide", 32, False)),
    "deep": (20, 2, RAGGED, 100, 50, ("deep", 16, True)),
    "deep, grouped": (70, 8, RAGGED, 100, 50, ("deep", 16, False)),
    "split, rows found in the launch": (40, 40, LONG, 260, 130, ("split", 16, True)),
    "split, 16 rows": (90, 30, RAGGED, 260, 130, ("split", 16, False)),
    "split, 32 rows": (320, 30, RAGGED, 1001, 501, ("split", 32, False)),
}


def _experts(r, e, skip=True):
    """One expert of several tiles, one of a full one, one row of the last, rows of none."""
    rng = np.random.default_rng(r + e)
    ex = rng.integers(0, min(e, 5), r)
    at = rng.permutation(r)
    ex[at[:r // 3]] = 0
    if e > 2 and r >= 40:
        ex[ex == 1] = 2
        ex[at[r // 3:r // 3 + 16]] = 1
    ex[at[-1]] = e - 1
    if skip:
        ex[at[-4:-1]] = [-1, e, -2**31]
    return ex.astype(np.int32)


def _shape(name, group, scale_dtype, glu):
    r, e, k, n, n_glu, form = SHAPES[name]
    k, n = k[group], n_glu if glu else n
    assert form_of(r, e, k, n, group, 2 if scale_dtype == BF16 else 4, glu) == form
    return r, e, k, n


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_each_form(name, glu, group, affine, scale_dtype):
    r, e, k, n = _shape(name, group, scale_dtype, glu)
    case = _case(r, e, k, n, group, affine, scale_dtype, glu, experts=_experts(r, e))
    for out_dtype in (BF16, F32):
        y = torch.full((r, n), 7.0, dtype=out_dtype, device=DEV)
        _call(case, scale_dtype, out_dtype, y=y)
        _check(y, case, out_dtype)
        none = (case[1] < 0) | (case[1] >= e)
        assert none.sum() == 3 and (y[to_dev(none)] == 7).all()


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
@pytest.mark.parametrize("name", SHAPES)
def test_exact_sums(name, group, affine, scale_dtype):
    r, e, k, n = _shape(name, group, scale_dtype, False)
    case = exact_case(r, e, k, n, group, affine, experts=_experts(r, e, skip=False))
    got = to_np(_call(case, scale_dtype, F32))
    assert np.array_equal(got, product(*case[:2], *case[2])[0].astype(np.float32))


def _rms(v):
    return np.sqrt(np.mean(np.square(v)))


def _rms_limit(x, ex, codes, scales, biases):
    group = 2 * codes.shape[-1] // scales.shape[-1]
    lim = np.zeros((x.shape[0], codes.shape[1]))
    chain = 2 * U * 33 * (group // 32)
    for e in np.unique(ex):
        sel = ex == e
        sq = np.square(x[sel].astype(np.float64))
        q2 = np.square(unpack(codes[e]).astype(np.float64))
        groups = sq.reshape(sel.sum(), -1, group)
        qx = np.einsum("rgk,ngk->rng", groups, q2.reshape(q2.shape[0], -1, group), optimize=True)
        xx = groups.sum(2)[:, None, :]
        s = scales[e].astype(np.float64)
        if biases is None:
            part = 2 * chain * np.sqrt(qx + 64 * xx) * s
            whole = np.sqrt(((qx + 64 * xx) * s * s).sum(2))
        else:
            b = np.abs(biases[e].astype(np.float64))
            part = chain * (np.sqrt(qx) * s + np.sqrt(xx) * b)
            whole = np.sqrt(2 * (qx * s * s + xx * b * b).sum(2))
        lim[sel] = part.sum(2) + (10 * s.shape[1] + 14) * U * whole
    return lim


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
@pytest.mark.parametrize("name", SHAPES)
def test_mean_square_error(name, group, affine, scale_dtype):
    r, e, k, n = _shape(name, group, scale_dtype, False)
    case = _case(r, e, k, n, group, affine, scale_dtype, experts=_experts(r, e, skip=False))
    y, _ = product(*case[:2], *case[2])
    err = to_np(_call(case, scale_dtype, F32)).astype(np.float64) - y
    assert _rms(err) <= _rms(_rms_limit(*case[:2], *case[2])) + U * _rms(y)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_nan_and_infinity_stay(name, affine):
    for group in (32, 64, 128):
        r, e, k, n = _shape(name, group, BF16, False)
        case = _case(r, e, k, n, group, affine, BF16, experts=_experts(r, e, skip=False))
        clean = _call(case, BF16, F32)
        x = case[0].copy()
        x[2, 3], x[5, -1] = np.nan, np.inf
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


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_infinite_scales_and_biases_stay_in_their_column(name, affine):
    r, e, k, n = _shape(name, 128, BF16, False)
    case = _case(r, e, k, n, 128, affine, BF16, experts=_experts(r, e, skip=False))
    clean = _call(case, BF16, F32)
    hit = torch.zeros((r, n), dtype=torch.bool, device=DEV)
    hit[to_dev(case[1] == 0), 7] = True
    for part in (1, 2) if affine else (1,):
        for group in (0, -1):
            w = [v if v is None else v.copy() for v in case[2]]
            w[part][0, 7, group] = np.inf
            got = _call((case[0], case[1], tuple(w), None), BF16, F32)
            assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_replayed_and_on_two_streams(name, glu):
    """A captured call on rows and ids that change, and two calls at once on two streams."""
    r, e, k, n = _shape(name, 64, BF16, glu)
    case = _case(r, e, k, n, 64, True, BF16, glu, experts=_experts(r, e))
    w, up = _dev(case[2], BF16), _dev(case[3], BF16) if glu else (None,) * 3
    x, ex = to_dev(_bits(case[0])), to_dev(case[1])
    ws = torch.empty(moe.moe_gather_gemm_int4_workspace_bytes(r, e), dtype=torch.uint8, device=DEV)
    y = torch.full((r, n), 7.0, dtype=BF16, device=DEV)

    def call(x, ex, y, **kw):
        moe.moe_gather_gemm_int4(x, ex, *w, w_up=up[0], w_up_scales=up[1], w_up_biases=up[2], y=y, **kw)
    call(x, ex, y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, ex, y, workspace=ws)
    for rep in range(3):
        x.copy_(torch.roll(x, 1, 0))
        ex.copy_(torch.roll(ex, 2, 0))
        y.fill_(7)
        ws.fill_(255)
        g.replay()
        got = y.clone()
        y.fill_(7)
        call(x, ex, y, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, y), rep
    other = torch.flip(x, (0,)).contiguous()
    want = torch.full_like(y, 7)
    call(other, ex, want)
    outs = [torch.full_like(y, 7) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, rows, out in zip(streams, (x, other), outs):
            call(rows, ex, out, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], y) and torch.equal(outs[1], want)
