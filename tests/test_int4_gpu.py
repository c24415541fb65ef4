"""4-bit integer quantisation and expert products against the oracle.

Quantisation: codes, scales and biases bit for bit.  Values: the fused step in
fp32 errs by half a step of the value and of the result's type.

Products, u = 2^-24.  A group's sum is up to 8 matrix instructions (4 over the
constant, 4 over the codes) of 32 products, exact in fp32, and the running sum;
each of those 33 additions may err by a whole step (2 u) of the largest partial
sum, which the oracle's bound covers (23 s sum |x| a group, |b| sum |x| beside it):
8 * 33 * 2 u.  Scaling and adding the groups takes two roundings a group, the four
parts of K three more:
    |got - exact| <= h |exact| + (528 + 2 K / G + 6) u bound,   h = 2^-8 or 2^-24.
With the up projection, |silu'| <= 1.1 and silu itself within 2^-20 (bf16) or
2^-21 (fp32: an exponential within 2 u, two more roundings):
    (h + 2^-20) |silu(g) u| + 1.1 err_g |u| + err_u |silu(g)| + 1.1 err_g err_u.
A piece of 8 products that is missing is a 16th of a group's sum of |x| or more.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle import codecs
from oracle.int4 import dequantize, product, quantize, silu
from tests.gpu_util import DEV, as_f32, to_dev, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def _bits(x):
    return codecs.f32_to_bf16_bits(np.ascontiguousarray(x, np.float32))


def _same_floats(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


# ------------------------------------------------------------ quantisation

def _same_quantize(x, dtype, group, affine, scale_dtype):
    """x float32 [R, K], exactly representable in dtype."""
    xd = to_dev(_bits(x) if dtype == BF16 else np.ascontiguousarray(x, np.float32))
    c, s, b = moe.moe_quantize_int4(xd, group, affine=affine, scale_dtype=scale_dtype)
    wc, ws, wb = quantize(x, group, affine, scale_dtype == BF16)
    _same_floats(as_f32(to_np(s)), ws)
    if affine:
        _same_floats(as_f32(to_np(b)), wb)
    else:
        assert b is None
    assert np.array_equal(to_np(c), wc)
    want = dequantize(wc, ws, wb)
    ok = ~np.isnan(want)
    for dt, h, top in ((BF16, 2.0 ** -8, (2 - 2.0 ** -8) * 2.0 ** 127), (F32, 0.0, (2 - 2.0 ** -24) * 2.0 ** 127)):
        got = as_f32(to_np(moe.moe_dequant_int4(c, s, b, out_dtype=dt))).astype(np.float64)
        assert np.array_equal(np.isnan(got), ~ok)
        # from half a step past the type's largest number on, the rounded value is infinite
        over = ok & (np.abs(want) >= top)
        assert np.isinf(got[over]).all()
        fits = ok & ~over
        err = np.abs(got[fits] - want[fits])
        assert (err <= (h + U) * np.abs(want[fits]) * (1 + 2.0 ** -8) + 2.0 ** -133).all()


FORMS = [(g, a, s) for g in (32, 64, 128) for a in (False, True) for s in (BF16, F32)]


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_normal(dtype, group, affine, scale_dtype):
    rng = np.random.default_rng(group)
    for r, k in ((1, group), (3, 2 * group), (17, 5 * group), (130, 1024), (1000, group)):
        x = (rng.standard_normal((r, k)) * np.exp2(rng.integers(-20, 20, (r, 1)))).astype(np.float32)
        if affine:
            x += rng.standard_normal((r, 1)).astype(np.float32)
        if dtype == BF16:
            x = codecs.bf16_bits_to_f32(_bits(x))
        x[0, :group] = 0.0
        x[-1, -group:] = -0.0
        x[r // 2, :group] = 2.75
        _same_quantize(x, dtype, group, affine, scale_dtype)


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
def test_quantize_ties_and_neighbours(group, affine, scale_dtype):
    """Quotients at every half integer and one fp32 step beside it, for many scales."""
    rng = np.random.default_rng(group + 1)
    rows = []
    for _ in range(300):
        s = np.float32(_one(rng, scale_dtype))
        halves = (rng.integers(0, 15, group) + 0.5 if affine else rng.integers(-7, 7, group) + 0.5).astype(np.float32)
        v = halves * s                                       # a tie where this is exact
        v = np.where(rng.random(group) < 0.5, v, np.nextafter(v, rng.choice([-9e9, 9e9], group).astype(np.float32)))
        v = v.astype(np.float32)
        v[0] = s * np.float32(15 if affine else 7)
        if affine:
            v[1] = 0.0
        rows.append(v)
    x = np.concatenate(rows).reshape(100, 3 * group)
    _same_quantize(x, F32, group, affine, scale_dtype)
    _same_quantize(codecs.bf16_bits_to_f32(_bits(x)), BF16, group, affine, scale_dtype)


def test_quantize_every_bf16_quotient():
    """Every mantissa of the largest magnitude, which fixes the scale, and every bf16
    number from it down to where all codes are 8, both signs, at several exponents."""
    for group, p in ((32, 0), (64, -40), (128, 90), (128, -99), (128, -101), (128, -121)):
        rows = []
        for m in range(128, 256):
            top = (np.uint32(m - 128) | np.uint32((p + 127) << 7)).astype(np.uint16)
            low = max(int(top) - 6 * 128, 0)
            v = np.arange(low, int(top) + 1).astype(np.uint16)
            v = np.concatenate([v, v | np.uint16(0x8000)])
            v = np.resize(v, (v.size + group - 2) // (group - 1) * (group - 1)).reshape(-1, group - 1)
            rows.append(np.concatenate([np.full((len(v), 1), top, np.uint16), v], 1))
        x = codecs.bf16_bits_to_f32(np.concatenate(rows))
        _same_quantize(x, BF16, group, False, BF16)


def _one(rng, scale_dtype):
    v = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-60, 60))
    return codecs.bf16_bits_to_f32(_bits(v.reshape(1)))[0] if scale_dtype == BF16 else v


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
def test_quantize_ends_of_the_range(group, affine, scale_dtype):
    rng = np.random.default_rng(group + 2)
    for p in (-149, -140, -133, -128, -127, -126, -125, -110, -101, -99, 100, 124, 127):
        x = np.ldexp(rng.uniform(-1.9, 1.9, (20, 2 * group)), p).astype(np.float32)
        _same_quantize(x, F32, group, affine, scale_dtype)
        _same_quantize(codecs.bf16_bits_to_f32(_bits(x) & np.uint16(0xFFF0)), BF16, group, affine, scale_dtype)
    x = rng.standard_normal((6, 3 * group)).astype(np.float32)
    x[0, 1], x[1, group + 2], x[2, 3 * group - 1] = np.nan, np.inf, -np.inf
    x[3, 0], x[3, 1] = 3e38, -3e38                           # the range overflows: affine only
    x[4, :group] = np.float32(np.finfo(np.float32).min)      # as a bf16 bias: infinite
    _same_quantize(x, F32, group, affine, scale_dtype)
    if scale_dtype == F32:
        x[4, :group] = -3e38
        _same_quantize(codecs.bf16_bits_to_f32(_bits(x)), BF16, group, affine, scale_dtype)


def test_dequant_every_code():
    codes = np.tile(np.arange(256, dtype=np.uint8), (3, 1))                  # K = 512
    rng = np.random.default_rng(0)
    for group in (32, 64, 128):
        s = rng.standard_normal((3, 512 // group)).astype(np.float32)
        b = rng.standard_normal((3, 512 // group)).astype(np.float32)
        for bias in (None, b):
            got = to_np(moe.moe_dequant_int4(to_dev(codes), to_dev(s), None if bias is None else to_dev(b), out_dtype=F32))
            want = dequantize(codes, s, bias)
            assert (np.abs(got - want) <= U * np.abs(want)).all()


# ------------------------------------------------------------ products

def _weights(rng, e, n, k, group, affine, scale_dtype):
    codes = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    s = (rng.uniform(0.5, 2.0, (e, n, k // group)) * 0.01).astype(np.float32)
    b = rng.standard_normal((e, n, k // group)).astype(np.float32) * np.float32(0.05) if affine else None
    if scale_dtype == BF16:
        s = codecs.bf16_bits_to_f32(_bits(s))
        b = codecs.bf16_bits_to_f32(_bits(b)) if affine else None
    return codes, s, b


def _dev(w, scale_dtype):
    put = lambda v: None if v is None else to_dev(_bits(v) if scale_dtype == BF16 else v)
    return to_dev(w[0]), put(w[1]), put(w[2])


def _case(r, e, k, n, group, affine=False, scale_dtype=BF16, glu=False, seed=0, experts=None):
    rng = np.random.default_rng(seed + r + e + k + n)
    x = codecs.bf16_bits_to_f32(_bits(rng.standard_normal((r, k))))
    ex = rng.integers(0, e, r).astype(np.int32) if experts is None else np.asarray(experts, np.int32)
    w = _weights(rng, e, n, k, group, affine, scale_dtype)
    up = _weights(rng, e, n, k, group, affine, scale_dtype) if glu else None
    return x, ex, w, up


def _call(case, scale_dtype, out_dtype, **kw):
    x, ex, w, up = case
    u = _dev(up, scale_dtype) if up is not None else (None, None, None)
    return moe.moe_gather_gemm_int4(to_dev(_bits(x)), to_dev(ex), *_dev(w, scale_dtype), w_up=u[0], w_up_scales=u[1],
                                    w_up_biases=u[2], out_dtype=out_dtype, **kw)


def _check(got, case, out_dtype):
    x, ex, w, up = case
    ok = np.nonzero((ex >= 0) & (ex < w[0].shape[0]))[0]
    h = 2.0 ** -8 if out_dtype == BF16 else U
    k, groups = x.shape[1], w[1].shape[-1]
    c = (528 + 2 * groups + 6) * U
    y, bound = product(x[ok], ex[ok], *w)
    err = c * bound
    if up is None:
        lim = h * np.abs(y) + err * (1 + h)
    else:
        u, ub = product(x[ok], ex[ok], *up)
        s, eu = silu(y), c * ub
        lim = ((h + 2.0 ** -20) * np.abs(s * u) + (1.1 * err * np.abs(u) + eu * np.abs(s) + 1.1 * err * eu) * (1 + h))
        y = s * u
    g = as_f32(to_np(got)).astype(np.float64)[ok]
    bad = ~(np.abs(g - y) <= lim + 2.0 ** -126)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], np.max(np.abs(g - y) - lim))


@pytest.mark.parametrize("group,affine,scale_dtype", FORMS)
@pytest.mark.parametrize("glu", [False, True])
def test_products_of_each_form(group, affine, scale_dtype, glu):
    for out_dtype in (BF16, F32):
        for r, e, k, n in ((1, 1, 128, 64), (5, 3, 384, 100), (40, 8, 1152, 33), (100, 4, 640, 70)):
            case = _case(r, e, k, n, group, affine, scale_dtype, glu)
            _check(_call(case, scale_dtype, out_dtype), case, out_dtype)


@pytest.mark.parametrize("r,e", [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (33, 1), (64, 1), (65, 1), (200, 1), (64, 64),
                                 (63, 5), (65, 70), (300, 7), (1000, 300), (129, 1024)])
@pytest.mark.parametrize("glu", [False, True])
def test_products_over_rows(r, e, glu):
    case = _case(r, e, 256, 36, 64, False, BF16, glu)
    _check(_call(case, BF16, BF16), case, BF16)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 31, 32, 63, 65, 127, 129, 258])
def test_products_over_columns(n, group):
    for glu in (False, True):
        for out_dtype in (BF16, F32):
            case = _case(20, 2, 512, n, group, True, F32, glu)
            _check(_call(case, F32, out_dtype), case, out_dtype)


@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 224, 256, 288, 480, 512, 544, 800, 1024, 1056, 2080, 4000])
@pytest.mark.parametrize("r", [3, 60])
def test_products_over_k(k, r):
    for affine in (False, True):
        case = _case(r, 2, k, 40, 32, affine, BF16)
        _check(_call(case, BF16, F32), case, F32)
    if k % 64 == 0:
        case = _case(r, 2, k, 40, 64, False, F32)
        _check(_call(case, F32, BF16), case, BF16)
    if k % 128 == 0:
        case = _case(r, 2, k, 40, 128, True, BF16, glu=True)
        _check(_call(case, BF16, BF16), case, BF16)


def test_products_decode_layer_size():
    """One layer's worth of experts at decode; the columns of a few rows are checked."""
    r, e, k, n = 256, 32, 7168, 2048
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.randn((r, k), generator=g, device=DEV).to(BF16)
    ex = torch.randint(0, e, (r,), generator=g, device=DEV, dtype=torch.int32)
    ws = [moe.moe_quantize_int4((torch.randn((e * n, k), generator=g, device=DEV) * 0.02).to(BF16)) for _ in range(2)]
    (wc, wsc, _), (uc, usc, _) = [(c.view(e, n, -1), s.view(e, n, -1), b) for c, s, b in ws]
    y = moe.moe_gather_gemm_int4(x, ex, wc, wsc, w_up=uc, w_up_scales=usc)
    pick = [0, 100, 255]
    hx, hex_ = as_f32(to_np(x[pick])), to_np(ex[pick])
    hw, hu = [(to_np(c[ex[pick].long()]), as_f32(to_np(s[ex[pick].long()])), None) for c, s in ((wc, wsc), (uc, usc))]
    _check(y[pick], (hx, np.arange(3), hw, hu), BF16)
    # the whole against one row at a time, which groups nothing
    for i in (1, 37):
        one = moe.moe_gather_gemm_int4(x[i:i + 1], ex[i:i + 1], wc, wsc, w_up=uc, w_up_scales=usc)
        assert torch.allclose(one.float(), y[i:i + 1].float(), rtol=2.0 ** -7, atol=1e-5)


@pytest.mark.parametrize("r", [12, 90])
def test_rows_without_an_expert_stay(r):
    ex = np.arange(r) % 3
    ex[::4], ex[1::5], ex[2::7] = -1, 3, -2**31
    case = _case(r, 3, 256, 48, 64, experts=ex)
    for dt in (BF16, F32):
        y = torch.full((r, 48), 7.0, dtype=dt, device=DEV)
        _call(case, BF16, dt, y=y)
        _check(y, case, dt)
        skip = (case[1] < 0) | (case[1] >= 3)
        assert (y[to_dev(skip)] == 7).all()
    # none at all
    none = (case[0], np.full(r, -1, np.int32), *case[2:])
    y = torch.full((r, 48), 7.0, dtype=BF16, device=DEV)
    _call(none, BF16, BF16, y=y)
    assert (y == 7).all()


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("r", [10, 70])
def test_nan_and_infinity_stay_in_their_row_and_column(r, affine):
    for group in (32, 128):
        case = _case(r, 2, 384, 50, group, affine, BF16)
        clean = _call(case, BF16, F32)
        x = case[0].copy()
        x[2, 3], x[5, 383] = np.nan, np.inf
        got = _call((x, *case[1:]), BF16, F32)
        rows = torch.ones(r, dtype=torch.bool, device=DEV)
        rows[[2, 5]] = False
        assert not torch.isfinite(got[~rows]).any() and torch.equal(got[rows], clean[rows])
        s = case[2][1].copy()
        s[0, 7, -1] = np.nan
        got = _call((case[0], case[1], (case[2][0], s, case[2][2]), None), BF16, F32)
        hit = torch.zeros((r, 50), dtype=torch.bool, device=DEV)
        hit[to_dev(case[1] == 0), 7] = True
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


def test_exact_where_sums_are():
    """Small integers and power-of-two scales: every partial sum is an fp32 number."""
    rng = np.random.default_rng(5)
    for group in (32, 64, 128):
        x = rng.integers(-8, 9, (20, 512)).astype(np.float32)
        w = (rng.integers(0, 256, (2, 40, 256), dtype=np.uint8),
             np.exp2(rng.integers(-3, 3, (2, 40, 512 // group))).astype(np.float32), None)
        ex = rng.integers(0, 2, 20).astype(np.int32)
        for biases in (None, rng.integers(-8, 9, w[1].shape).astype(np.float32)):
            case = (x, ex, (w[0], w[1], biases), None)
            assert np.array_equal(to_np(_call(case, F32, F32)), product(x, ex, w[0], w[1], biases)[0].astype(np.float32))


def test_every_code_at_every_place():
    """One code at a time against rows that are 1 at one place: w itself comes out."""
    k, n = 128, 16
    x = np.eye(128, dtype=np.float32)
    codes = np.empty((1, n, k // 2), np.uint8)
    for q in range(n):
        codes[0, q] = q | (((q + 5) % 16) << 4)
    for group in (32, 64, 128):
        s = np.exp2(np.arange(n * (k // group)).reshape(1, n, -1) % 5).astype(np.float32)
        case = (x, np.zeros(128, np.int32), (codes, s, None), None)
        assert np.array_equal(to_np(_call(case, F32, F32)), dequantize(codes, s)[0].T.astype(np.float32))


def test_repeatable_and_row_order():
    """The same bits on every call, and rows moved with their experts keep their results
    (a row's sum does not depend on the others)."""
    case = _case(200, 5, 768, 96, 64, True, BF16, True)
    a = _call(case, BF16, BF16)
    assert torch.equal(a, _call(case, BF16, BF16))
    perm = np.random.default_rng(0).permutation(200)
    b = _call((case[0][perm], case[1][perm], *case[2:]), BF16, BF16)
    assert torch.equal(b, a[to_dev(perm)])


def test_outputs_end_where_they_should():
    for r, n in ((3, 5), (70, 37)):
        for dt in (BF16, F32):
            case = _case(r, 2, 256, n, 64)
            flat = torch.full((r * n + 64,), 7.0, dtype=dt, device=DEV)
            y = flat[:r * n].view(r, n)
            _call(case, BF16, dt, y=y)
            _check(y, case, dt)
            assert (flat[r * n:] == 7).all()


def test_graph_replays_and_shared_workspace():
    """Two captured products that share a workspace, on rows that change between replays."""
    ws = torch.empty(moe.moe_gather_gemm_int4_workspace_bytes(300, 7), dtype=torch.uint8, device=DEV)
    steps = []
    for r, glu in ((300, True), (8, False)):
        case = _case(r, 7, 256, 64, 64, False, BF16, glu)
        w, up = _dev(case[2], BF16), _dev(case[3], BF16) if glu else (None,) * 3
        x, ex, y = to_dev(_bits(case[0])), to_dev(case[1]), torch.empty((r, 64), dtype=BF16, device=DEV)
        steps.append((x, y, ex, lambda x=x, ex=ex, w=w, up=up, y=y: moe.moe_gather_gemm_int4(
            x, ex, *w, w_up=up[0], w_up_scales=up[1], w_up_biases=up[2], y=y, workspace=ws)))
    graphs = []
    for x, y, ex, step in steps:
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for rep in range(4):
        for (x, y, ex, step), g in zip(steps, graphs):
            x.copy_(torch.roll(x, 1, 0))
            ex.copy_((ex + 1) % 7)
            y.fill_(7)
            ws.fill_(255)
            g.replay()
            got = y.clone()
            torch.cuda.synchronize()
            step()
            assert torch.equal(got, y), rep


def test_on_another_stream():
    case = _case(150, 4, 512, 80, 128, False, BF16, True)
    want = _call(case, BF16, BF16)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    w, up, x, ex = _dev(case[2], BF16), _dev(case[3], BF16), to_dev(_bits(case[0])), to_dev(case[1])
    torch.cuda.synchronize()
    for _ in range(3):
        got = moe.moe_gather_gemm_int4(x, ex, *w, w_up=up[0], w_up_scales=up[1], stream=st)
        c, s, b = moe.moe_quantize_int4(x, 64, affine=True, stream=st)
        v = moe.moe_dequant_int4(c, s, b, stream=st)
        st.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(v, moe.moe_dequant_int4(*moe.moe_quantize_int4(x, 64, affine=True)))


def test_no_rows():
    w = _dev(_weights(np.random.default_rng(0), 2, 8, 64, 64, False, BF16), BF16)
    y = moe.moe_gather_gemm_int4(torch.empty((0, 64), dtype=BF16, device=DEV),
                                 torch.empty(0, dtype=torch.int32, device=DEV), *w)
    assert y.shape == (0, 8)
    c, s, b = moe.moe_quantize_int4(torch.empty((0, 64), device=DEV), 32, affine=True)
    assert c.shape == (0, 32) and s.shape == b.shape == (0, 2)
    assert moe.moe_dequant_int4(c, s, b).shape == (0, 64)


def test_refusals():
    x = torch.zeros((4, 256), dtype=BF16, device=DEV)
    ex = torch.zeros(4, dtype=torch.int32, device=DEV)
    w, s, _ = moe.moe_quantize_int4(torch.zeros((16, 256), dtype=BF16, device=DEV), 64)
    w, s = w.view(2, 8, 128), s.view(2, 8, 4)
    f = lambda **kw: moe.moe_gather_gemm_int4(**{**dict(rows=x, row_expert=ex, w=w, w_scales=s), **kw})
    f()
    with pytest.raises(TypeError, match="rows"):
        f(rows=x.float())
    with pytest.raises(ValueError, match="rows must be"):
        f(rows=x[:, :128].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        f(rows=x[:, ::2])
    with pytest.raises(TypeError, match="row_expert"):
        f(row_expert=ex.long())
    with pytest.raises(ValueError, match="row_expert"):
        f(row_expert=ex[:3])
    with pytest.raises(ValueError, match="groups must hold"):
        f(w_scales=s[:, :, :1].contiguous())                 # groups of 256
    with pytest.raises(ValueError, match="groups must hold"):
        f(w_scales=s[:, :, :3].contiguous())
    with pytest.raises(TypeError, match="w_scales"):
        f(w_scales=s.half())
    with pytest.raises(TypeError, match="w_biases"):
        f(w_biases=s.float())
    with pytest.raises(ValueError, match="go together"):
        f(w_up=w)
    with pytest.raises(ValueError, match="go together"):
        f(w_up=w, w_up_scales=s, w_biases=s)
    with pytest.raises(ValueError, match="w_up_biases"):
        f(w_up_biases=s, w_biases=s)
    with pytest.raises(TypeError, match="w_up_scales"):
        f(w_up=w, w_up_scales=s.float())
    with pytest.raises(ValueError, match="w_up"):
        f(w_up=w[:1], w_up_scales=s[:1])
    with pytest.raises(TypeError, match="out_dtype"):
        f(out_dtype=torch.float16)
    with pytest.raises(ValueError, match="y"):
        f(y=torch.empty((4, 7), dtype=BF16, device=DEV))
    with pytest.raises(moe.MoeError, match="MOE_ERR_WORKSPACE"):
        f(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    for kw, err, match in ((dict(group=16), ValueError, "group"), (dict(scale_dtype=torch.float16), TypeError, "scale_dtype"),
                           (dict(scales=torch.empty((4, 3), device=DEV)), ValueError, "scales"),
                           (dict(biases=torch.empty((4, 2), device=DEV)), TypeError, "biases")):
        with pytest.raises(err, match=match):
            moe.moe_quantize_int4(x, **kw)
    with pytest.raises(ValueError, match="x must be"):
        moe.moe_quantize_int4(x[:, :96].contiguous(), 64)
    with pytest.raises(TypeError, match="out_dtype"):
        moe.moe_dequant_int4(w[0], s[0], out_dtype=torch.float16)


def test_a_layer_with_integer_experts():
    """Routing, its balance losses, dispatch, both products, combine, and the router's
    whole gradient, as a program runs them."""
    n, e, k, d, f = 50, 8, 2, 256, 128
    rng = np.random.default_rng(11)
    logits, x = rng.standard_normal((n, e)).astype(np.float32), _bits(rng.standard_normal((n, d)))
    ws = []
    for rows, cols in ((f, d), (f, d), (d, f)):
        wf = codecs.bf16_bits_to_f32(_bits(rng.standard_normal((e * rows, cols)) * cols ** -0.5))
        c, s, _ = moe.moe_quantize_int4(to_dev(_bits(wf)), 64)
        ws.append((c.view(e, rows, -1), s.view(e, rows, -1)))
    ld, xd = to_dev(logits), to_dev(x)
    idx, w = moe.moe_route_topk(ld, k)
    bal = moe.moe_balance_loss(ld, idx)
    disp = moe.moe_dispatch(xd, idx, e, sort=0)
    assert torch.equal(bal.counts[0], disp.expert_counts)
    h = moe.moe_gather_gemm_int4(disp.rows, disp.row_expert, *ws[0], w_up=ws[1][0], w_up_scales=ws[1][1])
    y = moe.moe_gather_gemm_int4(h, disp.row_expert, *ws[2], out_dtype=F32)
    out = moe.moe_combine(y, disp.dst_pos, w)

    host = [(to_np(c), as_f32(to_np(s))) for c, s in ws]
    xr, ex = as_f32(to_np(disp.rows)), to_np(disp.row_expert)
    g, u = (product(xr, ex, *host[i])[0] for i in (0, 1))
    _check(h, (xr, ex, (*host[0], None), (*host[1], None)), BF16)
    _check(y, (as_f32(to_np(h)), ex, (*host[2], None), None), F32)
    yw = product(as_f32(to_np(h)), ex, *host[2])[0]
    want = np.zeros((n, d))
    pos, wt = to_np(disp.dst_pos).reshape(n, k), to_np(w).astype(np.float64)
    for j in range(k):
        want += wt[:, j:j + 1] * yw[pos[:, j]]
    assert np.allclose(to_np(out), want, rtol=1e-4, atol=1e-4)

    d_w = to_dev(rng.standard_normal((n, k)).astype(np.float32))
    one = torch.full((1,), 0.01, device=DEV)
    d_logits = moe.moe_route_topk_backward(idx, w, d_w, e)
    alone = d_logits.clone()
    moe.moe_balance_loss_backward(ld, bal.counts, bal.tokens, k, one, one, d_logits=d_logits, accumulate=True)
    assert torch.equal(d_logits, alone + moe.moe_balance_loss_backward(ld, bal.counts, bal.tokens, k, one, one))
