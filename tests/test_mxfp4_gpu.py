"""MXFP4 quantisation and expert products against the oracle.

Quantisation and dequantisation are exact: codes, scales and values are
compared bit for bit.

Products.  The oracle's value is float64.  E2M1 products are exact and a block's
sum fits 13 bits, so what rounds is the accumulation over the K/32 blocks and
the result: the sibling fp8 matrix instructions accumulate to about 2^-14 of
their largest outputs, and 8 times that is allowed here as there:
    |got - exact| <= 2^-8 |exact| + 2^-11 magnitude
with 2^-8 the bf16 rounding and the magnitude the sum of the terms' absolute
values.  One missing block out of K/32, or a scale off by one, is 2^-5 of the
magnitude or more at the sizes here.  Where every partial sum is an exact fp32
number the result has to be the correctly rounded one
(test_products_exact_where_sums_are).  With the up projection, |silu'| <= 1.1:
    |got - silu(g) u| <= (2^-8 + 2^-20) |silu(g) u| + 2^-11 (1.1 mag_g |u| + mag_u |silu(g)|) + 2^-22 mag_g mag_u
the last term being the product of both errors.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle import codecs
from oracle.mxfp4 import dequantize, product, quantize, silu
from tests.gpu_util import DEV, as_f32, to_dev, to_np

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ quantisation

def _same_quantize(x, dtype):
    """x float32 [R, K], exactly representable in dtype."""
    xd = to_dev(codecs.f32_to_bf16_bits(x) if dtype == "bf16" else x)
    c, s = moe.moe_quantize_mxfp4(xd)
    wc, ws = quantize(x)
    assert np.array_equal(to_np(s), ws)
    assert np.array_equal(to_np(c), wc)
    for dt in (torch.bfloat16, torch.float32):
        got = as_f32(to_np(moe.moe_dequant_mxfp4(c, s, out_dtype=dt))).astype(np.float64)
        want = dequantize(wc, ws)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("r,k", [(1, 32), (3, 64), (1, 4096 + 32), (17, 96), (130, 7168), (4, 8192), (1000, 160)])
def test_quantize_normal(dtype, r, k):
    rng = np.random.default_rng(r + k)
    x = (rng.standard_normal((r, k)) * np.exp2(rng.integers(-8, 8, (r, 1)))).astype(np.float32)
    if dtype == "bf16":
        x = codecs.bf16_bits_to_f32(codecs.f32_to_bf16_bits(x))
    x[0, :32] = 0.0
    x[-1, -32:] = -0.0
    _same_quantize(x, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_beyond_the_cache(dtype):
    """More than 256 MB of x are loaded another way: the same codes as of its parts."""
    r, k = (4100, 32768) if dtype == torch.bfloat16 else (4100, 16416)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn((r, k), generator=g, device=DEV).to(dtype)
    c, s = moe.moe_quantize_mxfp4(x)
    for lo, hi in ((0, 2000), (2000, 4100)):
        pc, ps = moe.moe_quantize_mxfp4(x[lo:hi])
        assert torch.equal(c[lo:hi], pc) and torch.equal(s[lo:hi], ps)
    rows = [0, 1999, 4099]
    wc, ws = quantize(x[rows].float().cpu().numpy())
    assert np.array_equal(to_np(c[rows]), wc) and np.array_equal(to_np(s[rows]), ws)


def test_quantize_every_bf16_pattern():
    """Each finite bf16 value as the largest of a block with random smaller
    ones, and within a block of a random larger one."""
    rng = np.random.default_rng(1)
    bits = np.arange(65536, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    top = codecs.bf16_bits_to_f32(bits)
    frac = rng.uniform(-1, 1, (top.size, 32)).astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        x = codecs.bf16_bits_to_f32(codecs.f32_to_bf16_bits(frac * np.abs(top[:, None])))
        x[:, 5] = top
        _same_quantize(x, "bf16")
        big = np.minimum(np.abs(top) * np.exp2(rng.integers(0, 5, top.size)), 3e38).astype(np.float32)
        x[:, 9] = codecs.bf16_bits_to_f32(codecs.f32_to_bf16_bits(big))
        x[~np.isfinite(x)] = 0.0
        _same_quantize(x, "bf16")


def test_quantize_midpoints_and_neighbours_in_f32():
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float32)
    vals = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    vals = np.concatenate([vals, -vals])
    for p in (-126, -125, -124, -60, 0, 60, 124):
        x = np.zeros((vals.size, 32), np.float32)
        x[:, 0] = np.float32(4.0 * 2.0 ** p)
        x[:, 31] = vals * np.float32(2.0) ** p
        _same_quantize(x, "f32")
    sub = np.zeros((200, 32), np.float32)
    sub[:, :] = np.random.default_rng(2).integers(0, 1 << 24, sub.shape).astype(np.uint32).view(np.float32)
    _same_quantize(sub, "f32")                                      # subnormals


def test_quantize_blocks_with_nan_or_infinity():
    x = np.ones((4, 96), np.float32)
    x[0, 40], x[1, 0], x[2, 95] = np.nan, np.inf, -np.inf
    for dtype in ("f32", "bf16"):
        _same_quantize(x, dtype)


def test_dequant_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))                 # K = 512: 16 blocks
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    for dt in (torch.float32, torch.bfloat16):
        got = as_f32(to_np(moe.moe_dequant_mxfp4(to_dev(codes), to_dev(scales), out_dtype=dt)))
        want = dequantize(codes, scales)
        with np.errstate(over="ignore"):
            want = want.astype(np.float32)                                    # 6 * 2^127 overflows to inf
        if dt == torch.bfloat16:
            want = codecs.bf16_bits_to_f32(codecs.f32_to_bf16_bits(want))
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


# ------------------------------------------------------------ products

def _operand(rng, *shape, spread=6):
    k = shape[-1]
    codes = rng.integers(0, 256, shape[:-1] + (k // 2,), dtype=np.uint8)
    scales = rng.integers(127 - spread, 128 + spread, shape[:-1] + (k // 32,), dtype=np.uint8)
    return codes, scales


def _check(got_bits, rows, rs, experts, w, up, what):
    got = codecs.bf16_bits_to_f32(got_bits).astype(np.float64)
    g, mg = product(rows, rs, experts, *w)
    if up is None:
        err, bound = np.abs(got - g), 2.0 ** -8 * np.abs(g) + 2.0 ** -11 * mg
    else:
        u, mu = product(rows, rs, experts, *up)
        want = silu(g) * u
        err = np.abs(got - want)
        bound = ((2.0 ** -8 + 2.0 ** -20) * np.abs(want) +
                 2.0 ** -11 * (1.1 * mg * np.abs(u) + mu * np.abs(silu(g))) + 2.0 ** -22 * mg * mu)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside the bound, worst {np.max(err / bound):.3g}x"


def _run(kind, rows, rs, ids, w, up, y=None):
    """ids: the expert of each row, for the grouped form in ascending order."""
    args = [to_dev(rows), to_dev(rs)]
    kw = dict(y=y)
    if up is not None:
        kw.update(w_up=to_dev(up[0]), w_up_scales=to_dev(up[1]))
    if kind == "gather":
        return moe.moe_gather_gemm_mxfp4(*args, to_dev(ids), to_dev(w[0]), to_dev(w[1]), **kw)
    offs = np.searchsorted(ids, np.arange(w[0].shape[0] + 1)).astype(np.int32)
    return moe.moe_grouped_gemm_mxfp4(*args, to_dev(offs), to_dev(w[0]), to_dev(w[1]), **kw)


# rows, experts, K, N: one row; empty experts; K of 1, 2, 3, 7 and many 128s;
# N below, at and past every tile; rows at and past every tile
SHAPES = [(1, 1, 128, 1), (1, 4, 128, 8), (2, 3, 256, 33), (31, 2, 384, 64), (32, 1, 896, 127),
          (33, 8, 128, 128), (65, 3, 512, 129), (64, 2, 1024, 256), (129, 2, 1152, 257), (257, 1, 2048, 264),
          (300, 5, 640, 520), (1000, 4, 768, 136), (40, 64, 256, 72), (5, 300, 128, 40), (1, 1024, 128, 16),
          (2050, 2, 384, 300)]


@pytest.mark.parametrize("kind", ["grouped", "gather"])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("r,e,k,n", SHAPES)
def test_products(kind, glu, r, e, k, n):
    rng = np.random.default_rng(r + 7 * e + k + n)
    rows, rs = _operand(rng, r, k)
    if glu:                                   # gates of moderate size, as a network has them
        rs = (rs - np.uint8(4)).astype(np.uint8)
    w = _operand(rng, e, n, k)
    w = (w[0], (w[1] - np.uint8(3)).astype(np.uint8)) if glu else w
    up = _operand(rng, e, n, k) if glu else None
    ids = rng.integers(0, e, r).astype(np.int32)
    if e > 2:
        ids[ids == 1] = 0                     # an expert without rows
    if kind == "grouped":
        ids = np.sort(ids)
    y = _run(kind, rows, rs, ids, w, up)
    assert tuple(y.shape) == (r, n)
    with np.errstate(over="ignore"):
        _check(to_np(y), rows, rs, ids, w, up, f"{kind} glu={glu} R={r} E={e} K={k} N={n}")


@pytest.mark.parametrize("kind", ["grouped", "gather"])
@pytest.mark.parametrize("r,e,k,n", [(70, 3, 256, 100), (600, 2, 1024, 300), (3, 2, 128, 20), (9, 4, 4096, 64)])
def test_products_exact_where_sums_are(kind, r, e, k, n):
    """With every scale 2^0 all sums are multiples of 1/4 below 36 K <= 2^18:
    exact in fp32, so y is the correctly rounded value, whatever the order."""
    rng = np.random.default_rng(k + n)
    rows, w = (rng.integers(0, 256, s, dtype=np.uint8) for s in ((r, k // 2), (e, n, k // 2)))
    rs, ws = (np.full(s, 127, np.uint8) for s in ((r, k // 32), (e, n, k // 32)))
    ids = rng.integers(0, e, r).astype(np.int32)
    if kind == "grouped":
        ids = np.sort(ids)
    y = _run(kind, rows, rs, ids, (w, ws), None)
    want, _ = product(rows, rs, ids, w, ws)
    assert np.array_equal(as_f32(to_np(y)), as_f32(codecs.f64_to_bf16_bits(want)))


@pytest.mark.parametrize("kind", ["grouped", "gather"])
@pytest.mark.parametrize("r,k", [(40, 1408), (40, 1536), (300, 1408), (300, 1536), (300, 2048)])
def test_each_block_takes_its_own_scales(kind, r, k):
    """Every block's scale is raised in one row and in one column, by 2^3 and 2^4:
    the outputs move by those blocks' shares alone."""
    n, e = 48, 2
    rows = np.full((r, k // 2), 0x22, np.uint8)                      # ones
    w = np.full((e, n, k // 2), 0x22, np.uint8)
    rs, ws = np.full((r, k // 32), 127, np.uint8), np.full((e, n, k // 32), 127, np.uint8)
    ids = np.sort(np.arange(r) % e).astype(np.int32)
    for b in range(k // 32):
        rs[b % r, b] += 3
        ws[b % e, (5 * b) % n, b] += 4
    y = _run(kind, rows, rs, ids, (w, ws), None)
    want, _ = product(rows, rs, ids, w, ws)
    assert np.array_equal(as_f32(to_np(y)), as_f32(codecs.f64_to_bf16_bits(want)))


@pytest.mark.parametrize("kind", ["grouped", "gather"])
@pytest.mark.parametrize("r,k", [(6, 256), (200, 256), (200, 384), (70, 1024), (200, 1024)])
def test_extreme_scales_and_nan_scales(kind, r, k):
    """Scale bytes 0 and 254 (their product is finite again); 255 makes a row or
    a column NaN and leaves the others."""
    e, n = 1, 40
    rows, w = np.full((r, k // 2), 0x22, np.uint8), np.full((e, n, k // 2), 0x22, np.uint8)
    rs, ws = np.full((r, k // 32), 0, np.uint8), np.full((e, n, k // 32), 254, np.uint8)
    rs[1, 3], ws[0, 7, 2] = 255, 255
    y = as_f32(to_np(_run(kind, rows, rs, np.zeros(r, np.int32), (w, ws), None)))
    assert np.isnan(y[1]).all() and np.isnan(y[:, 7]).all()
    rest = np.delete(np.delete(y, 1, 0), 7, 1)
    assert (rest == k).all()                                         # 2^-127 2^127 = 1


def test_rows_outside_the_offsets_and_bad_ids_stay():
    rng = np.random.default_rng(5)
    e, k, n = 2, 256, 72
    rows, rs = _operand(rng, 30, k)
    w = _operand(rng, e, n, k)
    y = torch.full((30, n), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_grouped_gemm_mxfp4(to_dev(rows), to_dev(rs), to_dev(np.array([2, 10, 20], np.int32)),
                               to_dev(w[0]), to_dev(w[1]), y=y)
    yy = as_f32(to_np(y))
    assert (yy[:2] == 7).all() and (yy[20:] == 7).all()
    _check(to_np(y)[2:20], rows[2:20], rs[2:20], np.repeat([0, 1], [8, 10]), w, None, "inside")
    # offsets outside the buffer are cut to it
    y.fill_(7.0)
    moe.moe_grouped_gemm_mxfp4(to_dev(rows), to_dev(rs), to_dev(np.array([-5, 10, 99], np.int32)),
                               to_dev(w[0]), to_dev(w[1]), y=y)
    _check(to_np(y), rows, rs, np.repeat([0, 1], [10, 20]), w, None, "cut")
    ids = rng.integers(0, e, 30).astype(np.int32)
    ids[[0, 7, 29]] = [-1, e, 2**31 - 1]
    y.fill_(7.0)
    moe.moe_gather_gemm_mxfp4(to_dev(rows), to_dev(rs), to_dev(ids), to_dev(w[0]), to_dev(w[1]), y=y)
    good = (ids >= 0) & (ids < e)
    assert (as_f32(to_np(y))[~good] == 7).all()
    _check(to_np(y)[good], rows[good], rs[good], ids[good], w, None, "good ids")
    y.fill_(7.0)                                                     # no row has an expert
    moe.moe_gather_gemm_mxfp4(to_dev(rows), to_dev(rs), torch.full((30,), -1, dtype=torch.int32, device=DEV),
                              to_dev(w[0]), to_dev(w[1]), y=y)
    assert bool((y == 7).all())


def test_zero_rows():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    c, s = moe.moe_quantize_mxfp4(torch.zeros((0, 64), device=DEV))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert moe.moe_dequant_mxfp4(c, s).shape == (0, 64)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    assert moe.moe_grouped_gemm_mxfp4(z(0, 64), z(0, 4), i32(3), z(2, 8, 64), z(2, 8, 4)).shape == (0, 8)
    assert moe.moe_gather_gemm_mxfp4(z(0, 64), z(0, 4), i32(0), z(2, 8, 64), z(2, 8, 4)).shape == (0, 8)


# tiles of up to 128, 192 and 256 rows; few of them in all (300 columns), none too
# few (4200) and never few (6600); every number of K stages modulo 4, whole or not
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("n", [300, 4200, 6600])
@pytest.mark.parametrize("k", [128, 384, 640, 1024, 1152, 1536, 2048, 2688])
def test_tiles_of_every_height(k, n, glu):
    rng = np.random.default_rng(k + n)
    counts = [1, 130, 192, 300, 0, 128, 193, 512 + 129]
    e, r = len(counts), sum(counts)
    rows, rs = _operand(rng, r, k)
    w = _operand(rng, e, n, k)
    up = _operand(rng, e, n, k) if glu else None
    if glu:
        rs, w = (rs - np.uint8(4)).astype(np.uint8), (w[0], (w[1] - np.uint8(3)).astype(np.uint8))
    ids = np.repeat(np.arange(e), counts).astype(np.int32)
    y = to_np(_run("grouped", rows, rs, ids, w, up))
    cols = np.unique(np.concatenate([np.arange(0, n, 61), np.arange(250, 260), np.arange(n - 70, n)]))
    at = lambda m: None if m is None else (m[0][:, cols], m[1][:, cols])
    with np.errstate(over="ignore"):
        _check(y[:, cols], rows, rs, ids, at(w), at(up), f"K={k} N={n} glu={glu}")


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("k,n", [(384, 300), (640, 4200), (1024, 300), (1152, 700), (2048, 6600)])
def test_many_rows_in_any_order(k, n, glu):
    """Rows of every tile height in shuffled order, some without an expert."""
    rng = np.random.default_rng(k + n + glu)
    ids = rng.permutation(np.repeat([0, 1, 2, 3, 5, 6, 7, -1, 8], [1, 130, 192, 300, 128, 193, 641, 20, 9])).astype(np.int32)
    e, r = 8, ids.size
    rows, rs = _operand(rng, r, k)
    w = _operand(rng, e, n, k)
    up = _operand(rng, e, n, k) if glu else None
    if glu:
        rs, w = (rs - np.uint8(4)).astype(np.uint8), (w[0], (w[1] - np.uint8(3)).astype(np.uint8))
    y = torch.full((r, n), 7.0, dtype=torch.bfloat16, device=DEV)
    _run("gather", rows, rs, ids, w, up, y=y)
    good = (ids >= 0) & (ids < e)
    assert (as_f32(to_np(y))[~good] == 7).all()
    cols = np.unique(np.concatenate([np.arange(0, n, 61), np.arange(250, 260), np.arange(n - 70, n)]))
    at = lambda m: None if m is None else (m[0][:, cols], m[1][:, cols])
    with np.errstate(over="ignore"):
        _check(to_np(y)[good][:, cols], rows[good], rs[good], ids[good], at(w), at(up), f"K={k} N={n} glu={glu}")


# at least 128 rows per expert: every number of 256-wide K stages modulo 4, with
# and without a half stage at the end, row and column counts off the tile
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("k", [128, 256, 384, 512, 640, 896, 1024, 1280, 1408, 1792, 2176, 4224])
def test_products_of_many_rows(k, glu):
    rng = np.random.default_rng(k)
    e, r, n = 3, 700, 300
    rows, rs = _operand(rng, r, k)
    w = _operand(rng, e, n, k)
    up = _operand(rng, e, n, k) if glu else None
    if glu:
        rs, w = (rs - np.uint8(4)).astype(np.uint8), (w[0], (w[1] - np.uint8(3)).astype(np.uint8))
    ids = np.sort(rng.choice(e, r, p=[0.5, 0.1, 0.4])).astype(np.int32)
    with np.errstate(over="ignore"):
        _check(to_np(_run("grouped", rows, rs, ids, w, up)), rows, rs, ids, w, up, f"K={k}")


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("r,e,k,n", [(64, 7, 512, 70), (64, 64, 128, 36), (64, 1024, 256, 20), (17, 2, 640, 129),
                                     (64, 40, 1152, 8), (65, 7, 512, 70)])
def test_gather_of_a_small_batch(r, e, k, n, glu):
    """Up to 64 rows are grouped inside the product's launch: repeated experts
    past a tile of 16, ids outside the range between them, all rows one expert."""
    rng = np.random.default_rng(r + e)
    rows, rs = _operand(rng, r, k)
    w, up = _operand(rng, e, n, k), _operand(rng, e, n, k) if glu else None
    if glu:
        rs, w = (rs - np.uint8(4)).astype(np.uint8), (w[0], (w[1] - np.uint8(3)).astype(np.uint8))
    for ids in (rng.integers(0, e, r), np.full(r, e - 1), np.where(np.arange(r) % 3, e - 1, rng.integers(-2, e + 2, r)),
                np.sort(rng.integers(0, e, r))[::-1]):
        ids = ids.astype(np.int32)
        y = torch.full((r, n), 7.0, dtype=torch.bfloat16, device=DEV)
        _run("gather", rows, rs, ids, w, up, y=y)
        good = (ids >= 0) & (ids < e)
        assert (as_f32(to_np(y))[~good] == 7).all()
        with np.errstate(over="ignore"):
            _check(to_np(y)[good], rows[good], rs[good], ids[good], w, up, f"R={r} E={e} glu={glu}")


def test_weights_past_four_gibibytes():
    """Weight and output offsets beyond 2^32 bytes: the last expert of 4.6 GB."""
    e, n, k = 9, 65536, 16384
    w = torch.zeros((e, n, k // 2), dtype=torch.uint8, device=DEV)
    ws = torch.full((e, n, k // 32), 127, dtype=torch.uint8, device=DEV)
    w[-1] = 0x22
    r = 40
    rows, rs = torch.full((r, k // 2), 0x22, dtype=torch.uint8, device=DEV), torch.full((r, k // 32), 121, dtype=torch.uint8, device=DEV)
    ids = torch.full((r,), e - 1, dtype=torch.int32, device=DEV)
    ids[0] = 0
    for y in (moe.moe_gather_gemm_mxfp4(rows, rs, ids, w, ws),
              moe.moe_grouped_gemm_mxfp4(rows, rs, torch.tensor([0] + [1] * (e - 1) + [r], dtype=torch.int32, device=DEV), w, ws)):
        assert bool((y[0] == 0).all()) and bool((y[1:] == k / 64).all())


@pytest.mark.parametrize("r", [520_000, 530_000])
def test_rows_in_any_order_past_four_gibibytes(r):
    """Row offsets up to and beyond 2^32 bytes (8192 of codes a row)."""
    k, n = 16384, 16
    rows = torch.zeros((r, k // 2), dtype=torch.uint8, device=DEV)
    rs = torch.full((r, k // 32), 121, dtype=torch.uint8, device=DEV)
    w, ws = torch.full((2, n, k // 2), 0x22, dtype=torch.uint8, device=DEV), torch.full((2, n, k // 32), 127, dtype=torch.uint8, device=DEV)
    ws[1] += 1
    ids = torch.arange(r, dtype=torch.int32, device=DEV) % 2
    hot = torch.tensor([0, 1, r // 2, r - 2, r - 1], device=DEV)
    rows[hot] = 0x22
    y = moe.moe_gather_gemm_mxfp4(rows, rs, ids, w, ws)
    assert int((y != 0).any(1).sum()) == 5
    assert torch.equal(y[hot], ((ids[hot] + 1) * (k // 64)).to(y.dtype).unsqueeze(1).expand(5, n))


def test_refusals():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    f = lambda *s: torch.zeros(s, device=DEV)
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(f(4, 48))
    with pytest.raises(TypeError):
        moe.moe_quantize_mxfp4(f(4, 64).half())
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(f(4, 64), codes=z(4, 31))
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(f(4, 128)[:, ::2])
    with pytest.raises(ValueError):
        moe.moe_quantize_mxfp4(f(4, 64), scales=z(4, 3))
    with pytest.raises(ValueError):
        moe.moe_dequant_mxfp4(z(4, 32), z(4, 3))
    with pytest.raises(TypeError):
        moe.moe_dequant_mxfp4(z(4, 32), z(4, 2), out_dtype=torch.float16)
    for fn, idx in ((moe.moe_grouped_gemm_mxfp4, i32(3)), (moe.moe_gather_gemm_mxfp4, i32(4))):
        ok = (z(4, 64), z(4, 4), idx, z(2, 8, 64), z(2, 8, 4))
        fn(*ok)
        for i, bad in ((0, z(4, 32)), (1, z(4, 3)), (2, i32(5)), (3, z(2, 8, 32)), (4, z(2, 8, 5)), (3, z(16, 64))):
            with pytest.raises(ValueError):
                fn(*[bad if i == j else t for j, t in enumerate(ok)])
        with pytest.raises(ValueError):
            fn(*ok, w_up=z(2, 8, 64))
        with pytest.raises(ValueError):
            fn(*ok, w_up=z(2, 9, 64), w_up_scales=z(2, 9, 4))
        with pytest.raises(ValueError):
            fn(*ok, y=torch.zeros((4, 9), dtype=torch.bfloat16, device=DEV))
        with pytest.raises(TypeError):
            fn(*ok, y=f(4, 8))
        with pytest.raises(moe.MoeError):                            # K = 64: not a multiple of 128
            fn(z(4, 32), z(4, 2), idx, z(2, 8, 32), z(2, 8, 2))
    with pytest.raises(moe.MoeError):
        moe.moe_gather_gemm_mxfp4(z(4, 64), z(4, 4), i32(4), z(2, 8, 64), z(2, 8, 4), workspace=z(256))


def _ffn(x, idx, w, res, q, gather):
    """An MXFP4 expert layer: each token quantised once, scattered, gate/up with
    SwiGLU, quantised, down, combined."""
    codes, scales = moe.moe_quantize_mxfp4(x)
    k = w.shape[1]
    rows, rs = moe.moe_scatter_rows(codes, res.dst_pos, k), moe.moe_scatter_rows(scales, res.dst_pos, k)
    if gather:
        h = moe.moe_gather_gemm_mxfp4(rows, rs, res.row_expert, *q["gate"], *q["up"])
        y = moe.moe_gather_gemm_mxfp4(*moe.moe_quantize_mxfp4(h), res.row_expert, *q["down"])
    else:
        h = moe.moe_grouped_gemm_mxfp4(rows, rs, res.expert_offsets, *q["gate"], *q["up"])
        y = moe.moe_grouped_gemm_mxfp4(*moe.moe_quantize_mxfp4(h), res.expert_offsets, *q["down"])
    return h, y, moe.moe_combine(y, res.dst_pos, w)


@pytest.mark.parametrize("n,e,k,d,f", [(1, 16, 4, 256, 384), (70, 8, 2, 512, 256), (600, 4, 2, 256, 640)])
@pytest.mark.parametrize("gather", [False, True])
def test_expert_layer_as_it_is_used(n, e, k, d, f, gather):
    rng = np.random.default_rng(n + f)
    x = codecs.f32_to_bf16_bits(rng.standard_normal((n, d)).astype(np.float32))
    logits = rng.standard_normal((n, e)).astype(np.float32)
    host = {m: quantize((rng.standard_normal((e * o, i)) * i ** -0.5).astype(np.float32))
            for m, o, i in (("gate", f, d), ("up", f, d), ("down", d, f))}
    host = {m: (c.reshape(e, -1, c.shape[1]), s.reshape(e, -1, s.shape[1])) for m, (c, s) in host.items()}
    q = {m: (to_dev(c), to_dev(s)) for m, (c, s) in host.items()}
    idx, w, res = moe.moe_route_dispatch(to_dev(logits), to_dev(x), k, sort=0 if gather else 1)
    h, y, out = _ffn(to_dev(x), idx, w, res, q, gather)
    ids, src = to_np(res.row_expert), to_np(res.src_pair)
    xc, xs = quantize(as_f32(x))
    _check(to_np(h), xc[src // k], xs[src // k], ids, host["gate"], host["up"], "h")
    # the second product from the h that the first one wrote
    hc, hs = quantize(as_f32(to_np(h)))
    _check(to_np(y), hc, hs, ids, host["down"], None, "y")
    assert tuple(out.shape) == (n, d) and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("r,offs", [(90, [0, 10, 10, 40, 41, 75, 90]), (40, [0, 10, 10, 20, 21, 35, 40]),
                                    (600, [0, 100, 100, 300, 301, 555, 600])])
def test_products_on_another_stream_and_in_a_graph(r, offs):
    """Two captured layers that share a workspace replay one after the other;
    every replay equals the eager result bit for bit."""
    rng = np.random.default_rng(9)
    e, k, n = 6, 384, 200
    x = to_dev(rng.standard_normal((r, k)).astype(np.float32))
    w, up = ([to_dev(t) for t in _operand(rng, e, n, k)] for _ in range(2))
    ids = to_dev(rng.integers(0, e, r).astype(np.int32))
    offs = to_dev(np.array(offs, np.int32))
    ws = torch.empty(moe.moe_gather_gemm_mxfp4_workspace_bytes(r, e), dtype=torch.uint8, device=DEV)
    c, s = torch.empty((r, k // 2), dtype=torch.uint8, device=DEV), torch.empty((r, k // 32), dtype=torch.uint8, device=DEV)
    outs = [torch.empty((r, n), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    back = torch.empty((r, k), dtype=torch.bfloat16, device=DEV)

    def step(stream=None):
        moe.moe_quantize_mxfp4(x, codes=c, scales=s, stream=stream)
        moe.moe_dequant_mxfp4(c, s, out=back, stream=stream)
        moe.moe_gather_gemm_mxfp4(c, s, ids, *w, *up, y=outs[0], workspace=ws, stream=stream)
        moe.moe_gather_gemm_mxfp4(c, s, ids, *up, y=outs[1], workspace=ws, stream=stream)
        moe.moe_grouped_gemm_mxfp4(c, s, offs, *w, y=outs[2], stream=stream)

    step()
    torch.cuda.synchronize()
    kept = [c, s, back] + outs
    eager = [t.clone() for t in kept]
    side = torch.cuda.Stream()
    for t in kept:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    late = moe.moe_gather_gemm_mxfp4(c, s, ids, *w, *up, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, eager)) and torch.equal(late, eager[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in kept + [ws]:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))
        step()


def test_memory_still_in_use_on_the_current_stream():
    """An output allocated by a call on another stream may get memory that a
    freed tensor's kernels, queued on the current stream, still write."""
    r, k = 4096, 4096
    x = torch.randn((r, k), device=DEV)
    want = [t.clone() for t in moe.moe_quantize_mxfp4(x)]
    side = torch.cuda.Stream()
    for _ in range(3):
        old = [torch.empty((r, k // 2), dtype=torch.uint8, device=DEV), torch.empty((r, k // 32), dtype=torch.uint8, device=DEV)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for t in old:
            t.fill_(9)
        del t, old
        got = moe.moe_quantize_mxfp4(x, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
