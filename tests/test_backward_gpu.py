"""Gradients of routing, dispatch and combine against the float64 oracle.

Tolerances, u = 2^-24 (half a step of fp32, relative):
* d_y: one fp32 product, then one rounding to y's type: u for fp32;
  2^-8 + u relative for bf16, plus half the smallest bf16 subnormal (2^-134);
* d_w: a lane adds ceil(D / 64) + 8 products at most in an FMA chain, then the
  wave adds six times: (ceil(D / 64) + 14) u times the sum of |terms|;
* d_x: k additions: k u times the sum of |terms|, then the type's rounding;
* d_logits: every term passes at most k additions of the sum S, a product, a
  difference and one more product: (k + 4) u times the terms' size.  With the
  full softmax the probability exp(l_e - l_r) w_r adds the rounding of the
  difference (u |l_e - l_r| in the exponent), expf (2 ulp = 4 u), the weight
  (the forward rounds it once from a few fp32 roundings: 1e-6 < 17 u, the
  forward's own tolerance) and a product: (k + 4 + 22 + max|l_e - l_r|) u.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle import codecs
from oracle.backward import combine_backward, dispatch_backward, route_backward
from oracle.route import route_topk
from tests.gpu_util import DEV, as_f32, to_dev, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _half(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 0.0


def _draw(rng, shape, dtype):
    a = rng.standard_normal(shape).astype(np.float32)
    return codecs.f32_to_bf16_bits(a) if dtype == "bf16" else a


def _positions(rng, n, k, drop):
    pos = rng.permutation(n * k).astype(np.int32)
    if drop:
        pos[rng.random(n * k) < drop] = -1
        pos[::7] = np.where(pos[::7] >= 0, pos[::7], n * k + 5)      # past the end, too
    return pos


SIZES = [(1, 1, 1), (1, 64, 8), (3, 8, 2), (5, 7, 3), (16, 64, 2), (33, 1001, 5), (9, 520, 64),
         (130, 2056, 4), (64, 7168, 8), (1, 7168, 1)]


@pytest.mark.parametrize("n,d,k", SIZES)
@pytest.mark.parametrize("gt,yt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_combine_backward(n, d, k, gt, yt, drop):
    rng = np.random.default_rng(n * 1000 + d + k)
    g, y = _draw(rng, (n, d), gt), _draw(rng, (n * k, d), yt)
    w = rng.uniform(0.0, 1.0, (n, k)).astype(np.float32)
    w.flat[0] = 0.0
    pos = _positions(rng, n, k, drop)
    d_y = torch.full((n * k, d), 7.0, dtype=torch.bfloat16 if yt == "bf16" else torch.float32, device=DEV)
    got_y, got_w = moe.moe_combine_backward(to_dev(g), to_dev(y), to_dev(pos), to_dev(w), d_y=d_y)
    assert got_y is d_y
    want_y, want_w, mag = combine_backward(as_f32(g), as_f32(y), pos, w, k)
    gy, gw = as_f32(to_np(got_y)).astype(np.float64), to_np(got_w).astype(np.float64)
    named = np.zeros(n * k, bool)
    named[pos[(pos >= 0) & (pos < n * k)]] = True
    assert (gy[~named] == 7.0).all()                                 # rows of no pair stay
    err = np.abs(gy - want_y)[named]
    assert (err <= (_half(yt) + U) * np.abs(want_y[named]) + 2.0 ** -134).all()
    assert (np.abs(gw - want_w) <= (-(-d // 64) + 14) * U * mag).all()


@pytest.mark.parametrize("n,d,k", SIZES)
@pytest.mark.parametrize("rt,xt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_dispatch_backward(n, d, k, rt, xt, drop):
    rng = np.random.default_rng(n * 1000 + d + k + 1)
    r = _draw(rng, (n * k, d), rt)
    pos = _positions(rng, n, k, drop)
    if drop:
        pos[:k] = -1                                                 # a token with no row left
    got = as_f32(to_np(moe.moe_dispatch_backward(
        to_dev(r), to_dev(pos), k, out_dtype=torch.bfloat16 if xt == "bf16" else torch.float32)))
    want, mag = dispatch_backward(as_f32(r), pos, k)
    bound = k * U * mag + _half(xt) * (np.abs(want) + k * U * mag)
    assert (np.abs(got.astype(np.float64) - want) <= bound + 2.0 ** -134).all()
    if drop:
        assert (got[0] == 0).all()


def test_unaligned_rows_take_the_scalar_path():
    """Views that start 2 (4) bytes past a 16-byte boundary."""
    rng = np.random.default_rng(3)
    n, d, k = 6, 64, 2
    g, y = _draw(rng, (n, d), "f32"), _draw(rng, (n * k, d), "bf16")
    w = rng.uniform(0.1, 1, (n, k)).astype(np.float32)
    pos = _positions(rng, n, k, 0)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    gd, yd = shifted(to_dev(g)), shifted(to_dev(y))
    a = moe.moe_combine_backward(gd, yd, to_dev(pos), to_dev(w), d_y=shifted(torch.zeros_like(yd)))
    b = moe.moe_combine_backward(gd.clone(), yd.clone(), to_dev(pos), to_dev(w))
    assert torch.equal(a[0], b[0])
    assert torch.allclose(a[1], b[1], rtol=0, atol=1e-4)             # another order of the same sum
    x = moe.moe_dispatch_backward(yd, to_dev(pos), k)
    assert torch.equal(x, moe.moe_dispatch_backward(yd.clone(), to_dev(pos), k))


def test_infinities_and_nans_stay_in_their_rows():
    n, d, k = 4, 128, 2
    g = torch.ones((n, d), device=DEV)
    y = torch.ones((n * k, d), device=DEV)
    g[1, 3] = float("inf")
    y[5, 9] = float("nan")                                           # pair 5: token 2, slot 1
    pos = torch.arange(n * k, dtype=torch.int32, device=DEV)
    pos[6] = -1
    y[6] = float("nan")                                              # a dropped pair's row: not read
    w = torch.full((n, k), 0.5, device=DEV)
    d_y, d_w = moe.moe_combine_backward(g, y, pos, w, d_y=torch.zeros_like(y))
    dw = to_np(d_w)
    assert dw[0].tolist() == [128, 128] and np.isinf(dw[1]).all()
    assert dw[2, 0] == 128 and np.isnan(dw[2, 1]) and dw[3].tolist() == [0, 128]
    dy = to_np(d_y)
    assert np.isinf(dy[2:4, 3]).all() and np.isfinite(np.delete(dy, 3, 1)).all() and (dy[6] == 0).all()


@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (1, 8, 2), (7, 8, 8), (33, 63, 5), (4, 64, 64), (9, 65, 7),
                                   (16, 130, 3), (1000, 256, 8), (5, 300, 6), (6, 585, 64), (3, 1024, 8)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_topk_backward(n, e, k, renorm):
    rng = np.random.default_rng(n + e + k)
    l = (rng.standard_normal((n, e)) * 3).astype(np.float32)
    if e > k:
        l[0, -1] = -np.inf                                           # a masked expert
        l[-1, 0] = np.finfo(np.float32).min
    idx, w = route_topk(l, k, renorm)
    d = rng.standard_normal((n, k)).astype(np.float32)
    out = torch.full((n, e), 7.0, device=DEV)
    got = moe.moe_route_topk_backward(to_dev(idx), to_dev(w), to_dev(d), e, renorm,
                                      None if renorm else to_dev(l), d_logits=out)
    assert got is out
    want, scale = route_backward(idx, w, d, e, renorm, l)
    gap = 0.0
    if not renorm:                        # where the probability is not lost to underflow (exp(-104) < 2^-149)
        lf = np.where(np.isfinite(l), l, -104.0).astype(np.float64)
        gap = np.minimum(lf.max(1, keepdims=True) - lf, 104.0) + 22
    bound = (k + 4 + gap) * U * scale + 2.0 ** -126
    assert (np.abs(to_np(got).astype(np.float64) - want) <= bound).all()


def test_route_backward_skips_bad_ids_and_adds_repeated_ones():
    w = torch.tensor([[0.5, 0.25, 0.25], [0.5, 0.25, 0.25]], device=DEV)
    d = torch.tensor([[1.0, 2.0, 4.0], [1.0, 2.0, 4.0]], device=DEV)
    idx = torch.tensor([[2, 2, 0], [1, -1, 9]], dtype=torch.int32, device=DEV)
    got = to_np(moe.moe_route_topk_backward(idx, w, d, 4))
    # S = 2: w_j (d_j - S) = -0.5, 0, 0.5;  second row: S = 0.5, 0.5 * (1 - 0.5)
    assert got.tolist() == [[0.5, 0, -0.5, 0], [0, 0.25, 0, 0]]


@pytest.mark.parametrize("renorm", [True, False])
def test_rows_of_masked_experts(renorm):
    """Fewer experts left than slots: the masked slots weigh 0 and get gradient 0.
    Weights of NaN (a row with every expert masked) give NaN where they reach."""
    n, e, k = 5, 70, 4
    rng = np.random.default_rng(4)
    l = rng.standard_normal((n, e)).astype(np.float32)
    l[1, 2:] = -np.inf                          # two experts for four slots
    l[2, 1:] = -np.inf
    l[4, 3:] = np.finfo(np.float32).min
    idx, w = route_topk(l, k, renorm)
    l[3], w[3] = -np.inf, np.nan
    d = rng.standard_normal((n, k)).astype(np.float32)
    got = to_np(moe.moe_route_topk_backward(to_dev(idx), to_dev(w), to_dev(d), e, renorm, to_dev(l)))
    ok = [0, 1, 2, 4]
    want, scale = route_backward(idx[ok], w[ok], d[ok], e, renorm, l[ok])
    gap = 0.0 if renorm else np.where(np.isfinite(l[ok]), l[ok].max(1, keepdims=True) - l[ok], 104.0).clip(0, 104.0) + 22
    assert (np.abs(got[ok] - want) <= (k + 4 + gap) * U * scale + 2.0 ** -126).all()
    assert (got[1, 2:] == 0).all() and (got[2, 1:] == 0).all()
    assert np.isnan(got[3][idx[3]]).all()


def test_gradient_of_a_run_matches_autograd():
    """Route, dispatch, identity experts with a per-row gain, combine and back:
    the three gradients chained against torch's autograd in float64."""
    rng = np.random.default_rng(11)
    n, e, k, d = 48, 16, 4, 256
    logits, x = to_dev(rng.standard_normal((n, e)).astype(np.float32)), to_dev(_draw(rng, (n, d), "f32"))
    g = to_dev(_draw(rng, (n, d), "f32"))
    for renorm in (True, False):
        for sort in (0, 1):
            idx, w, res = moe.moe_route_dispatch(logits, x, k, renormalize=renorm, sort=sort)
            gain = 1.0 + res.row_expert.float().unsqueeze(1) / e
            y = (res.rows * gain).contiguous()
            d_y, d_w = moe.moe_combine_backward(g, y, res.dst_pos, w)
            d_x = moe.moe_dispatch_backward((d_y * gain).contiguous(), res.dst_pos, k)
            d_l = moe.moe_route_topk_backward(idx, w, d_w, e, renorm, logits)
            lx = logits.double().cpu().requires_grad_()
            xx = x.double().cpu().requires_grad_()
            i = idx.long().cpu()
            p = torch.softmax(lx.gather(1, i), 1) if renorm else torch.softmax(lx, 1).gather(1, i)
            out = ((p * (1.0 + i.double() / e)).sum(1, keepdim=True)) * xx
            out.backward(g.double().cpu())
            # sums of 256 unit terms through about 20 fp32 roundings each
            assert (d_x.double().cpu() - xx.grad).abs().max() <= 64 * U * 8
            assert (d_l.double().cpu() - lx.grad).abs().max() <= 64 * U * 256


def test_backward_refusals():
    t = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)
    pos, w = t(8, dt=torch.int32), t(4, 2)
    with pytest.raises(ValueError):
        moe.moe_combine_backward(t(4, 63), t(8, 64), pos, w)
    with pytest.raises(ValueError):
        moe.moe_combine_backward(t(4, 64), t(7, 64), pos, w)
    with pytest.raises(TypeError):
        moe.moe_combine_backward(t(4, 64).half(), t(8, 64), pos, w)
    with pytest.raises(TypeError):
        moe.moe_combine_backward(t(4, 64), t(8, 64), pos, w, d_y=t(8, 64, dt=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_combine_backward(t(4, 64), t(8, 64), pos, w, d_topk_w=t(8))
    with pytest.raises(ValueError):
        moe.moe_combine_backward(t(4, 128)[:, ::2], t(8, 64), pos, w)
    with pytest.raises(ValueError):
        moe.moe_dispatch_backward(t(8, 64), pos, 3)
    with pytest.raises(ValueError):
        moe.moe_dispatch_backward(t(8, 64), pos, 2, d_x=t(3, 64))
    with pytest.raises(TypeError):
        moe.moe_dispatch_backward(t(8, 64), pos, 2, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.moe_route_topk_backward(t(4, 2, dt=torch.int32), w, w, 8, renormalize=False)
    with pytest.raises(ValueError):
        moe.moe_route_topk_backward(t(4, 2, dt=torch.int32), w, w, 8, logits=t(4, 7), renormalize=False)
    with pytest.raises(moe.MoeError):
        moe.moe_route_topk_backward(t(4, 2, dt=torch.int32), w, w, 1)          # k > E
    with pytest.raises(ValueError):
        moe.moe_combine_backward(t(4, 64).cpu(), t(8, 64), pos, w)


def test_backward_of_no_tokens():
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=DEV)
    d_y, d_w = moe.moe_combine_backward(z(0, 64), z(0, 64), z(0, dt=torch.int32), z(0, 2))
    assert d_y.shape == (0, 64) and d_w.shape == (0, 2)
    assert moe.moe_dispatch_backward(z(0, 64), z(0, dt=torch.int32), 2).shape == (0, 64)
    assert moe.moe_route_topk_backward(z(0, 2, dt=torch.int32), z(0, 2), z(0, 2), 8).shape == (0, 8)


def test_backward_on_another_stream_and_in_a_graph():
    """Every replay, with eager work between, equals the eager result bit for bit."""
    rng = np.random.default_rng(12)
    n, d, k, e = 40, 512, 4, 16
    g, y = to_dev(_draw(rng, (n, d), "bf16")), to_dev(_draw(rng, (n * k, d), "bf16"))
    w, pos = to_dev(rng.uniform(0.1, 1, (n, k)).astype(np.float32)), to_dev(_positions(rng, n, k, 0))
    idx = to_dev(np.stack([rng.permutation(e)[:k] for _ in range(n)]).astype(np.int32))
    outs = [torch.empty_like(y), torch.empty_like(w), torch.empty_like(g), torch.empty((n, e), device=DEV)]

    def step(stream=None):
        moe.moe_combine_backward(g, y, pos, w, d_y=outs[0], d_topk_w=outs[1], stream=stream)
        moe.moe_dispatch_backward(outs[0], pos, k, d_x=outs[2], stream=stream)
        moe.moe_route_topk_backward(idx, w, outs[1], e, d_logits=outs[3], stream=stream)

    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    # allocated in the call on another stream than the current one
    late = moe.moe_combine_backward(g, y, pos, w, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, eager))
    assert torch.equal(late[0], eager[0]) and torch.equal(late[1], eager[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        step()


def test_rows_past_four_gibibytes():
    """Row offsets beyond 2^32 bytes: the last rows of a 4.4 GB buffer."""
    n, d, k = 300000, 3680, 2
    y = torch.zeros((n * k, d), dtype=torch.bfloat16, device=DEV)
    g = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(n * k, dtype=torch.int32, device=DEV)
    w = torch.full((n, k), 0.5, device=DEV)
    y[-1], g[-1] = 2.0, 3.0
    d_y, d_w = moe.moe_combine_backward(g, y, pos, w)
    assert float(d_w[-1, 1]) == 6.0 * d and float(d_w[-1, 0]) == 0.0
    assert bool((d_y[-2:] == 1.5).all()) and bool((d_y[:4] == 0).all())
    x = moe.moe_dispatch_backward(d_y, pos, k)
    assert bool((x[-1] == 3.0).all()) and bool((x[:2] == 0).all())


def test_more_pairs_than_one_launch_has_threads():
    """70 million pairs: a wave each is more than 2^32 threads."""
    n = 70_000_000
    pos = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV)
    g = torch.arange(n, device=DEV, dtype=torch.int32).remainder_(1000).float().unsqueeze(1)
    w = torch.full((n, 1), 0.5, device=DEV)
    d_y, d_w = moe.moe_combine_backward(g, torch.full((n, 1), 2.0, device=DEV), pos, w)
    assert torch.equal(d_w, 2 * g) and torch.equal(d_y.flip(0), 0.5 * g)
    del d_w
    x = moe.moe_dispatch_backward(d_y, pos, 1)
    assert torch.equal(x, 0.5 * g)
    assert torch.equal(moe.moe_combine(d_y, pos, w), 0.25 * g)        # the forward call, too
    del x, d_y
    idx = torch.zeros((n, 1), dtype=torch.int32, device=DEV)
    d = moe.moe_route_topk_backward(idx, w, g, 1)
    assert torch.equal(d, 0.5 * (g - 0.5 * g))
