"""Rows of the combine's gradient: those of dropped pairs in an output that the
call allocates, and hidden sizes of every load width, over many pairs.

Tolerances, u = 2^-24: d_y is one fp32 product and one rounding to its type
(2^-8 for bf16); a lane of d_w adds ceil(D / 64) + 8 products at most and the
wave six times more: (ceil(D / 64) + 14) u of the sum of |terms|.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle import codecs
from oracle.backward import combine_backward
from tests.gpu_util import DEV, as_f32, to_dev, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def _draw(rng, shape, dtype):
    a = rng.standard_normal(shape).astype(np.float32)
    return codecs.f32_to_bf16_bits(a) if dtype == "bf16" else a


def _case(n, d, k, gt, yt, drop):
    rng = np.random.default_rng(n + d + k)
    pos = rng.permutation(n * k).astype(np.int32)
    if drop:
        gone = rng.random(n * k) < drop
        pos[gone] = np.where(np.arange(n * k) % 2, -1, n * k + 3)[gone]
    return _draw(rng, (n, d), gt), _draw(rng, (n * k, d), yt), pos, rng.uniform(0.1, 1, (n, k)).astype(np.float32)


def _check(d_y, d_w, g, y, pos, w, yt):
    k, d = w.shape[1], y.shape[1]
    want_y, want_w, mag = combine_backward(as_f32(g), as_f32(y), pos, w, k)
    half = 2.0 ** -8 if yt == "bf16" else 0.0
    err = np.abs(as_f32(to_np(d_y)).astype(np.float64) - want_y)
    assert (err <= (half + U) * np.abs(want_y) + 2.0 ** -134).all()
    assert (np.abs(to_np(d_w).astype(np.float64) - want_w) <= (-(-d // 64) + 14) * U * mag).all()


@pytest.mark.parametrize("n,d,k", [(1, 1, 1), (5, 7, 3), (40, 520, 4), (129, 2052, 2), (64, 7168, 8)])
@pytest.mark.parametrize("gt,yt", TYPES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_rows_of_dropped_pairs_are_zero_by_default(n, d, k, gt, yt, drop):
    g, y, pos, w = _case(n, d, k, gt, yt, drop)
    t = [to_dev(a) for a in (g, y, pos, w)]
    used = torch.full_like(t[1], float("nan"))                       # memory that held other values
    del used
    d_y, d_w = moe.moe_combine_backward(*t)
    _check(d_y, d_w, g, y, pos, w, yt)


def test_default_rows_on_another_stream_and_in_a_graph():
    g, y, pos, w = _case(60, 1028, 4, "bf16", "bf16", 0.4)
    t = [to_dev(a) for a in (g, y, pos, w)]
    eager = moe.moe_combine_backward(*t)
    _check(*eager, g, y, pos, w, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    used = torch.full_like(t[1], float("nan"))
    del used
    late = moe.moe_combine_backward(*t, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(late, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = moe.moe_combine_backward(*t)
    for _ in range(4):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        moe.moe_combine_backward(*t)


def test_a_given_output_keeps_the_rows_of_no_pair():
    g, y, pos, w = _case(30, 260, 3, "f32", "f32", 0.5)
    d_y = torch.full((90, 260), 7.0, device=DEV)
    moe.moe_combine_backward(*[to_dev(a) for a in (g, y, pos, w)], d_y=d_y)
    gone = np.setdiff1d(np.arange(90), pos)
    assert gone.size and bool((d_y[gone] == 7).all())


# groups of 4 elements (hidden sizes that are 4 modulo 8), below, at and past a
# pass of the wave, with few long rows and with short ones
@pytest.mark.parametrize("n,d,k", [(3, 4, 2), (33, 12, 5), (9, 516, 3), (70, 1028, 2), (20, 2052, 4), (6, 4100, 8)])
@pytest.mark.parametrize("gt,yt", TYPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_groups_of_four(n, d, k, gt, yt, drop):
    g, y, pos, w = _case(n, d, k, gt, yt, drop)
    _check(*moe.moe_combine_backward(*[to_dev(a) for a in (g, y, pos, w)]), g, y, pos, w, yt)


# a wave per pair (4096 pairs and more) over rows of several passes: groups of 8,
# of 4 and single elements
@pytest.mark.parametrize("d", [2056, 4100, 2049, 7168])
@pytest.mark.parametrize("gt,yt", TYPES)
def test_many_pairs_of_long_rows(d, gt, yt):
    g, y, pos, w = _case(2100, d, 2, gt, yt, 0.1)
    _check(*moe.moe_combine_backward(*[to_dev(a) for a in (g, y, pos, w)]), g, y, pos, w, yt)
