"""moe_route_topk_backward with the full softmax, where slot 0 is not the row's
largest logit: ids out of range, slots in another order, extreme logits.

Tolerance, u = 2^-24.  A probability exp(l - max) / sum carries the rounding of
the difference (u (max - l) in the exponent), expf (2 ulp = 4 u) and, through
the sum, at most 21 additions of positive terms (16 per lane, 6 over the wave),
each term's expf (4 u) and its difference (u times the mean of max - l under
the softmax, at most ln E < 7), then a reciprocal and a product: 39 u + (max -
l) u.  The sum S adds k + 1 roundings, the product with it and the difference
2 more: (k + 42 + max - l) u of the terms' size, and the smallest normal where
results underflow.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle.backward import route_backward
from tests.gpu_util import DEV, to_dev, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _weights(l, idx):
    """Softmax weights of the slots in float64, rounded once; 0 at a bad id."""
    l = l.astype(np.float64)
    p = np.exp(l - l.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ok = (idx >= 0) & (idx < l.shape[1])
    return np.where(ok, np.take_along_axis(p, np.where(ok, idx, 0), 1), 0.5).astype(np.float32)


def _check(l, idx, w, d):
    e, k = l.shape[1], idx.shape[1]
    got = to_np(moe.moe_route_topk_backward(to_dev(idx), to_dev(w), to_dev(d), e, False, to_dev(l),
                                            d_logits=torch.full(l.shape, 7.0, device=DEV)))
    want, scale = route_backward(idx, w, d, e, False, l)
    lf = np.where(np.isfinite(l), l, l.max(1, keepdims=True) - 104.0).astype(np.float64)
    gap = np.minimum(lf.max(1, keepdims=True) - lf, 104.0)           # exp(-104) < 2^-149
    bound = (k + 42 + gap) * U * scale + 2.0 ** -126
    bad = ~(np.abs(got.astype(np.float64) - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside the bound"


SIZES = [(1, 1, 1), (1, 2, 2), (7, 8, 3), (33, 63, 5), (4, 64, 64), (9, 65, 7), (50, 130, 4), (300, 256, 8),
         (5, 300, 6), (6, 585, 64), (3, 1024, 8)]


def _draw(n, e, k, scale=3.0):
    rng = np.random.default_rng(n + 3 * e + k)
    l = (rng.standard_normal((n, e)) * scale).astype(np.float32)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, l, idx, rng.standard_normal((n, k)).astype(np.float32)


@pytest.mark.parametrize("n,e,k", SIZES)
def test_slot_zero_out_of_range(n, e, k):
    """A dropped best expert adds nothing to S; the probabilities stay those of
    all E logits."""
    rng, l, idx, d = _draw(n, e, k)
    idx[:, 0] = np.array([-1, e, 2**31 - 1])[np.arange(n) % 3]
    _check(l, idx, _weights(l, idx), d)
    idx[rng.random((n, k)) < 0.5] = -1                               # and more of them, rows without any
    _check(l, idx, _weights(l, idx), d)


@pytest.mark.parametrize("n,e,k", SIZES)
@pytest.mark.parametrize("scale", [3.0, 40.0, 2000.0])
def test_slots_in_any_order(n, e, k, scale):
    """Ascending and shuffled slots; logits far beyond exp's range."""
    rng, l, idx, d = _draw(n, e, k, scale)
    idx = idx[:, ::-1].copy()
    _check(l, idx, _weights(l, idx), d)
    idx = rng.permuted(idx, axis=1).copy()
    _check(l, idx, _weights(l, idx), d)


def test_masked_experts_and_large_logits():
    rng, l, idx, d = _draw(40, 100, 4)
    l[:, 5::7] = -np.inf
    l[1::2, 3] = np.finfo(np.float32).min
    l[2] += 1000.0
    l[3, 11] = 3e38
    l[4, 1:] = -np.inf
    idx = np.argsort(-l, axis=1, kind="stable")[:, :4].astype(np.int32)
    idx[::3, 0] = -1
    _check(l, idx, _weights(l, idx), d)


def test_slots_that_are_not_the_best():
    """Any k experts may carry the weights, the largest logit outside them."""
    rng, l, _, d = _draw(64, 200, 5, 10.0)
    idx = np.argsort(l, axis=1, kind="stable")[:, 20:25].astype(np.int32)
    _check(l, np.ascontiguousarray(idx), _weights(l, idx), d)
