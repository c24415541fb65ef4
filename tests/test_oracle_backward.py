"""Pins of the gradient oracle: central differences of the forward oracles."""
import numpy as np
import pytest

from oracle import dispatch as od
from oracle.backward import combine_backward, dispatch_backward, route_backward
from oracle.combine import combine_f64


def _case(seed=0, n=5, e=6, k=3, d=4):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(e)[:k] for _ in range(n)]).astype(np.int32)
    pos = od.dispatch(idx, e, 1, True)["dst_pos"]
    return rng, idx, pos


def test_combine_gradient_against_differences():
    rng, _, pos = _case()
    n, k, d = 5, 3, 4
    y = rng.standard_normal((n * k, d))
    w = rng.uniform(0.1, 1.0, (n, k)).astype(np.float32)
    g = rng.standard_normal((n, d))
    d_y, d_w, _ = combine_backward(g, y, pos, w, k)
    h = 2.0 ** -8                     # the forward is linear in y and in w: the difference is exact
    for i in range(y.shape[0]):       # up to float64 rounding
        for c in range(d):
            up, dn = y.copy(), y.copy()
            up[i, c] += h
            dn[i, c] -= h
            num = ((combine_f64(up, pos, w, k) - combine_f64(dn, pos, w, k)) * g).sum() / (2 * h)
            assert abs(num - d_y[i, c]) <= 1e-11
    for t in range(n):
        for j in range(k):
            up, dn = w.copy(), w.copy()
            up[t, j] += np.float32(h)
            dn[t, j] -= np.float32(h)
            step = float(up[t, j]) - float(dn[t, j])
            num = ((combine_f64(y, pos, up, k) - combine_f64(y, pos, dn, k)) * g).sum() / step
            assert abs(num - d_w[t, j]) <= 1e-11


def test_dispatch_gradient_is_the_transpose():
    """<rows(x), r> = <x, d_x(r)> for every x and r (the copy is linear)."""
    rng, idx, pos = _case(1)
    x = rng.standard_normal((5, 4)).astype(np.float32)
    rows = od.dispatch(idx, 6, 1, True, x=x)["rows"].astype(np.float64)
    r = rng.standard_normal(rows.shape)
    d_x, _ = dispatch_backward(r, pos, 3)
    assert abs((rows * r).sum() - (x * d_x).sum()) <= 1e-12 * np.abs(rows * r).sum()


def test_dropped_pairs_hold_nothing():
    pos = np.array([0, -1, 3, 99], np.int32)
    g, y = np.ones((2, 3)), np.ones((4, 3))
    d_y, d_w, _ = combine_backward(g, y, pos, np.ones((2, 2)), 2)
    assert d_w.tolist() == [[3, 0], [3, 0]] and d_y[:, 0].tolist() == [1, 0, 0, 1]
    d_x, _ = dispatch_backward(y, pos, 2)
    assert (d_x == 1).all()
    d_x, _ = dispatch_backward(y, np.array([-1, -1, 1, 2]), 2)
    assert (d_x[0] == 0).all() and (d_x[1] == 2).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    rng = np.random.default_rng(2)
    n, e, k = 4, 7, 3
    l = rng.standard_normal((n, e))
    idx = np.argsort(-l, axis=1)[:, :k]
    d = rng.standard_normal((n, k))

    def weights(l):
        sel = np.take_along_axis(l, idx, 1)
        den = np.exp(sel).sum(1) if renorm else np.exp(l).sum(1)
        return np.exp(sel) / den[:, None]

    got, _ = route_backward(idx, weights(l), d, e, renorm, l)
    h = 1e-5
    for t in range(n):
        for c in range(e):
            up, dn = l.copy(), l.copy()
            up[t, c] += h
            dn[t, c] -= h
            num = ((weights(up) - weights(dn)) * d).sum() / (2 * h)
            # third derivative of a softmax is below 1: h^2 |d| + rounding 2^-53 / h
            assert abs(num - got[t, c]) <= 1e-9
    assert np.abs(got.sum(1)).max() <= 1e-12       # a shift of all logits changes nothing
