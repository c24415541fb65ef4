"""Pins of the balance-loss oracle."""
import numpy as np
import pytest

from oracle.balance import balance, balance_backward


def test_even_and_one_expert_in_closed_form():
    n, e = 12, 4
    idx = np.stack([(np.arange(n) + j) % e for j in range(2)], 1)
    r = balance(np.zeros((n, e)), idx)
    assert r["loss"][0] == 1.0 and (r["counts"] == 6).all() and (r["probs"] == 0.25).all()
    assert np.isclose(r["z_loss"][0], np.log(4.0) ** 2, rtol=1e-15)
    one = np.zeros((n, e))
    one[:, 1] = 1000.0                                   # everything on expert 1
    r = balance(one, np.ones((n, 1), int))
    assert r["loss"][0] == e and r["z_loss"][0] == 1e6 and r["counts"].tolist() == [[0, n, 0, 0]]


def test_written_out():
    l = np.log(np.array([[1.0, 3.0], [1.0, 1.0], [3.0, 1.0], [7.0, 1.0]]))
    idx = np.array([[1], [0], [0], [5]])                 # the last slot was dropped
    r = balance(l, idx, offs=[0, 2, 2, 4], mask=[1, 1, 1, 1])
    assert r["tokens"].tolist() == [2, 0, 2]
    assert r["counts"].tolist() == [[1, 1], [0, 0], [1, 0]]
    assert np.allclose(r["probs"], [[0.375, 0.625], [0, 0], [0.8125, 0.1875]], rtol=1e-15)
    assert np.allclose(r["loss"], [1.0, 0.0, 0.8125], rtol=1e-15)
    assert np.allclose(r["z_loss"], [(np.log(4) ** 2 + np.log(2) ** 2) / 2, 0, (np.log(4) ** 2 + np.log(8) ** 2) / 2])


def test_masked_tokens_and_empty_rows_do_not_count():
    rng = np.random.default_rng(0)
    l = rng.standard_normal((9, 5))
    l[4] = -np.inf
    l[6, 2] = -np.inf
    idx = rng.integers(0, 5, (9, 2))
    mask = np.array([1, 0, 1, 1, 1, 1, 1, 0, 1])
    keep = [0, 2, 3, 5, 6, 8]
    a, b = balance(l, idx, mask=mask), balance(l[keep], idx[keep])
    for name in a:
        assert np.allclose(a[name], b[name], rtol=1e-14), name
    assert a["probs"][0].sum() == pytest.approx(1.0)


@pytest.mark.parametrize("offs", [None, [0, 3, 3, 7]])
def test_gradient_against_differences(offs):
    rng = np.random.default_rng(1)
    n, e, k = 8, 6, 2
    l, idx = rng.standard_normal((n, e)), rng.integers(0, e, (n, k))
    l[2, 1] = -np.inf
    mask = np.array([1, 1, 1, 0, 1, 1, 1, 1])
    r = balance(l, idx, offs, mask)
    b = r["loss"].size
    dl, dz = rng.standard_normal(b), rng.standard_normal(b)
    g = balance_backward(l, r["counts"], r["tokens"], k, dl, dz, offs, mask)

    def value(x):                                        # the ids, so the counts, stay as they are
        v = balance(x, idx, offs, mask)
        return (dl * v["loss"]).sum() + (dz * v["z_loss"]).sum()

    for t in range(n):
        for j in range(e):
            if np.isinf(l[t, j]):
                assert g[t, j] == 0
                continue
            h = np.zeros_like(l)
            h[t, j] = 1e-5
            assert (value(l + h) - value(l - h)) / 2e-5 == pytest.approx(g[t, j], abs=1e-9), (t, j)
    if offs:
        assert (g[7] == 0).all()
    assert (g[3] == 0).all()


def test_gradient_of_a_batch_in_two_parts():
    """Counts and tokens summed over the parts give the gradient of the whole."""
    rng = np.random.default_rng(2)
    l, idx = rng.standard_normal((10, 7)), rng.integers(0, 7, (10, 3))
    whole = balance(l, idx)
    parts = [balance(l[s], idx[s]) for s in (slice(0, 4), slice(4, 10))]
    counts, tokens = sum(p["counts"] for p in parts), sum(p["tokens"] for p in parts)
    g = balance_backward(l, whole["counts"], whole["tokens"], 3, [0.7], [0.3])
    for s in (slice(0, 4), slice(4, 10)):
        assert np.allclose(balance_backward(l[s], counts, tokens, 3, [0.7], [0.3]), g[s], rtol=1e-13)
