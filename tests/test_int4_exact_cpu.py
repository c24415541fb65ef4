"""The inputs of the exact product tests: their sums are fp32 numbers in any order, and a
kernel that kept fewer than three bf16 terms of a group's sum would change the products."""
import numpy as np
import pytest

from oracle.int4 import product, unpack
from tests.int4_forms import bf16, exact_case, form_of, three_terms


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("affine", [False, True])
def test_every_partial_sum_is_exact(group, affine):
    x, ex, w, _ = exact_case(40, 4, 1280, 6, group, affine)
    assert np.array_equal(bf16(x), x) and np.array_equal(bf16(w[1]), w[1])
    y, _ = product(x, ex, *w)
    # the sum of all magnitudes, codes and constant terms apart, bounds any partial sum
    mag = np.abs(x).astype(np.float64)
    g = mag.reshape(40, -1, group).sum(2)
    for i in range(40):
        q = unpack(w[0][ex[i]])
        s = w[1][ex[i]]
        b = np.abs(w[2][ex[i]]) if affine else 8 * s
        top = ((q * mag[i]).reshape(6, -1, group).sum(2) * s).sum(1) + (b * g[i]).sum(1)
        assert (top < 2 ** 23).all()
    assert np.array_equal(2 * y, np.rint(2 * y)) and np.array_equal(y.astype(np.float32), y)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("terms,share", [(1, 0.9), (2, 0.1), (3, 0.0)])
def test_fewer_terms_of_the_group_sums_would_show(group, terms, share):
    """One term leaves a row's large sum a remainder of up to 2^9, hardly ever 0; two hold that
    but where it is odd and above 2^8, in a quarter of the rows (200 of them: +- 3%)."""
    x, ex, w, _ = exact_case(200, 4, 1280, 6, group, True)
    kept = three_terms(x, group, terms)
    lost = x.astype(np.float64).reshape(200, -1, group).sum(2) - kept
    off = np.einsum("rg,rng->rn", lost, w[2][ex].astype(np.float64))
    if terms == 3:
        assert (off == 0).all()
    else:
        assert (off != 0).any(1).mean() > share


def test_forms_by_size():
    """The sizes that the kernels' comments name take the forms that they say."""
    assert form_of(8, 256, 2048, 7168, 128, 2, False) == ("wide", 16, True)
    assert form_of(48, 8, 14336, 4096, 64, 4, False) == ("wide", 16, True)
    assert form_of(1, 1, 7168, 2113, 64, 2, False) == ("deep", 16, True)
    assert form_of(1024, 256, 7168, 2048, 128, 2, True) == ("wide", 16, False)
    assert form_of(128, 8, 4096, 14336, 32, 2, True) == ("wide", 32, False)
    assert form_of(320, 30, 416, 1001, 32, 2, False) == ("split", 32, False)
