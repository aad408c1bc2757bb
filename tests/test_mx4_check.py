"""The products' comparisons themselves, with mistakes planted in what they are
given: NaN, a lost block, a lost run of blocks, a wrong sign."""
import numpy as np
import pytest
import torch

import mx4_check


def test_nan_is_not_within_a_tolerance():
    a, b = np.ones((3, 64)), np.full((5, 64), 0.5)
    tol = mx4_check.sum_tolerance(a, b, torch.float32)
    want = a @ b.T
    mx4_check.assert_within(want, want, tol, "the same")
    for bad in (np.full_like(want, np.nan), want + 1, want[:, :4]):
        with pytest.raises(AssertionError):
            mx4_check.assert_within(bad, want, tol, "planted")
    one = want.copy()
    one[2, 4] = np.nan
    with pytest.raises(AssertionError):
        mx4_check.assert_within(one, want, tol, "planted")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(1, 40, 65_536), (1, 40, 65_568), (3, 50, 21_857)])
def test_a_lost_block_differs_from_the_whole_sum(m, n, k, dtype):
    x, w = mx4_check.whole((m, k), 1), mx4_check.whole((n, k), 2)
    want = mx4_check.whole_product(x, w, dtype)
    mx4_check.assert_equal(want.clone(), want, "the same")
    nan = want.clone()
    nan[m - 1, 7] = float("nan")
    with pytest.raises(AssertionError):
        mx4_check.assert_equal(nan, want, "planted")
    for lost in (32, 16 * 32):
        with pytest.raises(AssertionError):
            mx4_check.assert_equal(mx4_check.whole_product(x[:, :-lost], w[:, :-lost], dtype), want, "planted")
