"""The four-bit cache's comparison rejects what is not a number (no GPU needed)."""

import numpy as np
import pytest

from kvq_check import assert_within


def test_close_values_pass():
    assert_within(np.array([1.0, 2.0, 0.0]), np.array([1.01, 2.0, 0.0]), np.array([0.02, 0.0, 0.0]))
    assert_within(np.zeros((0, 4)), np.zeros((0, 4)), np.zeros((0, 4)))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 1.5])
def test_others_do_not(bad):
    for tol in (0.1, np.full(3, 0.1)):
        with pytest.raises(AssertionError):
            assert_within(np.array([1.0, bad, 1.0]), np.ones(3), tol)


def test_infinite_tolerances_let_no_nan_through():
    for bad in (np.nan, np.inf):
        with pytest.raises(AssertionError):
            assert_within(np.array([bad]), np.ones(1), np.inf)
    with pytest.raises(AssertionError):
        assert_within(np.ones(1), np.array([np.nan]), np.inf)
