"""The comparison of computed rows with a reference: a value that is no number fails it."""

import numpy as np


def assert_within(got, want, tol):
    """Every value of `got` is a finite number at most `tol` from `want`."""
    ok = np.abs(got - want) <= tol                           # False where either is NaN
    ok &= np.isfinite(got)
    assert ok.all(), (np.argwhere(~ok)[:3], got[~ok][:3], want[~ok][:3], np.broadcast_to(tol, got.shape)[~ok][:3])
