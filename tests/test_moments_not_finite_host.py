"""The oracle's rule for moments that are not finite: the code of NaN for them, scale and
codes of their group's others as if they were zeros."""

import numpy as np
import pytest

from oracle import e4m3, training_step as ots


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_codes_of_nan_beside_the_others(bad, second):
    rng = np.random.default_rng(1)
    x = np.abs(rng.standard_normal(300)).astype(np.float32)
    at = [0, 127, 130, *range(256, 300)]
    zeroed, lost = x.copy(), x.copy()
    zeroed[at], lost[at] = 0, bad
    q, s = ots.encode_moments(lost, 5, second)
    qz, sz = ots.encode_moments(zeroed, 5, second)
    assert (q[at] == 0x7F).all() and np.isnan(e4m3.decode(q[at])).all()
    others = np.setdiff1d(np.arange(300), at)
    assert np.array_equal(q[others], qz[others]) and np.array_equal(s, sz)
    assert np.isfinite(s).all() and s[2] == 0
    assert np.isnan(ots.decode_moments(q, s)[at]).all()
