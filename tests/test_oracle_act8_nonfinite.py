"""The oracle's 8-bit format where a block holds a NaN or an infinity."""
import numpy as np

import oracle


def test_a_block_with_what_is_not_finite():
    x = np.tile(np.linspace(-1, 1, 64), (4, 2))
    x[1, 3], x[2, 70], x[3, 0], x[3, 1] = np.nan, -np.inf, np.inf, np.nan
    codes, a = oracle.act8(x)
    assert np.isnan(a[1, 0]) and a[2, 1] == np.inf and np.isnan(a[3, 0]) and np.isfinite(a[[0, 0, 1, 2, 3], [0, 1, 1, 0, 1]]).all()
    assert not codes[1, :64].any() and not codes[2, 64:].any() and not codes[3, :64].any()
    v = oracle.act8_values(codes, a)
    assert np.isnan(v[1, :64]).all() and np.isnan(v[2, 64:]).all() and np.isnan(v[3, :64]).all()
    assert np.array_equal(v[0], np.r_[v[1, 64:], v[1, 64:]]) and np.array_equal(codes[0, :64], codes[2, :64])
