"""What lets the kernel that writes a 4-bit cache choose NF4's nearest code by an approximate quotient: how far the quotients of bf16
values stay from every midpoint of two codes, against the error of its comparison there."""
import numpy as np

import oracle


def test_quotients_stay_further_from_every_midpoint_than_the_comparison_errs():
    """The kernel compares y = fl32(x fl32(16 / a) + 16) with fl32(16 m + 16): the reciprocal is within 2^-23 of its value, both sides
    are rounded once. Values have 8 significant bits and magnitudes up to the maximum's."""
    code = oracle.codebook().astype(np.float64)
    p = np.arange(1, 256, dtype=np.float64)      # 128..255 are the significands; below, subnormal ones
    r = np.unique((p[:, None] / p[None, :])[..., None] * 2.0 ** np.arange(-30, 9))
    r = r[r <= 1]
    r = np.concatenate([-r[::-1], [0.0], r])
    nearest = []
    for m in (code[1:] + code[:-1]) / 2:
        distance = np.abs(r - m).min()
        step = 2.0 ** (np.floor(np.log2(16 * m + 16)) - 23)
        error = abs(m) * 2.0 ** -23 + (step / 2 + step / 2) / 16
        assert distance > 1.5 * error, m
        nearest.append((distance, error, m))
    distance, error, m = min(nearest)
    assert 2.1e-7 < distance < 2.2e-7 and error < 1.3e-7 and abs(m - 0.0398) < 1e-4
    assert sorted(nearest)[1][0] > 2.9e-7 and max(e for _, e, _ in nearest) < 2.3e-7
