"""Pins of the group-scaled 4-bit weights' oracle: groups that are not finite."""
import numpy as np

from oracle import group4


def test_a_group_that_is_not_finite_by_hand():
    w = np.zeros((1, 96), np.float32)
    w[0, 0], w[0, 1] = 7.0, np.nan
    w[0, 32], w[0, 33] = 3.5, -7.0
    w[0, 64] = -np.inf
    c, packed, s = group4.pack(w.astype(np.float16), "fp16", 32)
    assert np.isnan(s[0, 0]) and s[0, 1] == 1.0 and np.isnan(s[0, 2])
    assert not c[0, :32].any() and not c[0, 64:].any() and c[0, 32:34].tolist() == [4, -7]
    assert not packed[0, :16].any() and not packed[0, 32:].any()
