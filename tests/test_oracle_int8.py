"""Pins of the oracle's INT8 quantisation: hand values and rational arithmetic."""
from fractions import Fraction

import numpy as np

from oracle import moe_oracle as O


def test_hand_values():
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 0.0], [0.0] * 8, [254.0, 1.0, 3.0, 5.0, -1.0, 2.0, 0.9, 1.1]])
    q, s = O.quantize_int8(x)
    assert list(s) == [1.0, 1.0, 2.0]
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, 126, 0] and not q[1].any()
    assert q[2].tolist() == [127, 0, 2, 2, 0, 1, 0, 1]


def test_bad_rows_and_tiny_rows():
    x = np.array([[1.0, np.nan], [np.inf, 2.0], [2.0 ** -149, 0.0], [2.0 ** -115, -2.0 ** -121]])
    q, s = O.quantize_int8(x)
    assert np.isnan(s[:2]).all() and not q[:2].any()
    assert s[2] == s[3] == np.float32(2.0 ** -120) and q[2].tolist() == [0, 0] and q[3].tolist() == [32, 0]


def test_codes_are_the_nearest_integers():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 64)) * np.exp2(rng.integers(-140, 120, (40, 1)).astype(float))).astype(np.float32)
    q, s = O.quantize_int8(x)
    for r in range(40):
        sf = Fraction(float(s[r]))
        top = Fraction(float(np.abs(x[r]).max())) / 127
        assert s[r] == np.float32(2.0 ** -120) or abs(sf - top) <= top / 2 ** 24
        for c in range(64):
            v = Fraction(float(x[r, c])) / sf
            assert abs(v - int(q[r, c])) <= Fraction(1, 2)
    assert np.abs(q).max() == 127
