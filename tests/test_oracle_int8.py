"""Oracle self-tests of the 8-bit integer linear: codes against exact rational
arithmetic, ties, rows without a finite scale, sums against Python integers."""

from fractions import Fraction

import numpy as np

from oracle import matmul_int8, quantize_int8


def nearest(x, s):
    """Nearest whole number to x / s, ties to even, in exact arithmetic."""
    return max(-127, min(127, round(Fraction(float(x)) / Fraction(float(s)))))


def test_codes_are_nearest():
    r = np.random.default_rng(0)
    X = (r.normal(size=(40, 57)) * 10.0 ** r.integers(-30, 30, size=(40, 1))).astype(np.float32)
    X[0] = np.float32(1e-43) * np.arange(57)  # subnormal scale
    codes, scale = quantize_int8(X)
    for i in range(40):
        assert scale[i] == np.float32(np.abs(X[i]).max() / np.float32(127))
        assert [int(c) for c in codes[i]] == [nearest(x, scale[i]) for x in X[i]]


def test_ties_go_to_the_even_code():
    X = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -125.5]], dtype=np.float32)
    assert quantize_int8(X)[0].tolist() == [[127, 0, 2, 2, 0, -2, 126, -126]]


def test_rows_without_a_finite_scale():
    X = np.ones((4, 8), dtype=np.float32)
    X[1, 3], X[2, 5], X[3] = np.inf, np.nan, 0.0
    codes, scale = quantize_int8(X)
    assert np.isinf(scale[1]) and np.isnan(scale[2]) and scale[3] == 0
    assert not codes[1:].any() and (codes[0] == 127).all()


def test_product_in_whole_numbers():
    r = np.random.default_rng(1)
    xq, wq = r.integers(-127, 128, (3, 301)), r.integers(-127, 128, (5, 301))
    got = matmul_int8(xq, np.ones(3), wq, np.full(5, 2.0))
    want = [[2 * sum(int(a) * int(b) for a, b in zip(x, w)) for w in wq] for x in xq]
    assert got.tolist() == want
