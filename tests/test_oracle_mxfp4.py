"""The oracle of 4-bit floating point, pinned by hand cases and by exact
rational arithmetic."""
from fractions import Fraction

import numpy as np

from oracle import mxfp4


def test_hand_cases():
    row = np.zeros((1, 32))
    row[0, :9] = [6.0, -5.0, 0.25, 0.75, 2.5, 3.5, -0.2, 7.9, 0.3]
    codes, scales = mxfp4.quantize(row)
    assert scales.tolist() == [[127]]           # floor(log2 7.9) = 2
    assert mxfp4.values(codes, scales)[0, :9].tolist() == [6, -4, 0, 1, 2, 4, -0.0, 6, 0.5]
    assert codes[0, 0] == 7 | (6 + 8) << 4      # 6, then -5 to the even of -4 and -6
    codes, scales = mxfp4.quantize(np.zeros((2, 64)))
    assert not codes.any() and not scales.any()
    row = np.full((1, 64), 2.0 ** -140)
    row[0, 33] = np.inf
    codes, scales = mxfp4.quantize(row)
    assert scales.tolist() == [[0, 255]] and not codes.any()
    assert np.isnan(mxfp4.values(codes, scales)[0, 32:]).all()


def test_nearest_value_in_rationals():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(20, 64)) * np.exp2(rng.integers(-30, 30, (20, 64)))
    codes, scales = mxfp4.quantize(x)
    got = mxfp4.values(codes, scales)
    every = [Fraction(s) * Fraction(v) for v in (0, 1, 2, 3, 4, 6, 8, 12) for s in (Fraction(1, 2), Fraction(-1, 2))]
    for m in range(20):
        for b in range(2):
            peak = max(abs(Fraction(v)) for v in x[m, 32 * b:32 * b + 32])
            step = Fraction(2) ** (int(scales[m, b]) - 127)
            assert 4 * step <= peak < 8 * step
            for k in range(32 * b, 32 * b + 32):
                best = min(abs(Fraction(x[m, k]) / step - v) for v in every)
                assert abs(Fraction(x[m, k]) / step - Fraction(got[m, k]) / step) == best


def test_linear_is_the_product_of_the_values():
    rng = np.random.default_rng(1)
    c = rng.integers(0, 256, (3, 32), dtype=np.uint8)
    w = rng.integers(0, 256, (5, 32), dtype=np.uint8)
    cs, ws = (rng.integers(120, 135, (n, 2), dtype=np.uint8) for n in (3, 5))
    z, y, size = mxfp4.linear64(c, cs, w, ws)
    a, b = mxfp4.values(c, cs), mxfp4.values(w, ws)
    for m in range(3):
        for n in range(5):
            assert Fraction(z[m, n]) == sum(Fraction(p) * Fraction(q) for p, q in zip(a[m], b[n]))
    assert np.all(size >= np.abs(y))
