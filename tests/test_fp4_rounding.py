"""The quotient that the 4-bit cache's quantiser takes (CPU only): x * hi +
x * lo with hi + lo = 1 / d decides every border between two codes exactly,
whatever last bit the reciprocal's approximation has."""

import numpy as np

from oracle import fp4 as F

f32 = np.float32


def fma(a, b, c):
    """One rounding: the products below have at most 48 bits and stay exact in extended precision."""
    return f32(np.longdouble(a) * np.longdouble(b) + np.longdouble(c))


def recip(d, ulp):
    r = np.array([f32(1) / f32(d)], f32)
    hi = (r.view(np.int32) + ulp).view(f32)[0]
    return hi, f32(fma(-f32(d), hi, f32(1)) * hi)


def times(x, hi, lo):
    return fma(x, hi, f32(x * lo))


def test_every_border_between_codes_is_exact():
    mids = (F.E2M1[1:] + F.E2M1[:-1]) / 2
    for s in F.e4m3_table()[1:]:
        for ulp in (-1, 0, 1):  # the approximation is off by at most one
            hi, lo = recip(s, ulp)
            for m in mids:
                assert times(f32(m * s), hi, lo) == f32(m)


def test_neighbours_of_a_border_stay_on_their_side():
    """11-bit numbers next to border * s (fp16 and bf16 have at most 11 bits)."""
    mids = (F.E2M1[1:] + F.E2M1[:-1]) / 2
    for s in F.e4m3_table()[1:]:
        hi, lo = recip(s, 0)
        for m in mids:
            x = m * s
            step = 2.0 ** (np.floor(np.log2(x)) - 10)
            assert times(f32(x + step), hi, lo) > f32(m) > times(f32(x - step), hi, lo)


def test_every_border_between_scales_is_exact():
    hi = f32(1) / f32(6)
    lo = f32(1 / 6 - float(hi))
    t = F.e4m3_table()
    for a, b in zip(t[:-1], t[1:]):
        m = (a + b) / 2
        assert times(f32(6 * m), hi, lo) == f32(m)
        step = 2.0 ** (np.floor(np.log2(6 * m)) - 10)
        assert times(f32(6 * m + step), hi, lo) > f32(m) > times(f32(6 * m - step), hi, lo)
