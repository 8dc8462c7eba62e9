"""Signs and borders of the 4-bit cache's quotients (CPU only, an emulation of
the kernel's arithmetic): x * hi + x * lo with 0 <= lo keeps the sign of x, that
of a zero too, and decides every 16-bit x as the exact quotient does."""

import numpy as np

from oracle import fp4 as F
from tests.test_fp4_rounding import f32, fma, times

MIDS = (F.E2M1[1:] + F.E2M1[:-1]) / 2


def recip(d, ulp):
    """hi two steps below an approximation that is off by `ulp` steps, lo = what is left of 1 / d."""
    r = np.array([f32(1) / f32(d)], f32)
    hi = (r.view(np.int32) + ulp - 2).view(f32)[0]
    return hi, f32(fma(-f32(d), hi, f32(1)) * hi)


def magnitudes():
    """Every finite magnitude of fp16 and bf16 that a block's scale leaves in range."""
    h = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    b = (np.arange(0x7F80, dtype=np.uint32) << 16).view(f32).astype(np.float64)
    x = np.unique(np.concatenate([h, b]))
    return x[x <= 6.25 * 448]


def test_a_zero_keeps_its_sign_under_every_scale():
    for s in F.e4m3_table()[1:]:
        for ulp in (-1, 0, 1):  # the approximation is off by at most one
            hi, lo = recip(s, ulp)
            assert lo >= 0
            y = times(np.array([-0.0, 0.0], f32), hi, lo)
            assert np.signbit(y).tolist() == [True, False] and not y.any()


def test_every_16_bit_number_is_decided_as_its_exact_quotient():
    x = magnitudes()
    for s in F.e4m3_table()[1:]:
        v = x[x <= 6.5 * s]
        for ulp in (-1, 0, 1):
            hi, lo = recip(s, ulp)
            y = times(v.astype(f32), hi, lo).astype(np.float64)
            for side in ("left", "right"):  # below, on or above each border (their products with s are exact)
                assert np.array_equal(np.searchsorted(MIDS, y, side), np.searchsorted(MIDS * s, v, side))
            assert np.signbit(times((-v).astype(f32), hi, lo)).all()
