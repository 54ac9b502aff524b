"""The arithmetic by which the quantiser rounds (a quotient formed with a reciprocal of up to one unit in the
last place off, 1 + 2^-17 times too large, its last 8 bits dropped) gives the rounding of the exact quotient,
ties included: every bf16 significand over every E4M3 fraction, and every bf16 significand over 6, on the CPU
in float32 against exact comparisons in float64."""
import numpy as np

import _quant_ref as ref

ABOVE = np.float32(1 + 2.0 ** -17)


def _snapped(x, factor):
    v = (x * factor).astype(np.float32)
    return (v.view(np.uint32) & np.uint32(0xffffff00)).view(np.float32).astype(np.float64)


def test_codes():
    for fraction in range(8, 16):
        s = fraction / 8.0
        r = np.float32(1 / s)
        for near in (r, np.nextafter(r, np.float32(0)), np.nextafter(r, np.float32(9))):
            for e in range(-14, 4):
                x = (np.arange(128, 256) / 128.0 * 2.0 ** e).astype(np.float32)
                exact = x.astype(np.float64) / s
                got = ref.nearest(_snapped(x, np.float32(near * ABOVE)), ref.E2M1)
                assert np.array_equal(got, ref.nearest(exact, ref.E2M1)), (fraction, e)


def test_block_scales():
    for e in range(-16, 11):
        x = (np.arange(128, 256) / 128.0 * 2.0 ** e).astype(np.float32)
        got = ref.nearest(_snapped(x, np.float32(ABOVE / np.float32(6))), ref.E4M3)
        assert np.array_equal(got, ref.nearest(x.astype(np.float64), 6 * ref.E4M3)), e
