"""kv_append's quotient x / scale (a rounded reciprocal, a product, one corrected step), as a model of its float32
arithmetic: the E4M3 code must be that of the correctly rounded quotient.

Codes change at numbers of at most five significant bits (halfway points between two codes), so it is enough that
the computed quotient lies on the same side of every such number as the rounded one.  Powers of two change nothing
within the kernel's ranges, so mantissas suffice: scales in [1, 2), borders in [1, 2), and every x within four units of
scale * border (further away the quotient is more than a unit from the border, and the model's is within one)."""
import numpy as np
import pytest


def _f32(v):
    return v.astype(np.float32).astype(np.float64)


def wrong_side(mantissas):
    """How many (scale, x) end on the wrong side of a border; mantissas: integers in [0, 2^23)."""
    s = (mantissas + (1 << 23)).astype(np.float64) * 2.0 ** -23
    inv = _f32(1.0 / s)                         # (float64 quotients round correctly to float32: 53 > 2 * 24 + 1)
    bad = 0
    for b in range(16, 32):
        border = b / 16.0
        x0 = _f32(s * border)
        unit = np.where(x0 >= 2, 2.0 ** -22, 2.0 ** -23)
        for d in range(-4, 5):
            x = x0 + d * unit
            is_f32 = _f32(x) == x
            y = _f32(x * inv)                   # the product of two float32 is exact in float64
            r = _f32(x - s * y)                 # fmaf(-s, y, x): exact in float64, rounded once
            # fmaf(r, inv, y): y + t in float64 with its error, which decides where float64 ends halfway
            t = r * inv
            q = y + t
            back = q - y
            e = (y - (q - back)) + (t - back)
            ulp = np.where(np.abs(q) >= 2, 2.0 ** -22, np.where(np.abs(q) >= 1, 2.0 ** -23, 2.0 ** -24))
            low = np.floor(q / ulp) * ulp
            halfway = (q - low == ulp / 2) & (e != 0)
            got = np.where(halfway, np.where(e > 0, low + ulp, low), _f32(q))
            want = _f32(x / s)
            bad += int((is_f32 & (np.sign(got - border) != np.sign(want - border))).sum())
    return bad


@pytest.mark.parametrize("part", range(4))
def test_codes_are_those_of_the_rounded_quotient(part):
    """A spread of the 2^23 mantissas (all of them were checked once)."""
    assert wrong_side(np.arange(part, 1 << 23, 4 * 67, dtype=np.int64)) == 0


def test_scales_near_the_borders_own_multiples():
    """Where x / scale can come closest to halfway between a border and its neighbour: mantissas next to multiples of
    2^20 (M = border +- half a unit is odd, so scale * M is near a float32 only there)."""
    at = np.concatenate([(k << 20) + np.arange(-64, 65) for k in range(9)])
    assert wrong_side(at[(at >= 0) & (at < 1 << 23)]) == 0
