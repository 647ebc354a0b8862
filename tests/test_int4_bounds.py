"""How far a 4-bit row may be from the row that was written: the bounds that the header promises, from the definition in
exact arithmetic, at scales where they are nearly reached (CPU)."""

from fractions import Fraction

import numpy as np
import pytest

import oracle.int4 as O4

# half a step of the type: relative to normal values, absolute for subnormal ones, and its smallest normal value
TYPES = {"f16": (2.0 ** -11, 2.0 ** -25, 2.0 ** -14), "bf16": (2.0 ** -8, 2.0 ** -134, 2.0 ** -126)}


def _group(lo, top, dtype):
    """64 values of T from lo to lo + top (as near as T comes), the ends included."""
    x = O4.round_to(np.float32(lo) + np.linspace(0, 1, 64).astype(np.float32) * np.float32(top), dtype)
    return np.clip(x, x[0], x[-1])


def _excess(x, dtype):
    """(x_max - (z + 15 s), s) and the largest |x - (z + c s)| of the elements up to z + 15 s, exactly."""
    codes, pairs = O4.quantize(x[None], dtype)
    s, z = Fraction(float(pairs[0, 0, 0])), Fraction(float(pairs[0, 0, 1]))
    exact = [Fraction(float(v)) for v in x]
    inside = [abs(v - (z + int(c) * s)) for v, c in zip(exact, codes[0]) if v <= z + 15 * s]
    return max(exact) - (z + 15 * s), s, max(inside)


def _promised(s, dtype):
    relative, subnormal, normal = TYPES[dtype]
    return 15 * (s * Fraction(relative) if s >= Fraction(normal) else Fraction(subnormal))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rounded_scales_stay_inside_the_promised_bounds(dtype):
    """Ranges around 15 steps of scales next to the lower end of a binade (where half a step is largest), in the middle
    of the type and where the scale is subnormal. fp32's own roundings are 2^-20 of a bound at most."""
    relative, subnormal, normal = TYPES[dtype]
    past_old = 0                                  # how often half of the promise would not have held
    rng = np.random.default_rng(3)
    scales = [2.0 ** e * (1 + f * relative) for e in (-3, 0, 4) for f in (0.5, 0.9, 0.99, 1, 1.5, 2.9, 2.99)]
    scales += [subnormal * f for f in (0.5, 0.9, 1, 1.5, 2.5, 2.9, 2.99, 6.9, 14.9)] + [normal * 1.25]
    for s in scales:
        for lo in (0.0, -float(s) * 7, -float(s) * 15):
            x = _group(lo, 15 * s * rng.uniform(0.999, 1.0), dtype)
            excess, rounded, inside = _excess(x, dtype)
            slack = 1 + Fraction(2) ** -20
            assert excess <= _promised(rounded, dtype) * slack
            assert inside <= rounded / 2 * slack
            past_old += excess > _promised(rounded, dtype) / 2
    assert past_old >= 3


def test_a_range_too_small_for_a_scale_reads_as_its_offset():
    """fp16: a range of 7 smallest steps has a scale of 7/15 of one, which rounds to 0; 15 2^-25 covers it."""
    x = np.zeros(64)
    x[1] = 7 * 2.0 ** -24
    codes, pairs = O4.quantize(x[None], "f16")
    assert pairs[0, 0, 0] == 0 and not codes.any()
    excess, s, _ = _excess(x, "f16")
    assert s == 0 and 0 < excess <= 15 * Fraction(2.0 ** -25)
