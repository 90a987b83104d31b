"""The rotation plan's words, f / (2 pi) in 2^-64 turns, against integer
arithmetic of 2400 bits: any f64 frequency, far above 1 too (host work)."""
import math
from fractions import Fraction

import numpy as np
import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_abi import L  # noqa: F401  (the built library as a fixture)

BITS = 2400


def _atan_inverse(n):
    """atan(1 / n) in 2^-(BITS + 64), each term truncated."""
    term = total = (1 << BITS + 64) // n
    k, sign = 1, -1
    while term:
        term //= n * n
        k += 2
        total += sign * (term // k)
        sign = -sign
    return total


# pi in 2^-(BITS + 64); Machin's formula, a few thousand truncations
PI = 16 * _atan_inverse(5) - 4 * _atan_inverse(239)


def turns64(f, pos=1):
    """pos * f / (2 pi) modulo 1 in 2^-64, as a Fraction (off by less than 2^-200)."""
    v = Fraction(f) * pos * (1 << BITS + 64) / (2 * PI)
    return (v - math.floor(v)) * 2 ** 64


def off(word, want):
    d = abs(word - want)
    return min(d, 2 ** 64 - d)


FREQ = [0.0, 5e-324, 1e-300, 2.0 ** -76, 1e-12, 1 / 3, 0.5, 1.0, 2 * math.pi, 7.0, 1000.0, 1e6 + 0.1, 2.0 ** 53 + 2, 1e19,
        1.5e30, 6e200, 1.7976931348623157e308]


def test_words_are_the_nearest_for_any_frequency(L):
    rng = np.random.default_rng(1)
    freq = FREQ + [float(2.0 ** rng.uniform(-70, 1020) * rng.uniform(1, 2)) for _ in range(128 - len(FREQ))]
    plan = te.rope_axes_plan(256, (256,), freq=freq)
    for f, word in zip(freq, plan.turn):
        # half a unit, and what the bits past the 128 that are used may add: 2^-11
        assert off(word, turns64(f)) <= Fraction(1, 2) + Fraction(1, 2048), f


@pytest.mark.parametrize("theta,whole", [(10000.0, False), (10000.0, True), (1e-6, False), (5e5, True)])
def test_words_of_the_powers(L, theta, whole):
    sec = (64, 90, 102)
    plan = te.rope_axes_plan(256, sec, theta=theta, whole=whole)
    p = 0
    for s in sec:
        for i in range(s // 2):
            f = theta ** (-2.0 * p / sum(sec) if whole else -2.0 * i / s)
            # the power may be the neighbouring f64 of another libm's
            near = [turns64(v) for v in (math.nextafter(f, 0), f, math.nextafter(f, math.inf))]
            assert min(off(plan.turn[p], w) for w in near) <= 1
            p += 1


def test_powers_past_an_f64_are_refused_and_the_plan_is_left(L):
    import ctypes
    plan = te.rope_axes_plan(64, (64,))
    before = bytes(plan)
    sec = (ctypes.c_int32 * 1)(256)
    assert L.te_rope_axes_init(ctypes.byref(plan), 256, 1, sec, 5e-324, 0, te.TE_ROPE_ADJACENT, None) == te.TE_EINVAL
    assert bytes(plan) == before
