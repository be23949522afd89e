"""Frequencies as fractions of a turn, against exact fractions on the host.

A frequency f is held as n / 2^64 turns.  2 pi and the quotient |f| / 2 pi round to 53 bits each, 2^-53 of it, whole turns come off exactly, and
the fraction rounds to half of 2^-64: at position p the angle is off by at most |p| (2^-65 + 1.001 * 2^-52 |f| / 2 pi) turns, whatever the frequency's size
and sign.
"""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from llama_transformer_decode_gb300 import _native

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module")
def lib():
    try:
        return _native.load()
    except OSError as e:
        pytest.skip(f"cannot load the CUDA runtime here: {e}")


def worst(lib, freqs):
    """Largest error over its bound, of each frequency at some positions."""
    n = len(freqs)
    plan = _native.L2RopePlan()
    assert lib.l2_rope_plan(ctypes.byref(plan), 2 * n, 0, (ctypes.c_double * n)(*freqs), 1.0) == 0
    most = Fraction(0)
    for f, turns in zip(freqs, plan.turns):
        turn = Fraction(f) / TWO_PI
        for p in (1, -1, 3, 8191, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
            off = (Fraction(turns, 1 << 64) - turn) * p % 1
            off = min(off, 1 - off)
            most = max(most, off / (abs(p) * (Fraction(1, 1 << 65) + Fraction(1001, 1000) * Fraction(1, 1 << 52) * abs(turn))))
    return float(most)


@pytest.mark.parametrize("freqs", [
    [1.0, 0.5, 1e-3, 1e-6],
    [-1.0, -0.5, -1e-3, -1e-6, -1e-7, -1e-9],           # turning back, as slow pairs do
    [1e-9, 1e-12, -1e-12, 1e-18, -1e-18, 1e-30, -1e-300, 0.0, -0.0],
    [7.5, -7.5, 100.0, -100.0, 1e9, -1e9, 2 ** 40 + 0.3, -(2 ** 40 + 0.3)],
    [2 * float(TWO_PI), -2 * float(TWO_PI), float(TWO_PI) * (1 - 2 ** -53), -float(TWO_PI) * (1 - 2 ** -53)],
])
def test_far_positions_are_off_by_what_is_stated(lib, freqs):
    assert worst(lib, freqs) <= 1


@pytest.mark.parametrize("base", [1e4, 5e5, 1e7])
def test_a_models_own_frequencies(lib, base):
    f = (ctypes.c_double * 64)()
    assert lib.l2_rope_freqs(128, base, 0, 1.0, 0.0, 0.0, 0.0, f) == 0
    assert worst(lib, list(f)) <= 1
    assert worst(lib, [-x for x in f]) <= 1


def test_random_frequencies_of_either_sign(lib):
    rng = np.random.default_rng(3)
    for _ in range(20):
        f = np.exp(rng.uniform(np.log(1e-14), np.log(1e4), 128)) * rng.choice([-1, 1], 128)
        assert worst(lib, f.tolist()) <= 1
