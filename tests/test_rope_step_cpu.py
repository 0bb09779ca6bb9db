"""The 64-bit fixed-point turns of a pair against exact rationals: the angle after
2^31 positions, for frequencies of both signs and of every size that is allowed."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# 2 pi to 50 digits
TWO_PI = Fraction(62831853071795864769252867665590057683943387987502, 10 ** 49)
TURN = 1 << 64


@pytest.fixture(scope="module")
def step(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rope") / "rope_step.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ffp-contract=off", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "grouped_query_decode_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "rope_step_on_host.cpp"), "-o", so], check=True)
    fn = ctypes.CDLL(so).rope_step
    fn.restype, fn.argtypes = ctypes.c_ulonglong, [ctypes.c_double]
    return fn


def off(step, f, t):
    """Radians by which the angle at position t differs from t f, modulo a turn."""
    got = Fraction(step(f) * t % TURN, TURN)
    d = (got - Fraction(f) * t / TWO_PI) % 1
    return float(min(d, 1 - d) * TWO_PI)


# Truncations to 2^-64 turns, two of them, 2^31 times: 2^-32 turns, 2^-29.3 radians.
# What rest lacks, 2^-104 of f, is below that up to f = 1e15 (2^50, times 2^31): 2^-23.
SIZES = [2.0 ** -40, 3.1e-7, 1e-6, 1.3e-4, 0.01, 0.1, 1 / 3, 1.0, 2.5, math.pi, 6.283185307179586, 100.0, 12345.678]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("t", [1, 12345, (1 << 31) - 1, -(1 << 31)])
def test_angles_at_every_position(step, t, sign):
    for f in SIZES + [10000.0 ** (-2 * i / 128) for i in range(64)]:
        assert off(step, sign * f, t) < 2.0 ** -29, (sign * f, t, off(step, sign * f, t))


@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_frequencies(step, sign):
    for f in (1e9 + 0.1, 1e12 / 3, 1e15):
        assert off(step, sign * f, (1 << 31) - 1) < 2.0 ** -22


def test_the_sign_turns_the_other_way(step):
    for f in SIZES:
        assert (step(f) + step(-f)) % TURN == 0
    assert step(0.0) == 0 and step(-0.0) == 0
