"""The head norm's angles in turns, on the host, against exact arithmetic."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import pytest

from precision_transformer_gemms_gb300 import build

SOURCE = r"""
#include "turns.h"
extern "C" uint64_t angle(double frequency, int64_t position) {
  const lpq::Turns t = lpq::turns_of(frequency);
  return t.high * (uint64_t)position + (lpq::is_far(position) ? lpq::low_part(t.low, position) : 0);
}
"""
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)


@pytest.fixture(scope="module")
def angle(tmp_path_factory):
    folder = tmp_path_factory.mktemp("turns")
    (folder / "turns.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + build.CSRC, str(folder / "turns.cpp"), "-o",
                    str(folder / "turns.so")], check=True)
    f = ctypes.CDLL(os.path.join(folder, "turns.so")).angle
    f.argtypes, f.restype = [ctypes.c_double, ctypes.c_int64], ctypes.c_uint64
    return f


FREQUENCIES = [1.0, 0.5, 3.0, 2 * math.pi, math.pi, 1e-3, 500000.0 ** (-126 / 128), 1e6 ** (-254 / 256), 2.0 ** -30, 1e-9, 1e-12, 2.0 ** -60,
               1e-25, 1e-40, 123456.789, 1e15, 1e300, 5e-324, 0.0]
POSITIONS = [0, 1, 2, 511, 100003, (1 << 31) - 1, 1 << 40, (1 << 45) + 12345, (1 << 50) - 1, (1 << 60) + 3, (1 << 63) - 1]


@pytest.mark.parametrize("frequency", [f * s for f in FREQUENCIES for s in (1, -1)])
def test_angles(angle, frequency):
    """The frequency in turns is off by its own and 1 / (2 pi)'s rounding, 2^-52 of itself, and
    by 2^-96 of a turn, 2^-33 at any position."""
    for position in [p * s for p in POSITIONS for s in (1, -1)] + [-(1 << 63)]:
        want = Fraction(frequency) * position / (2 * PI)
        error = (Fraction(angle(frequency, position), 1 << 64) - want) % 1
        error = min(error, 1 - error)
        assert error <= abs(want) / 2 ** 52 + Fraction(1, 1 << 33), (position, float(error), float(abs(want) / 2 ** 52))
