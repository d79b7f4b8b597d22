"""The kernel's own angle arithmetic (csrc/rotary_angle.cuh), compiled for the host, against
exact arithmetic."""
import math
import os
import random
import shutil
import struct
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
RATES = [0.0, 1.0, 0.5, 10000.0 ** -0.3, 1e-4, 1e-12, -0.75, -1.0, 6.25, 7.0, 7.25, -7.25,
         20 * math.pi, -20 * math.pi, 2.0 ** 20 * math.pi, -1e9, 1e25, 1e-300]


@pytest.fixture(scope="module")
def phases(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("host") / "rotary_angle")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run([cc, "-O2", "-std=c++17", "-o", exe, os.path.join(ROOT, "tests", "host", "rotary_angle.cpp"),
                    "-I", os.path.join(ROOT, "differentiable_image_quality_gb300", "csrc"),
                    "-I", os.path.join(cuda, "include")], check=True)

    def run(kind, cases):
        text = "".join(f"{kind} {x if kind == 'i' else float(x).hex()} {f.hex()}\n" for x, f in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        return [int(v) for v in out.split()]

    return run


def off(phase, x, f):
    """Turns between the phase and the exact angle."""
    d = (Fraction(phase, 2 ** 64) - Fraction(x) * Fraction(f) / (2 * PI)) % 1
    return min(d, 1 - d)


def bound(x, f):
    """1 / (2 pi) and the quotient round to 53 bits, 2^-52 of it together; the fraction of a
    turn and the part of a position are cut at 2^-64, their product once more."""
    turns = abs(Fraction(f)) / (2 * PI)
    size = abs(Fraction(x))
    return size * turns * Fraction(2) ** -52 + (size + turns + 2) * Fraction(2) ** -63


def single(x):
    return struct.unpack("f", struct.pack("f", x))[0]


def test_whole_positions(phases):
    rng = random.Random(1)
    at = [0, 1, -1, 77, -4096, 10 ** 6 + 3, 2 ** 31 - 1, -2 ** 40, 2 ** 63 - 1, -2 ** 63] + \
        [rng.randrange(-2 ** 40, 2 ** 40) for _ in range(50)]
    cases = [(x, f) for x in at for f in RATES]
    for (x, f), phase in zip(cases, phases("i", cases)):
        assert off(phase, x, f) <= bound(x, f), (x, f)


def test_float_positions(phases):
    rng = random.Random(2)
    at = [0.0, 0.5, -0.5, 0.375, -0.375, 1.0, -1.0, 2.0 ** -40, single(0.1), 1e4 + 0.25, -4096.5,
          2.0 ** 24 + 2, 2.0 ** 62, -(2.0 ** 62), single(8.9e18)]
    at += [single(rng.uniform(-1, 1)) for _ in range(60)] + [single(rng.uniform(-2000, 2000)) for _ in range(60)]
    cases = [(x, f) for x in at for f in RATES]
    for (x, f), phase in zip(cases, phases("f", cases)):
        assert off(phase, x, f) <= bound(x, f), (x, f)


def test_one_angle_for_a_whole_number_of_either_type(phases):
    cases = [(x, f) for x in (0, 1, -1, 3, -77, 2 ** 24, -2 ** 24) for f in RATES]
    assert phases("i", cases) == phases("f", cases)


def test_signs(phases):
    """The angle is odd in the position and in the frequency."""
    cases = [(single(0.1 * n), f) for n in range(1, 20) for f in RATES if f > 0]
    there = phases("f", cases)
    for a, b in ((-1, 1), (1, -1)):
        back = phases("f", [(a * x, b * f) for x, f in cases])
        assert all((p + q) % 2 ** 64 == 0 for p, q in zip(there, back))
    assert phases("f", [(-x, -f) for x, f in cases]) == there
