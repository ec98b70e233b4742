"""The fractions of a turn of dustin_norm_rope, compiled for the host, against whole
numbers of any length."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from _turns import INV_2PI, turn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def turn_of(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("turns")
    src = d / "turns.cpp"
    src.write_text('#include "turns.h"\nextern "C" uint64_t turn_of(uint32_t x) { return dustin::turn_of(x); }\n')
    so = str(d / "turns.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sparse_kv_verify_gb300", "csrc"), str(src), "-o", so], check=True)
    f = ctypes.CDLL(so).turn_of
    f.restype, f.argtypes = ctypes.c_uint64, [ctypes.c_uint32]
    return f


def test_pi_by_hand():
    assert abs(float(INV_2PI) - 1 / (2 * np.pi)) < 1e-16 and float(turn(2 * np.pi, 1000)) == pytest.approx(
        1000 * (float(np.float32(2 * np.pi)) / (2 * np.pi) - 1), abs=1e-12)


def far(turn_of, freq, pos):
    """How far the angle is off, in turns."""
    f = np.float32(freq)
    got = turn_of(int(f.view(np.uint32))) * pos % (1 << 64)
    off = (got - int(turn(f, pos) * (1 << 64))) % (1 << 64)
    return min(off, (1 << 64) - off) * 2.0 ** -64


def test_turns_at_the_farthest_positions(turn_of):
    rng = np.random.default_rng(0)
    freqs = np.concatenate([2.0 ** rng.uniform(-149, 39, 400), 10000.0 ** (-np.arange(64) / 64), [0.0, 1.0, 2 ** 39 * (1 - 2 ** -24),
                            1e-45, 1.1754944e-38, 2 * np.pi, 2 * np.pi * 1000]]).astype(np.float32)
    for f in np.concatenate([freqs, -freqs]):
        for pos in (1, 3, 2 ** 20, 2 ** 31 - 1, -2 ** 31):
            # half a unit of 2^-64 and |freq| 2^-105 per position, and the reference's own cut to 64 bits
            assert far(turn_of, f, pos) <= abs(pos) * (2.0 ** -65 + abs(float(f)) * 2.0 ** -105) + 2.0 ** -63, (f, pos)
            assert far(turn_of, f, pos) <= 2.0 ** -33, (f, pos)


def test_any_bits_give_a_fraction(turn_of):
    """Frequencies out of range, infinities and NaN: no shift past the word's width."""
    for f in (2.0 ** 39, 2.0 ** 100, np.finfo(np.float32).max, np.inf, np.nan, -np.inf):
        bits = int(np.float32(f).view(np.uint32))
        assert 0 <= turn_of(bits) < 1 << 64
