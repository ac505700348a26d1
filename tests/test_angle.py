"""Cosine and sine of a fraction of a turn (csrc/angle.h), built by the host compiler, against long
double: the bound that the file states, and no worse on average than factors rounded from fp64."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "angle.h"
extern "C" void factors(const unsigned long long* turn, long long n, float scale, float* c, float* s) {
    for (long long i = 0; i < n; ++i) infllmv2::cos_sin_of_turn(turn[i], scale, c + i, s + i);
}
"""


@pytest.fixture(scope="module")
def factors(tmp_path_factory):
    path = tmp_path_factory.mktemp("angle")
    src, so = path / "angle.cpp", path / "angle.so"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "block_sparse_long_infllm_gb300", "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-Werror", "-ffp-contract=off", "-shared",
                    "-fPIC", "-I", inc, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def call(turn, scale):
        c, s = np.empty(len(turn), dtype=np.float32), np.empty(len(turn), dtype=np.float32)
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        lib.factors(p(turn), ctypes.c_longlong(len(turn)), ctypes.c_float(scale), p(c), p(s))
        return c, s
    return call


def _exact(turn, scale):
    """In fp64 from the exact quarter and rest: the rest of 62 bits is rounded to 53, 2^-55 of a turn."""
    quarter = ((turn + np.uint64(1 << 61)) >> np.uint64(62)).astype(np.int64)
    rest = (turn - (quarter.astype(np.uint64) << np.uint64(62))).view(np.int64)
    x = rest.astype(np.float64) * (2.0 * np.pi / 2.0 ** 64)
    c, s = np.cos(x), np.sin(x)
    cs = np.choose(quarter & 3, [c, -s, -c, s]), np.choose(quarter & 3, [s, c, -s, -c])
    return [np.float64(np.float32(scale)) * v for v in cs]


def _turns(rng, n):
    some = rng.integers(0, 1 << 64, n, dtype=np.uint64)
    edges = [(e << 61) + d for e in range(8) for d in (-2 ** 40, -2 ** 31, -1, 0, 1, 2 ** 30, 2 ** 31, 2 ** 40)]
    small = [1 << k for k in range(64)]
    return np.concatenate([some, np.array([x % (1 << 64) for x in edges + small], dtype=np.uint64)])


@pytest.mark.parametrize("scale", [1.0, 1.2079441541679836, 0.75, 1e-3, 3.9])
def test_factors_are_rounded_about_once(factors, scale):
    turn = _turns(np.random.default_rng(1), 400000)
    got, ref = factors(turn, scale), _exact(turn, scale)
    scale = float(np.float32(scale))
    for g, r in zip(got, ref):
        half_unit = np.spacing(np.abs(r).astype(np.float32)).astype(np.float64) / 2
        # beyond half a unit: cos - 1 rounded to 2^-26, the angle's cut below 2^-31, the series below 2^-28, and
        # the sums inside them (terms up to 0.08 and 0.016 rounded at 2^-25 of them, a few of each)
        assert np.all(np.abs(g - r) <= half_unit + scale * (2.0 ** -26 + 2.0 ** -28 + 2.0 ** -28))


@pytest.mark.parametrize("scale", [1.0, 1.2079441541679836])
def test_factors_lose_little_against_fp64(factors, scale):
    """On average at most a tenth more than factors computed in fp64 and rounded once: half a unit's mean
    square is 1/12, what comes before it (at most 2^-26 against a unit of 2^-24, mean square 1/192 for
    half of the factors) adds a few hundredths."""
    turn = np.random.default_rng(2).integers(0, 1 << 64, 1 << 20, dtype=np.uint64)
    got, ref = factors(turn, scale), _exact(turn, scale)
    for g, r in zip(got, ref):
        once = np.sqrt(np.mean((r.astype(np.float32) - r) ** 2))
        assert np.sqrt(np.mean((g - r) ** 2)) <= 1.1 * once


def test_quarters_are_exact(factors):
    turn = np.array([0, 1 << 62, 2 << 62, 3 << 62], dtype=np.uint64)
    c, s = factors(turn, 1.5)
    assert c.tolist() == [1.5, 0.0, -1.5, 0.0] and s.tolist() == [0.0, 1.5, 0.0, -1.5]
