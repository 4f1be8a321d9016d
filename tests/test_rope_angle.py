"""The position rotation's angle in fp32 (csrc/rope_angle.cuh), compiled for the host, against extended precision."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import speculative_decoding_verification_72_gb300 as sv

CSRC = os.path.join(os.path.dirname(sv.__file__), "csrc")


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("rope")
    (at / "t.cpp").write_text('#include "rope_angle.cuh"\nextern "C" void turns(const int* p, const float* f, float* to, long n) '
                              "{ for (long i = 0; i < n; ++i) to[i] = sv::rope_turn(p[i], f[i]); }\n")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", f"-I{CSRC}", str(at / "t.cpp"), "-o",
                    str(at / "t.so")], check=True)
    lib = ctypes.CDLL(str(at / "t.so"))
    lib.turns.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_long]

    def call(p, f):
        p, f = np.ascontiguousarray(p, np.int32), np.ascontiguousarray(f, np.float32)
        to = np.empty(len(p), np.float32)
        lib.turns(p.ctypes.data, f.ctypes.data, to.ctypes.data, len(p))
        return to

    return call


@pytest.mark.skipif(np.finfo(np.longdouble).nmant < 63, reason="no extended precision")
@pytest.mark.parametrize("bits,bound,size", [(12, 2.0 ** -24, 1.0), (24, 1.8 * 2.0 ** -24, 1.0), (31, 2.0 ** -17, 64.0)])
@pytest.mark.parametrize("base", [1.0, 0.9478, 0.5, 0.1, 1e-3, 1e-6])
def test_turns(turns, bits, bound, size, base):
    """Bounds as derived in the header: below 2^12 positions there is one product, and what it leaves is below 2^-12, so one
    sum is rounded to 2^-25 and the rest to 2^-36."""
    rng = np.random.default_rng(bits)
    n = 400_000
    p = rng.integers(0, 1 << bits, n)
    p[:3] = 0, 1, (1 << bits) - 1
    f = (base * (1 - 0.5 * rng.random(n) * (np.arange(n) % 2))).astype(np.float32)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    want = p.astype(np.longdouble) * f.astype(np.longdouble) / two_pi
    got = turns(p, f)
    off = got.astype(np.longdouble) - want
    off = np.abs(off - np.rint(off))
    assert np.abs(got).max() <= size and off.max() <= bound + 2.0 ** -34, float(off.max())


def test_no_turn_at_the_start(turns):
    assert (turns(np.zeros(4), [1.0, 0.3, 1e-30, 0.0]) == 0).all() and turns([1 << 30], [0.0])[0] == 0
