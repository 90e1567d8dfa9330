"""The rotary tables' frequencies against 60 digits (no GPU).

A position up to 2^31 keeps its fraction of a turn to 2^-30 if a pair's turns a position are right to 2^-61.
The counts here are integers in steps of 2^-64 made from sums of two doubles: each of some 10 operations on
them, 128 more for the last pair, is off by at most 2^-100 of a value below 1 / 6, which is 2^-31 steps
in all (where fast / (fast - slow) <= 2 multiplies it), and the rounding by half a step: one step covers both.
In 53 bits the power alone can be off by 2^8 steps.
"""

import ctypes
import os
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")

CSRC = os.path.join(os.path.dirname(__file__), "..", "selected_block_attention_gb300", "csrc")
TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194989")
STEPS = 1


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    at = tmp_path_factory.mktemp("turns")
    src, lib = at / "turns.cpp", at / "turns.so"
    src.write_text('#include "rotary_turns.h"\n'
                   'extern "C" void turns(int rot, double base, double factor, int original, double slow, double fast,\n'
                   '                      unsigned long long* to) {\n'
                   '  sba::rotary_turns(rot, base, factor, original, slow, fast, to);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    fn = ctypes.CDLL(str(lib)).turns
    fn.argtypes = [ctypes.c_int] + [ctypes.c_double] * 2 + [ctypes.c_int] + [ctypes.c_double] * 2 + [ctypes.c_void_p]
    fn.restype = None
    return fn


def exact(i, rot, base, factor, original, slow, fast):
    """In steps of 2^-64 turns."""
    f = (-2 * Decimal(i) / rot * Decimal(base).ln()).exp() / TWO_PI
    keep = Decimal(0)
    if original:
        keep = min(Decimal(1), max(Decimal(0), (original * f - Decimal(slow)) / (Decimal(fast) - Decimal(slow))))
    return f * (keep + (1 - keep) / Decimal(factor)) * 2 ** 64


@pytest.mark.parametrize("rot", [16, 48, 128, 256])
@pytest.mark.parametrize("base", [1.0, 1.5, 1e4, 5e5, 1e6, 123456.789, 1e30, 1.7e308])
@pytest.mark.parametrize("factor,original,slow,fast", [(1.0, 0, 1.0, 32.0), (31.5, 0, 1.0, 32.0), (8.0, 16384, 1.0, 32.0),
                                                       (2.0, 500, 0.0, 1.5), (40.0, 4096, 16.0, 32.0), (1e9, 2 ** 31 - 1, 3.0, 1e8)])
def test_turns(turns, rot, base, factor, original, slow, fast):
    getcontext().prec = 60
    got = (ctypes.c_ulonglong * (rot // 2))()
    turns(rot, base, factor, original, slow, fast, got)
    for i in range(rot // 2):
        off = abs(got[i] - exact(i, rot, base, factor, original, slow, fast))
        assert off <= STEPS, f"pair {i}: {float(off):.3g} steps of 2^-64 turns"
