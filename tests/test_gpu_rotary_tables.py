"""GPU parity of the rotary tables, held to what the kernel's own steps allow.

In units of 2^-24, half a step of fp32 at 1, with u = r^2 and r in [-1, 1] eighths of a turn:
  r           conversion 1, sum of its two parts 1                                        2 relative
  sin side    S = s0 + u (s1 + ..): s0 1, its sum 1, a tenth of (s1 1, its sum 1, u 5)    2.7
              r S: r 2, the product 1                                                     5.7 relative
  cos side    A + u C, |u C| <= 0.31 A: A 1, the sum 1, u 5, c0 1, its sum 1,
              a twentieth of 7 behind it                                                  4.3 A
sin side values are at most 0.71 A: 4.1.  The fits, 2.4e-9 and 1.9e-10, and the angle, position * 2^-64
turns, are below a tenth.  So 5 units of the amplitude cover every value, and 6 relative ones a sine
of up to an eighth of a turn.  The exact values are of 60 digits.
"""

import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from tests._parity import to_np
from tests.test_rotary_turns import exact

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNIT = 2.0 ** -24


@pytest.fixture(scope="module")
def sba():
    import __graft_entry__

    __graft_entry__.build()
    import selected_block_attention_gb300 as m

    return m


def angles(positions, rot, base=1e4, factor=1.0, original_length=0, slow=1.0, fast=32.0):
    """Radians within a turn, [positions, rot / 2]."""
    getcontext().prec = 60
    turns = [exact(i, rot, base, factor, original_length, slow, fast) / 2 ** 64 for i in range(rot // 2)]
    return np.array([[2 * math.pi * float((t * int(p) + Decimal("0.5")) % 1 - Decimal("0.5")) for t in turns] for p in positions])


@pytest.mark.parametrize("length,rot", [(1, 16), (3, 128), (300, 48), (5000, 256), (1 << 24, 16)])
@pytest.mark.parametrize("kw", [dict(), dict(base=5e5, amplitude=0.5), dict(base=1.0), dict(factor=4.0),
                                dict(base=3e4, factor=8.0, original_length=2048, amplitude=1.2),
                                dict(factor=2.0, original_length=500, slow=0.0, fast=1.5, amplitude=3.7e4)])
def test_values(sba, length, rot, kw):
    cos, sin = sba.rotary_tables(length, rot, device=DEV, **kw)
    amplitude = kw.get("amplitude", 1.0)
    rng = np.random.default_rng(length)
    pos = np.unique(np.r_[0, min(1, length - 1), length - 1, max(0, length - 2), rng.integers(0, length, 40)])
    angle = angles(pos, rot, **{k: v for k, v in kw.items() if k != "amplitude"})
    at = torch.from_numpy(pos).to(DEV)
    for got, ref in ((cos, np.cos(angle)), (sin, np.sin(angle))):
        assert np.abs(to_np(got[at]) / amplitude - ref).max() <= 5 * UNIT
    # sines of small angles, relative
    got, small = to_np(sin[at]) / amplitude, (np.abs(angle) <= math.pi / 4) & (angle != 0)
    assert (np.abs(got[small] / np.sin(angle[small]) - 1) <= 6 * UNIT + 2.0 ** -64 * pos.max() / np.abs(angle[small])).all()
