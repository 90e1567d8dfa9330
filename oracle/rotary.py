"""fp64 oracle: rotary tables and the rotation of heads by position.  (TEST INFRASTRUCTURE)

Pair i of the first ``rot_dim`` dimensions is a complex number that is multiplied by
``amplitude * exp(1j * position * f_i)``; its conjugate turns gradients back.
"""

from __future__ import annotations

import numpy as np


def rotary_frequencies(rot_dim, base=10000.0, factor=1.0, original_length=0, slow=1.0, fast=32.0):
    """Radians a position of each pair."""
    f = []
    for i in range(rot_dim // 2):
        w = float(base) ** (-2.0 * i / rot_dim)
        if original_length:
            turns = original_length * w / (2.0 * np.pi)
            keep = 1.0 if turns >= fast else 0.0 if turns <= slow else (turns - slow) / (fast - slow)
        else:
            keep = 0.0
        f.append(keep * w + (1.0 - keep) * w / factor)
    return np.array(f)


def rotary_tables(length, rot_dim, *, amplitude=1.0, **scaling):
    """cos and sin, ``[length, rot_dim / 2]``."""
    angle = np.arange(length, dtype=np.float64)[:, None] * rotary_frequencies(rot_dim, **scaling)
    return amplitude * np.cos(angle), amplitude * np.sin(angle)


def rotary_embed(x, cos, sin, positions, *, interleaved=False, inverse=False):
    """``x`` [..., H, D] with positions [...]; negative positions leave their token as it is."""
    x = np.array(x, dtype=np.float64)
    positions = np.asarray(positions)
    rot = 2 * np.asarray(cos).shape[1]
    first, second = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (
        np.arange(rot // 2), np.arange(rot // 2, rot))
    at = np.maximum(positions, 0)
    turn = (np.asarray(cos, np.float64)[at] + 1j * np.asarray(sin, np.float64)[at])[..., None, :]
    z = (x[..., first] + 1j * x[..., second]) * (np.conj(turn) if inverse else turn)
    y = x.copy()
    y[..., first], y[..., second] = z.real, z.imag
    return np.where((positions >= 0)[..., None, None], y, x)
