"""Pins of the rotary oracle (CPU, fp64): rotation matrices, exact angles, transposes."""

from fractions import Fraction

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_rotation_is_the_matrix_of_its_angle(interleaved):
    rng = np.random.default_rng(0)
    cos, sin = oracle.rotary_tables(40, 16)
    x = rng.standard_normal((5, 2, 24))
    pos = np.array([0, 3, 39, 17, -1])
    y = oracle.rotary_embed(x, cos, sin, pos, interleaved=interleaved)
    for n, p in enumerate(pos):
        m = np.eye(24)
        for i in range(8):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
            angle = max(p, 0) * 10000.0 ** (-2 * i / 16)
            m[[a, a, b, b], [a, b, a, b]] = np.cos(angle), -np.sin(angle), np.sin(angle), np.cos(angle)
        np.testing.assert_allclose(y[n], x[n] @ (m if p >= 0 else np.eye(24)).T, atol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_transpose(interleaved):
    rng = np.random.default_rng(1)
    cos, sin = oracle.rotary_tables(64, 32, amplitude=1.3)
    x, g = rng.standard_normal((2, 64, 3, 48))
    pos = rng.permutation(64)
    f = lambda z, **kw: oracle.rotary_embed(z, cos, sin, pos, interleaved=interleaved, **kw)  # noqa: E731
    assert np.isclose((f(x) * g).sum(), (x * f(g, inverse=True)).sum())
    np.testing.assert_allclose(f(f(x), inverse=True)[..., :32], 1.69 * x[..., :32], atol=1e-12)


def test_products_depend_on_the_distance_only():
    rng = np.random.default_rng(2)
    cos, sin = oracle.rotary_tables(1000, 64, base=5e5)
    q, k = rng.standard_normal((2, 1, 1, 64))
    dot = lambda a, b: (oracle.rotary_embed(q, cos, sin, [a]) * oracle.rotary_embed(k, cos, sin, [b])).sum()  # noqa: E731
    assert np.isclose(dot(30, 7), dot(930, 907))


def test_frequencies_of_a_stretched_context():
    plain = oracle.rotary_frequencies(128, base=1e4)
    assert np.allclose(plain, [float(Fraction(1)) * 1e4 ** (-i / 64) for i in range(64)])
    np.testing.assert_allclose(oracle.rotary_frequencies(128, base=1e4, factor=4.0), plain / 4)
    f = oracle.rotary_frequencies(128, base=1e4, factor=8.0, original_length=4096, slow=1.0, fast=32.0)
    turns = 4096 * plain / (2 * np.pi)
    np.testing.assert_array_equal(f[turns >= 32], plain[turns >= 32])
    np.testing.assert_allclose(f[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    share = (plain[mid] - f[mid]) / (plain[mid] - plain[mid] / 8)   # of the way to the stretched one
    np.testing.assert_allclose(share, (32 - turns[mid]) / 31)
    assert (np.diff(f) < 0).all()
