"""Pins of the paged-cache oracle (CPU): e4m3 rounding against torch's cast, the rotation as
a complex product, attention and selection against the contiguous oracles."""

import numpy as np
import pytest
import torch

import oracle
from oracle import paged


def test_e4m3_rounding_is_the_cast():
    """Every e4m3 value, every midpoint between neighbours (ties to even) and its two sides."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    vals = torch.unique(codes[codes.isfinite()])
    mid = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    want = x.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged.round_e4m3(x.numpy()), want)
    assert paged.round_e4m3(1e9) == 448.0 and paged.round_e4m3(-np.inf) == -448.0
    assert np.isnan(paged.round_e4m3(np.nan))


@pytest.mark.parametrize("amax", [448.0, 448.0000001, 1.0, 0.875, 0.8750001, 1e-30, 3e38, 0.0, 1e-45])
def test_scale_is_the_least_power_of_two(amax):
    s = paged.pow2_scale(amax)
    assert 448 * s >= amax and (448 * s / 2 < amax or s == 2.0 ** -126)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(5)
    x, th = rng.standard_normal((3, 64)), rng.standard_normal((7, 16))
    y = paged.rotate(x, 4, np.cos(th), np.sin(th), interleaved)
    a, b = (x[:, 0:32:2], x[:, 1:32:2]) if interleaved else (x[:, :16], x[:, 16:32])
    z = (a + 1j * b) * np.exp(1j * th[4])
    got = y[:, 0:32:2] + 1j * y[:, 1:32:2] if interleaved else y[:, :16] + 1j * y[:, 16:32]
    assert np.abs(got - z).max() < 1e-14 and np.array_equal(y[:, 32:], x[:, 32:])


def _cache(rng, pages, hkv, P, D, f8):
    c = {n: rng.standard_normal((pages, hkv, P, D)) for n in "kv"}
    c["ks"] = c["vs"] = None
    if f8:
        for n in "kv":
            c[n] = paged.round_e4m3(c[n] * 100)
            c[n + "s"] = 2.0 ** rng.integers(-8, -5, (pages, hkv))
    return c


def _contiguous(c, name, table, L, S):
    hkv, D = c[name].shape[1], c[name].shape[3]
    x = np.zeros((len(L), S, hkv, D))
    for b, n in enumerate(L):
        for h in range(hkv):
            x[b, :n, h] = paged.row_values(c, name, table[b], int(n), h)
    return x


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("left,right,cap,sinks", [(-1, -1, 0, 0), (7, 0, 0, 0), (3, 2, 5.0, 3), (-1, 0, 0, 2)])
def test_attention_is_the_contiguous_one(f8, left, right, cap, sinks):
    rng = np.random.default_rng(9)
    c = _cache(rng, 12, 2, 16, 8, f8)
    table, L, Q = rng.permutation(12).reshape(3, 4), np.array([33, 4, 64]), 3
    q = rng.standard_normal((9, 4, 8))
    bias = rng.standard_normal((4, sinks)) if sinks else None
    out, lse, _ = oracle.paged_attention(q, c, table, L, np.arange(0, 10, 3), window_left=left,
                                         window_right=right, logits_soft_cap=cap, sink_bias=bias)
    ref, rl = oracle.ragged_flash_attention(
        q.reshape(3, Q, 4, 8), _contiguous(c, "k", table, L, 64), _contiguous(c, "v", table, L, 64),
        np.zeros(3, int), L, window_left=left, window_right=right, logits_soft_cap=cap or None, sink_bias=bias)
    assert np.abs(out - ref.reshape(out.shape)).max() < 1e-12
    assert np.abs(lse - rl.reshape(lse.shape)).max() < 1e-12


def test_selection_is_the_last_tokens_of_the_contiguous_one():
    rng = np.random.default_rng(10)
    c = _cache(rng, 8, 2, 16, 8, True)
    table, L, Q = rng.permutation(8).reshape(2, 4), np.array([64, 64]), 3
    q = rng.standard_normal((2, 64, 4, 8))
    idx = rng.integers(-1, 3, (2, 64, 2, 4))
    ref, rl = oracle.nsa_select_attention(q, _contiguous(c, "k", table, L, 64),
                                          _contiguous(c, "v", table, L, 64), idx, 3, 32)
    out, lse, _ = oracle.nsa_select_paged(q[:, -Q:], c, table, L, idx[:, -Q:], 3, 32)
    fin = ~np.isneginf(lse)
    assert np.array_equal(fin, ~np.isneginf(rl[:, -Q:]))
    assert np.abs(out - ref[:, -Q:]).max() < 1e-12 and np.abs(lse[fin] - rl[:, -Q:][fin]).max() < 1e-12


def test_append_token_by_token_ends_near_append_at_once():
    """Powers of two only move exponents, so a page filled one by one differs by what became
    subnormal: at most half a subnormal step (2^-10) of the final scale, once per growth
    (the last growth to each scale dominates: in all below one step)."""
    rng = np.random.default_rng(11)
    n, P = 37, 16
    k = rng.standard_normal((n, 1, 8)) * np.exp(rng.standard_normal((n, 1, 1)) * 2)
    table = np.array([[2, 0, 1]])
    once, steps = _cache(rng, 3, 1, P, 8, True), _cache(rng, 3, 1, P, 8, True)
    paged.paged_kv_append(once, k, k, table, [n], [0, n])
    for t in range(n):
        paged.paged_kv_append(steps, k[t:t + 1], k[t:t + 1], table, [t + 1], [0, 1])
    assert np.array_equal(once["ks"], steps["ks"])
    a, b = (paged.row_values(c, "k", table[0], n, 0) for c in (once, steps))
    s = once["ks"][table[0][np.arange(n) // P], 0][:, None]
    assert (np.abs(a - b) <= 2.0 ** -9 * s).all()
    assert (np.abs(a - k[:, 0]) <= 2.0 ** -4 * np.abs(k[:, 0]) + 2.0 ** -10 * s).all()
