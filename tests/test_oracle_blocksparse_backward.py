"""Pins of the block-sparse gradient oracle (CPU, fp64): autograd of attention under a dense token
mask, central differences of the forward oracle, and closed cases."""

import numpy as np
import pytest
import torch

import oracle


def _case(seed, B=2, T=48, Hq=4, Hkv=2, D=8, qb=16, kb=8, causal=True, left=-1, right=-1, sorted_rows=True):
    rng = np.random.default_rng(seed)
    q, k, v, g = (rng.standard_normal((B, T, h, D)) for h in (Hq, Hkv, Hkv, Hq))
    seg = np.sort(rng.integers(0, 3, (B, T)), axis=1) if sorted_rows else rng.integers(0, 3, (B, T))
    seg[:, -5:] = -1
    pos = np.broadcast_to(np.arange(T), (B, T)).copy()
    if not sorted_rows:
        pos = rng.permuted(pos, axis=1)
    mask = dict(causal=causal, window_left=left, window_right=right)
    ints = (pos, seg, pos, seg)
    bounds = oracle.sparse_mask_bounds(*ints, qb, kb, **mask)
    return q, k, v, g, ints, bounds, qb, kb, mask


def _token_mask(ints, bounds, qb, kb, mask, T):
    pos, seg = ints[0], ints[1]
    see = (seg[:, :, None] == seg[:, None, :]) & (seg[:, :, None] != -1)
    gap = pos[:, :, None] - pos[:, None, :]
    if mask["causal"]:
        see &= gap >= 0
    if mask["window_left"] >= 0:
        see &= gap <= mask["window_left"]
    if mask["window_right"] >= 0:
        see &= -gap <= mask["window_right"]
    blk = np.arange(T) // kb
    lo, up = (np.repeat(np.asarray(x)[:, 0], qb, axis=1)[:, :, None] for x in bounds[:2])
    return see & (blk >= lo) & (blk < up)


CASES = [dict(), dict(left=10, right=0), dict(causal=False, left=7, right=4), dict(causal=False, right=3),
         dict(Hq=3, Hkv=1, kb=16), dict(sorted_rows=False, left=20)]


@pytest.mark.parametrize("kw", CASES)
def test_autograd_of_attention_under_the_token_mask(kw):
    q, k, v, g, ints, bounds, qb, kb, mask = _case(1, **kw)
    B, T, Hq, D = q.shape
    G = Hq // k.shape[2]
    see = torch.from_numpy(_token_mask(ints, bounds, qb, kb, mask, T))
    leaves = [torch.from_numpy(x).requires_grad_() for x in (q, k, v)]
    tq = leaves[0].transpose(1, 2)
    tk, tv = (x.transpose(1, 2).repeat_interleave(G, 1) for x in leaves[1:])
    s = (tq @ tk.transpose(-1, -2) / D ** 0.5).masked_fill(~see[:, None], float("-inf"))
    some = see.any(-1)[:, None, :, None]
    p = torch.where(some, torch.softmax(torch.where(some, s, torch.zeros_like(s)), -1), torch.zeros_like(s))
    o = p @ tv
    ref = torch.autograd.grad(o, leaves, torch.from_numpy(g).transpose(1, 2))
    out, lse = oracle.blocksparse_attention(q, k, v, *ints, *bounds[:2], qb, kb, **mask)
    got = oracle.blocksparse_attention_backward(q, k, v, out, lse, g, *ints, *bounds[:2], qb, kb, **mask)
    for a, b in zip(got, ref):
        np.testing.assert_allclose(a, b.numpy(), rtol=1e-9, atol=1e-11)


def test_central_differences_of_the_forward_oracle():
    q, k, v, g, ints, bounds, qb, kb, mask = _case(2, B=1, T=32, Hq=2, Hkv=1, D=4, left=9)
    loss = lambda *x: (oracle.blocksparse_attention(*x, *ints, *bounds[:2], qb, kb, **mask)[0] * g).sum()  # noqa: E731
    out, lse = oracle.blocksparse_attention(q, k, v, *ints, *bounds[:2], qb, kb, **mask)
    got = oracle.blocksparse_attention_backward(q, k, v, out, lse, g, *ints, *bounds[:2], qb, kb, **mask)
    for i in range(3):
        for at in np.ndindex(*got[i].shape):
            x = [q.copy(), k.copy(), v.copy()]
            x[i][at] += 1e-5
            up = loss(*x)
            x[i][at] -= 2e-5
            assert abs((up - loss(*x)) / 2e-5 - got[i][at]) < 1e-7


def test_rows_without_keys_and_keys_without_rows():
    q, k, v, g, ints, bounds, qb, kb, mask = _case(3)
    out, lse = oracle.blocksparse_attention(q, k, v, *ints, *bounds[:2], qb, kb, **mask)
    dq, dk, dv = oracle.blocksparse_attention_backward(q, k, v, out, lse, g, *ints, *bounds[:2], qb, kb, **mask)
    assert not dq[:, -5:].any() and not dk[:, -5:].any() and not dv[:, -5:].any()
    # one key: P = 1, dS = 0
    assert np.isclose(dq[:, 0], 0).all()


def test_full_blocks_take_every_key_and_magnitudes_bound_the_sums():
    q, k, v, g, ints, bounds, qb, kb, mask = _case(4)
    shape = np.asarray(bounds[0]).shape
    every = dict(lower_full=np.zeros(shape, int), upper_full=np.full(shape, 1))
    plain = dict(causal=False)
    none = (ints[0], np.zeros_like(ints[1]), ints[2], np.zeros_like(ints[3]))
    lo, up = np.zeros(shape, int), np.full(shape, 1)
    out, lse = oracle.blocksparse_attention(q, k, v, *none, lo, up, qb, kb, **plain)
    a = oracle.blocksparse_attention_backward(q, k, v, out, lse, g, *none, lo, up, qb, kb, **plain)
    b = oracle.blocksparse_attention_backward(q, k, v, out, lse, g, *ints, lo, up, qb, kb, **mask, **every, magnitudes=True)
    for x, y, m in zip(a, b[:3], b[3:]):
        np.testing.assert_array_equal(x, y)
        assert (np.abs(y) <= m + 1e-12).all()


def test_rows_add_up():
    q, k, v, g, ints, bounds, qb, kb, mask = _case(5)
    out, lse = oracle.blocksparse_attention(q, k, v, *ints, *bounds[:2], qb, kb, **mask)
    f = lambda rows: oracle.blocksparse_attention_backward(q, k, v, out, lse, g, *ints, *bounds[:2], qb, kb, rows=rows, **mask)  # noqa: E731
    pairs = [(b, t) for b in range(2) for t in range(48)]
    whole, one, two = f(None), f(pairs[::2]), f(pairs[1::2])
    for i in (1, 2):
        np.testing.assert_allclose(one[i] + two[i], whole[i], rtol=0, atol=1e-12)
    np.testing.assert_array_equal(np.where(np.isnan(one[0]), two[0], one[0]), whole[0])
