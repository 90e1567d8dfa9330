"""fp64 oracle: gradients of attention over SparseMask bounds.  (TEST INFRASTRUCTURE)

No page prints them; they are the softmax backward over the key sets of
``blocksparse_attention`` (same source page).  ``out`` and ``lse`` are what the forward left, so
the probabilities are ``exp(scale q.k - lse)`` and ``Delta = rowsum(d_out * out)`` of the values
given.  Each row's keys are found one row at a time.
"""

from __future__ import annotations

import math

import numpy as np


def blocksparse_attention_backward(q, k, v, out, lse, d_out, q_positions, q_segment_ids,
                                   kv_positions, kv_segment_ids, lower, upper, q_blocksize,
                                   kv_blocksize, *, causal=True, window_left=-1, window_right=-1,
                                   padding_segment_id=-1, softmax_scale=None, rows=None,
                                   lower_full=None, upper_full=None, magnitudes=False):
    """``dq`` [B, T, Hq, D], ``dk`` and ``dv`` [B, T, Hkv, D] (float64).

    ``rows``: (b, t) pairs whose contribution is computed (all by default); dq of the others is
    NaN.  ``lower_full`` / ``upper_full``: keys of these blocks need no token test.  With
    ``magnitudes`` also three arrays for error bounds, the sums with every factor replaced by its
    magnitude: ``sum_k |dS| |k|``, ``sum |dS| |q|``, ``sum P |d_out|`` (the first two times scale),
    where |dS| counts the magnitudes of both terms of its difference.
    """
    q, k, v, out, d_out = (np.asarray(x, dtype=np.float64) for x in (q, k, v, out, d_out))
    lse = np.asarray(lse, dtype=np.float64)
    q_pos, q_seg, kv_pos, kv_seg = (np.asarray(x, dtype=np.int64)
                                    for x in (q_positions, q_segment_ids, kv_positions, kv_segment_ids))
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if softmax_scale is None or softmax_scale <= 0 else float(softmax_scale)
    dq = np.full(q.shape, np.nan if rows is not None else 0.0)
    dk, dv = np.zeros(k.shape), np.zeros(v.shape)
    mq, mk, mv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b, t in rows if rows is not None else [(b, t) for b in range(B) for t in range(T)]:
        qb = t // q_blocksize
        key = np.arange(int(lower[b, 0, qb]) * kv_blocksize, min(int(upper[b, 0, qb]) * kv_blocksize, T))
        keep = (kv_seg[b, key] == q_seg[b, t]) & (q_seg[b, t] != padding_segment_id)
        if causal:
            keep &= kv_pos[b, key] <= q_pos[b, t]
        if window_left >= 0:
            keep &= q_pos[b, t] - kv_pos[b, key] <= window_left
        if window_right >= 0:
            keep &= kv_pos[b, key] - q_pos[b, t] <= window_right
        if lower_full is not None:
            keep |= (key // kv_blocksize >= lower_full[b, 0, qb]) & (key // kv_blocksize < upper_full[b, 0, qb])
        key = key[keep]
        dq[b, t] = 0.0
        if key.size == 0:
            continue
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            kk, vv = k[b, key, h], v[b, key, h]
            p = np.exp(scale * (q[b, t, hs] @ kk.T) - lse[b, t, hs, None])
            p[np.isneginf(lse[b, t, hs])] = 0.0
            g = d_out[b, t, hs]
            ds = p * (g @ vv.T - (g * out[b, t, hs]).sum(-1, keepdims=True))
            dq[b, t, hs] = scale * (ds @ kk)
            dk[b, key, h] += scale * (ds.T @ q[b, t, hs])
            dv[b, key, h] += p.T @ g
            if magnitudes:
                big = p * (np.abs(g) @ np.abs(vv).T + np.abs(g * out[b, t, hs]).sum(-1, keepdims=True))
                mq[b, t, hs] = scale * (big @ np.abs(kk))
                mk[b, key, h] += scale * (big.T @ np.abs(q[b, t, hs]))
                mv[b, key, h] += p.T @ np.abs(g)
    return (dq, dk, dv, mq, mk, mv) if magnitudes else (dq, dk, dv)
