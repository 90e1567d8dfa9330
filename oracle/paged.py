"""fp64 oracle: paged KV caches.  (TEST INFRASTRUCTURE)

A cache is a dict with ``k`` and ``v`` pools [num_pages, Hkv, P, D] holding the codes'
values (float64), ``ks`` and ``vs`` scales [num_pages, Hkv] or None (bf16 cache).
"""

from __future__ import annotations

import math

import numpy as np

from .nsa import selected_key_set


def round_e4m3(x):
    """Nearest e4m3 value, ties to even; magnitudes over 448 (and infinities) become 448."""
    x = np.clip(np.asarray(x, dtype=np.float64), -448.0, 448.0)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isnan(x), 0.0, x))
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.rint(x / step) * step


def pow2_scale(amax):
    """Least 2^e, e >= -126, with 448 * 2^e >= amax."""
    e = -126
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def rotate(x, pos, cos, sin, interleaved):
    """x [heads, D] at position pos."""
    if cos is None:
        return x
    y = np.array(x, dtype=np.float64)
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(cos[pos, i]), float(sin[pos, i])
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


def paged_kv_append(cache, k, v, table, lens, cu, *, cos=None, sin=None, interleaved=False):
    """Updates ``cache`` in place; k, v [N, Hkv, D].  bf16 pools get the unrounded value."""
    P = cache["k"].shape[2]
    Hkv = cache["k"].shape[1]
    for b in range(len(lens)):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        start = int(lens[b]) - (t1 - t0)
        at = {}
        for t in range(t0, t1):
            p = start + t - t0
            if p >= 0:
                at.setdefault(p // P, []).append((p, t))
        for j, tokens in at.items():
            pg = int(table[b, j])
            first = tokens[0][0] % P
            for name, x, turn in (("k", k, True), ("v", v, False)):
                new = np.stack([rotate(x[t], p, cos if turn else None, sin, interleaved)
                                for p, t in tokens])          # [n, Hkv, D]
                for h in range(Hkv):
                    rows = new[:, h]
                    if cache[name + "s"] is None:
                        cache[name][pg, h, first:first + len(rows)] = rows
                        continue
                    fin = np.abs(rows[np.isfinite(rows)])
                    need = pow2_scale(fin.max() if fin.size else 0.0)
                    if first > 0:
                        old = float(cache[name + "s"][pg, h])
                        need = max(old, need)
                        if need != old:
                            kept = cache[name][pg, h, :first]
                            cache[name][pg, h, :first] = round_e4m3(kept * (old / need))
                    cache[name + "s"][pg, h] = need
                    cache[name][pg, h, first:first + len(rows)] = round_e4m3(rows / need)


def row_values(cache, name, table_row, length, h):
    """[length, D] keys or values of one row and head."""
    P = cache[name].shape[2]
    pages = np.asarray(table_row[:-(-length // P)], dtype=np.int64)
    x = cache[name][pages, h]
    if cache[name + "s"] is not None:
        x = x * cache[name + "s"][pages, h][:, None, None]
    return x.reshape(-1, x.shape[-1])[:length]


def _softmax(s, v):
    """s [rows, n] -> output, LSE and sum of p |v| (what rounding errors of p scale with)."""
    out = np.zeros((s.shape[0], v.shape[1]))
    mag = np.zeros_like(out)
    lse = np.full(s.shape[0], -np.inf)
    for r in range(s.shape[0]):
        ok = ~np.isneginf(s[r])
        if not ok.any():
            continue
        x = s[r, ok]
        m = x.max()
        e = np.exp(x - m)
        out[r] = e @ v[ok] / e.sum()
        mag[r] = e @ np.abs(v[ok]) / e.sum()
        lse[r] = m + math.log(e.sum())
    return out, lse, mag


def paged_attention(q, cache, table, lens, cu, *, softmax_scale=None, window_left=-1,
                    window_right=-1, logits_soft_cap=None, sink_bias=None):
    """q [N, Hq, D]; returns (out, lse, mag), NaN for token rows of nobody."""
    N, Hq, D = q.shape
    Hkv = cache["k"].shape[1]
    G = Hq // Hkv
    scale = softmax_scale or 1.0 / math.sqrt(D)
    cap = logits_soft_cap or 0.0
    bias = None
    if sink_bias is not None:
        bias = np.broadcast_to(np.asarray(sink_bias, dtype=np.float64), (Hq, np.shape(sink_bias)[-1]))
    out, mag = np.full((N, Hq, D), np.nan), np.full((N, Hq, D), np.nan)
    lse = np.full((N, Hq), np.nan)
    for b in range(len(lens)):
        L = int(lens[b])
        key = np.arange(L)
        for h in range(Hkv):
            if int(cu[b + 1]) == int(cu[b]):
                continue
            k, v = (row_values(cache, n, table[b], L, h) for n in "kv")
            for t in range(int(cu[b]), int(cu[b + 1])):
                p = L - int(cu[b + 1]) + t
                see = np.ones(L, dtype=bool)
                if window_left >= 0:
                    see &= key >= p - window_left
                if window_right >= 0:
                    see &= key <= p + window_right
                hs = slice(h * G, (h + 1) * G)
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (q[t, hs] @ k.T)
                    if cap > 0:
                        s = cap * np.tanh(s / cap)
                if bias is not None:
                    n = min(bias.shape[1], L)
                    s[:, :n] += bias[hs, :n]
                    see = see | (key < bias.shape[1])
                s = np.where(see, s, -np.inf)
                out[t, hs], lse[t, hs], mag[t, hs] = _softmax(s, v)
    return out, lse, mag


def nsa_select_paged(q, cache, table, lens, block_indices, block_counts, block_size, *, causal=True,
                     softmax_scale=None, g_slc=None):
    """q [B, Q, Hq, D], block_indices [B, Q, Hkv, S]; returns (out, lse, mag)."""
    B, Q, Hq, D = q.shape
    Hkv = cache["k"].shape[1]
    G = Hq // Hkv
    scale = softmax_scale or 1.0 / math.sqrt(D)
    out, mag, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((B, Q, Hq), -np.inf)
    for b in range(B):
        L = int(lens[b])
        for h in range(Hkv):
            k, v = (row_values(cache, n, table[b], L, h) for n in "kv")
            for i in range(Q):
                n = int(block_counts if np.ndim(block_counts) == 0 else block_counts[b, i, h])
                keys = selected_key_set(block_indices[b, i, h], n, L, block_size, L - Q + i, causal)
                if keys.size == 0:
                    continue
                hs = slice(h * G, (h + 1) * G)
                out[b, i, hs], lse[b, i, hs], mag[b, i, hs] = _softmax(scale * (q[b, i, hs] @ k[keys].T),
                                                                       v[keys])
    if g_slc is not None:
        g = np.asarray(g_slc, dtype=np.float64)[..., None]
        out, mag = out * g, mag * np.abs(g)
    return out, lse, mag
