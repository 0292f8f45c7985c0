"""Full (dense) causal attention and rotary position embedding in fp64, the definitions only.

Plain numpy, one query row of a group at a time, no code shared with the library or with the block-sparse oracle.
``attend`` also returns, per output element, the weighted sum of the absolute values of v
(``sum_s p_s |v_s|``): the scale that rounding errors of the probabilities are measured in.
"""
from __future__ import annotations

import numpy as np

__all__ = ["as_f64", "rope", "attend", "prefill_varlen", "paged_rows", "prefill_paged",
           "decode_paged"]


def as_f64(t) -> np.ndarray:
    """A torch tensor (any device and float type) or array as float64."""
    if hasattr(t, "detach"):
        return t.detach().to("cpu").double().numpy()
    return np.asarray(t, dtype=np.float64)


def rope(x, pos, inv_freq, interleaved=False) -> np.ndarray:
    """x [T][heads][d] turned by pos[t] * inv_freq[j]; dimensions past 2*len(inv_freq) kept."""
    y = as_f64(x).copy()
    w = as_f64(inv_freq)
    r = 2 * len(w)
    a = np.asarray(pos, dtype=np.float64)[:, None] * w[None, :]
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    first = slice(0, r, 2) if interleaved else slice(0, r // 2)
    second = slice(1, r, 2) if interleaved else slice(r // 2, r)
    u, v = y[..., first].copy(), y[..., second].copy()
    y[..., first] = u * c - v * s
    y[..., second] = v * c + u * s
    return y


def attend(q, k, v, scale, first_pos):
    """q [n][H][d] at positions first_pos.. over k, v [L][G][d]: (out, sum p|v|).

    Keys that a row does not see take no part: their values may be anything."""
    q, k, v = as_f64(q), as_f64(k), as_f64(v)
    n, H, d = q.shape
    L, G = k.shape[0], k.shape[1]
    out, mag = np.zeros((n, H, d)), np.zeros((n, H, d))
    hg = H // G
    for g in range(G):
        heads = slice(g * hg, (g + 1) * hg)
        for i in range(n):
            m = min(L, first_pos + i + 1)
            if m == 0:
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                z = scale * (q[i, heads] @ k[:m, g].T)
                p = np.exp(z - z.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                out[i, heads] = p @ v[:m, g]
                mag[i, heads] = p @ np.abs(v[:m, g])
    return out, mag


def prefill_varlen(q, k, v, cu, scale):
    q, k, v = as_f64(q), as_f64(k), as_f64(v)
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for a, e in zip(cu[:-1], cu[1:]):
        if e > a:
            out[a:e], mag[a:e] = attend(q[a:e], k[a:e], v[a:e], scale, 0)
    return out, mag


def paged_rows(cache, table_row, L) -> np.ndarray:
    """Rows 0..L-1 of one sequence of an fp64 cache."""
    page = cache.shape[1]
    p = np.arange(L)
    return cache[np.asarray(table_row)[p // page], p % page]


def prefill_paged(q, k_cache, v_cache, table, cu, seq_lens, scale):
    q = as_f64(q)
    kc, vc = as_f64(k_cache), as_f64(v_cache)
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        if e > a:
            L = int(seq_lens[b])
            out[a:e], mag[a:e] = attend(q[a:e], paged_rows(kc, table[b], L),
                                        paged_rows(vc, table[b], L), scale, L - (e - a))
    return out, mag


def decode_paged(q, k_cache, v_cache, table, seq_lens, scale):
    """One row per sequence; an empty sequence gives zeros."""
    q = as_f64(q)
    kc, vc = as_f64(k_cache), as_f64(v_cache)
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for b, L in enumerate(seq_lens):
        if L > 0:
            out[b:b + 1], mag[b:b + 1] = attend(q[b:b + 1], paged_rows(kc, table[b], L),
                                                paged_rows(vc, table[b], L), scale, L - 1)
    return out, mag
