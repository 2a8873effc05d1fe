"""CPU oracle of the paged-cache operators in float64 (test infrastructure only):
norm and rotation, attention of new tokens over a paged cache, the attention
weights its keys received, and eviction by them.

A batch is a list of streams (new tokens n, cached keys kv) and a page table;
pools are [pages, kv_heads, page_size, d].
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, w, pos, axis_dims, theta=10000.0, halves=False, eps=1e-6):
    """x [tokens, heads, d] -> normed (w not None) and rotated by pos [tokens, axes]."""
    y = np.asarray(x, np.float64)
    if w is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    out, at, R = y.copy(), 0, int(sum(axis_dims))
    for a, n in enumerate(axis_dims):
        for i in range(n // 2):
            ang = (np.asarray(pos)[:, a].astype(np.float64) * float(theta) ** (-2.0 * i / n))[:, None]
            c0, c1 = (at, at + R // 2) if halves else (2 * at, 2 * at + 1)
            out[..., c0] = y[..., c0] * np.cos(ang) - y[..., c1] * np.sin(ang)
            out[..., c1] = y[..., c0] * np.sin(ang) + y[..., c1] * np.cos(ang)
            at += 1
    return out


def gather(pool, table, kv):
    """[kv_heads, kv, d] of one stream; a page that is none gives zeros."""
    n_pages, hk, page, d = pool.shape
    out = np.zeros((hk, kv, d))
    for j in range(kv):
        pg = int(table[j // page])
        if 0 <= pg < n_pages:
            out[:, j] = pool[pg, :, j % page]
    return out


def visible(n, kv, m):
    """Keys that each new token sees: the first this many."""
    if m == 0:
        return [kv] * n
    return [min(max(kv - n + (t // m + 1) * m, 0), kv) for t in range(n)]


def attend(q, k_pool, v_pool, seqs, tables, mask, scale=None, rows=None):
    """(o, lse, mag): outputs, logarithms of the sums, and sum_j p_j |v_j|, the
    scale that a bound of the output's error needs.  rows: only these (token rows)."""
    q = np.asarray(q, np.float64)
    T, H, d = q.shape
    hk = k_pool.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, mag, lse, at = np.zeros((T, H, d)), np.zeros((T, H, d)), np.full((T, H), -np.inf), 0
    for (n, kv), table in zip(seqs, tables):
        K, V = gather(k_pool, table, kv), gather(v_pool, table, kv)
        for t, lim in enumerate(visible(n, kv, mask)):
            if lim == 0 or (rows is not None and at + t not in rows):
                continue
            for h in range(H):
                g = h // (H // hk)
                s = K[g, :lim] @ q[at + t, h] * scale
                top = s.max()
                p = np.exp(s - top)
                o[at + t, h] = p @ V[g, :lim] / p.sum()
                mag[at + t, h] = p @ np.abs(V[g, :lim]) / p.sum()
                lse[at + t, h] = top + np.log(p.sum())
        at += n
    return o, lse, mag


def weights(q, k_pool, lse, w_in, seqs, tables, mask, decay, scale=None):
    """The accumulated weights, zero from each stream's kv on."""
    q = np.asarray(q, np.float64)
    _, H, d = q.shape
    hk = k_pool.shape[1]
    scale = d ** -0.5 if scale is None else scale
    w, at = np.zeros(w_in.shape), 0
    for b, ((n, kv), table) in enumerate(zip(seqs, tables)):
        K = gather(k_pool, table, kv)
        w[b, :, :kv] = np.asarray(w_in, np.float64)[b, :, :kv] * decay
        for t, lim in enumerate(visible(n, kv, mask)):
            for h in range(H):
                if lse[at + t, h] == -np.inf:
                    continue
                g = h // (H // hk)
                w[b, g, :lim] += np.exp(K[g, :lim] @ q[at + t, h] * scale - float(lse[at + t, h]))
        at += n
    return w


def keep(w, kv, budget, sink, recent):
    """Indices of the keys that stay, of one stream and key head."""
    if kv <= budget:
        return list(range(kv))
    rank = lambda j: (1, 0.0) if np.isnan(w[j]) else (0, -float(w[j]))
    mid = sorted(range(sink, kv - recent), key=lambda j: (rank(j), j))[:budget - sink - recent]
    return sorted(list(range(sink)) + mid + list(range(kv - recent, kv)))
