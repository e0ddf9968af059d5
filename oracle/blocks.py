"""Rotary positions and a cache with a scale per block of rows and head (oracle).

A cache is a dict: k, v float64 [Hkv][cap][128] (the values of the codes), ks, vs
float32 [Hkv][cap // R], R, e4m3.  Rows of key t: a sequence's table row names its
pages.
"""

from __future__ import annotations

import numpy as np

from .rounding import e4m3 as e4m3_grid

F = np.float32


def angles(freq, positions):
    """[n][h][2] float32, the product and the functions in float64."""
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(freq, np.float64)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(F)


def rotate(x, cs, interleaved, dtype=F):
    """x [n][heads][128], cs [n][h][2]; every operation in dtype."""
    h = cs.shape[1]
    y = np.array(x, dtype)
    c, s = cs[:, None, :, 0].astype(dtype), cs[:, None, :, 1].astype(dtype)
    a, b = (np.s_[..., 0:2 * h:2], np.s_[..., 1:2 * h:2]) if interleaved else (np.s_[..., :h], np.s_[..., h:2 * h])
    u, w = y[a].copy(), y[b].copy()
    y[a], y[b] = u * c - w * s, w * c + u * s
    return y


def round_codes(u, e4m3):
    if e4m3:
        return np.asarray(e4m3_grid(u), np.float64)
    u = np.where(np.isnan(u), 0, u)                                    # (an integer has no NaN)
    return np.clip(np.rint(u), -127, 127).astype(np.float64) + 0.0     # (and no -0)


def rows_of(table, page, keys):
    keys = np.asarray(keys, np.int64)
    return table[keys // page].astype(np.int64) * page + keys % page


def append(cache, name, x, start, table, page):
    """The rows x [n][Hkv][128] (float32) of one sequence, as keys start, start + 1, ...
    Elements that are not finite do not enter a block's scale."""
    R, e4m3 = cache["R"], cache["e4m3"]
    top = F(448 if e4m3 else 127)
    x = np.asarray(x, F)
    end = start + len(x)
    for key0 in range(start // R * R, end, R):
        lo, hi = max(start, key0), min(end, key0 + R)
        at = rows_of(table, page, np.arange(key0, hi))
        new = x[lo - start:hi - start].transpose(1, 0, 2)
        for h in range(x.shape[1]):
            s = np.divide(np.where(np.isfinite(new[h]), np.abs(new[h]), F(0)).max(), top, dtype=F)
            if lo > key0:
                was = cache[name + "s"][h, at[0] // R]
                if s > was:
                    f = np.divide(was, s, dtype=F)
                    kept = at[:lo - key0]
                    cache[name][h, kept] = round_codes((cache[name][h, kept].astype(F) * f).astype(F), e4m3)
                s = max(s, was)
            cache[name + "s"][h, at[0] // R] = s
            u = np.divide(new[h], s, dtype=F) if s > 0 else np.zeros_like(new[h])
            cache[name][h, at[lo - key0:]] = round_codes(u, e4m3)


def values(cache, name, rows):
    """float64 [Hkv][n][128]."""
    rows = np.asarray(rows, np.int64)
    return cache[name][:, rows] * cache[name + "s"][:, rows // cache["R"]].astype(np.float64)[..., None]


def decode(q, cache, table, page, ctx, sm_scale=None):
    """(out, mass, size), float64: out and mass = sum softmax |V| are [B][M][Hq][128],
    size [B][M][Hq] = the largest sum_i |q_i K_i| * sm_scale over the row's keys (what an
    error of the scores scales with)."""
    q = np.asarray(q, np.float64)
    B, M, Hq, d = q.shape
    Hkv = cache["k"].shape[0]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if sm_scale is None else sm_scale
    out, mass, size = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3])
    for b in range(B):
        if ctx[b] == 0:
            continue
        at = rows_of(table[b], page, np.arange(int(ctx[b]) + M - 1))
        K, V = values(cache, "k", at), values(cache, "v", at)
        for j in range(M):
            n = int(ctx[b]) + j
            for h in range(Hkv):
                heads = np.s_[b, j, h * g:h * g + g]
                s = q[heads] @ K[h, :n].T * scale
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[heads], mass[heads] = w @ V[h, :n], w @ np.abs(V[h, :n])
                size[heads] = (np.abs(q[heads]) @ np.abs(K[h, :n]).T).max(1) * abs(scale)
    return out, mass, size
