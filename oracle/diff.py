"""Differential decode attention over the int8 cache (oracle).

Query heads and kv planes come in pairs.  Head i of the H = Hq / 2
differential heads has the query heads 2i, 2i + 1, the key planes 2p, 2p + 1
and the 256 value channels of planes 2p and 2p + 1, with p = i // g,
g = Hq / Hkv:

    out = softmax(s_0) V - lam * softmax(s_1) V

The query codes and the scores s are those of attention.py (float32, each
product one rounding); everything after them is float64.
"""

from __future__ import annotations

import numpy as np

from .attention import default_sm_scale, qk_int, scale_scores
from .quant import quantize_queries


def decode(q, k8, ks, v8, vs, rows, ctx, lam, sm_scale=None):
    """(out, mass), both float64 [B][M][H][256].

    q float32 [B][M][Hq][d]; k8, v8 int8 [Hkv][cap][d]; ks, vs float32
    [Hkv][cap]; rows: per sequence the cache rows of its keys 0, 1, ... (at
    least ctx[b] + M - 1 of them); ctx [B]; lam [H] or [B][M][H].
    mass = sum softmax(s_0) |V| + |lam| sum softmax(s_1) |V|: the size of what
    is added up, which an error of the weights scales with.
    """
    q = np.asarray(q, np.float32)
    B, M, Hq, d = q.shape
    Hkv = k8.shape[0]
    g, H = Hq // Hkv, Hq // 2
    scale = default_sm_scale(d) if sm_scale is None else np.float32(sm_scale)
    q8, qs = quantize_queries(q)
    lam = np.broadcast_to(np.asarray(lam, np.float64), (B, M, H))
    out = np.zeros((B, M, H, 2 * d))
    mass = np.zeros_like(out)
    for b in range(B):
        for j in range(M):
            at = np.asarray(rows[b][:int(ctx[b]) + j], np.int64)
            for p in range(Hkv // 2):
                V = np.concatenate([v8[2 * p + c, at].astype(np.float64)
                                    * vs[2 * p + c, at].astype(np.float64)[:, None]
                                    for c in (0, 1)], axis=1)
                heads = np.arange(p * g, p * g + g)
                for a, sign in ((0, np.ones(g)), (1, -lam[b, j, heads])):
                    S = qk_int(q8[b, j, 2 * heads + a], k8[2 * p + a, at])
                    s = scale_scores(S, qs[b, j, 2 * heads + a], ks[2 * p + a, at], scale)
                    s = s.astype(np.float64)
                    w = np.exp(s - s.max(axis=1, keepdims=True))
                    w = w / w.sum(axis=1, keepdims=True) * sign[:, None]
                    out[b, j, heads] += w @ V
                    mass[b, j, heads] += np.abs(w) @ np.abs(V)
    return out, mass
