"""Latent attention in fp64 on the CPU (numpy), one query at a time from the formulas in include/kda.h.

Correctness reference for the smoke check and the tests; never on the product path.
"""
from __future__ import annotations

import numpy as np


def rotate(x, pos, inv_freq, interleaved=False):
    """R(p) x for rows x [..., 64] at position pos: pair i turned by pos * inv_freq[i]."""
    x = np.asarray(x, dtype=np.float64)
    angle = float(pos) * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(angle), np.sin(angle)
    y = np.empty_like(x)
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def attend(q, k, v, scale):
    """Softmax attention of one query q [D] over keys k [L, D] and values v [L, V]: (out [V], lse)."""
    if len(k) == 0:
        return np.zeros(v.shape[-1]), -np.inf
    s = scale * (np.asarray(k, dtype=np.float64) @ np.asarray(q, dtype=np.float64))
    m = s.max()
    p = np.exp(s - m)
    return (p @ np.asarray(v, dtype=np.float64)) / p.sum(), m + np.log(p.sum())


def decode(q, rows, scale, tokens=1):
    """q [N * tokens, H, D] over rows, a list of each sequence's cached rows [L, D]: token t of sequence n sees
    the first L - tokens + t + 1.  Returns (out [N * tokens, H, 512], lse)."""
    out, lse = np.zeros((*q.shape[:2], 512)), np.zeros(q.shape[:2])
    for r in range(q.shape[0]):
        n, t = divmod(r, tokens)
        seen = rows[n][: max(0, len(rows[n]) - tokens + t + 1)]
        for h in range(q.shape[1]):
            out[r, h], lse[r, h] = attend(q[r, h], seen, seen[:, :512], scale)
    return out, lse


def prefill(q, k, v, k_rope, scale, cu, cu_k):
    """q [T, H, dk], k, v [S, H, 128], k_rope [S, dk - 128] or None, causal and aligned at the sequences' ends.
    Returns (out [T, H, 128], lse [T, H])."""
    out, lse = np.zeros((*q.shape[:2], 128)), np.zeros(q.shape[:2])
    for n in range(len(cu) - 1):
        for i in range(cu[n], cu[n + 1]):
            end = cu_k[n + 1] - (cu[n + 1] - 1 - i)
            for h in range(q.shape[1]):
                kk = k[cu_k[n]:max(end, cu_k[n]), h]
                if k_rope is not None:
                    kk = np.concatenate([kk, k_rope[cu_k[n]:max(end, cu_k[n])]], axis=1)
                out[i, h], lse[i, h] = attend(q[i, h], kk, v[cu_k[n]:max(end, cu_k[n]), h], scale)
    return out, lse
