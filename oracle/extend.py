"""Attention of several new tokens over a cached sequence, in fp64: the definition, row by row.

Query i of n stands at position p = L - n + i of a sequence of L cached
tokens and sees tokens j <= p, with a window only those with j > p - window
or j < sinks.  A query that sees nothing gives zeros.
"""
from __future__ import annotations

import numpy as np


def visible(L, n, window=0, sinks=0):
    """Boolean [n, L]: which tokens each query sees."""
    p = np.arange(L - n, L)[:, None]
    j = np.arange(L)[None, :]
    see = j <= p
    if window:
        see = see & ((j > p - window) | (j < sinks))
    return see


def extend_attention(q, K, V, scale, window=0, sinks=0):
    """q [n, Hq, D], K, V [L, Hkv, D] -> fp64 [n, Hq, D]."""
    q = np.asarray(q, np.float64)
    n, hq, d = q.shape
    L, hkv, _ = K.shape
    out = np.zeros((n, hq, d))
    if L == 0 or n == 0:
        return out
    see = visible(L, n, window, sinks)
    with np.errstate(invalid="ignore"):
        for h in range(hq):
            k, v = K[:, h // (hq // hkv)].astype(np.float64), V[:, h // (hq // hkv)].astype(np.float64)
            for i in range(n):
                t = np.flatnonzero(see[i])
                if not t.size:
                    continue
                s = scale * (k[t] @ q[i, h])
                e = np.exp(s - s.max())
                out[i, h] = (e / e.sum()) @ v[t]
    return out
