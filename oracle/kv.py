"""The 4-bit key/value cache and its attention, float64, by plain definition.

DFlash README ("How it works", the architecture note): every fourth layer of the hybrid target is
full attention over a quantised cache, and draft trees are verified under a mask that follows
the parent pointers.  The format is this library's reading: 32 channels share a power of two 2^e,
elements are the 4-bit floats of GRID with a sign, rounded to nearest even.

    stored(x)     the values the cache holds for rows x [..., d]
    stored_pair   the same for the key and value rows of one (token, head): a NaN or an infinity
                  in either makes the key NaN and the value zero
    attention     softmax attention with a visibility matrix; rows that see nothing are zero
    visible_*     the causal and the tree visibility
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MAX_EXP = 125


def block_exponent(amax):
    """e of a block with largest magnitude amax: two below its binary exponent, one more where
    amax / 2^floor(log2 amax) exceeds 1.75; within [-125, 125]."""
    if amax == 0.0:
        return -MAX_EXP
    m, ex = np.frexp(amax)  # amax = m 2^ex, m in [0.5, 1)
    e = int(ex) - 3 + (1 if m > 0.875 else 0)
    return max(-MAX_EXP, min(MAX_EXP, e))


def nearest(y):
    """Nearest grid value of y >= 0, ties to the even code, at most 6."""
    gap = np.abs(np.asarray(y)[..., None] - GRID)
    best = gap.min(axis=-1, keepdims=True)
    tied = gap == best
    even = tied & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), tied.argmax(-1))
    return GRID[pick]


def stored(x):
    x = np.asarray(x, dtype=np.float64)
    xb = x.reshape(-1, 32)
    out = np.empty_like(xb)
    for i, row in enumerate(xb):
        unit = 2.0 ** block_exponent(np.abs(row).max())
        out[i] = np.copysign(nearest(np.abs(row) / unit), row) * unit
    return out.reshape(x.shape)


def stored_pair(k, v):
    """k, v [..., d] of the same tokens and heads."""
    k, v = np.asarray(k, dtype=np.float64), np.asarray(v, dtype=np.float64)
    bad = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1))
    ks = stored(np.where(bad[..., None], 0.0, k))
    vs = stored(np.where(bad[..., None], 0.0, v))
    ks[bad], vs[bad] = np.nan, 0.0
    return ks, vs


def visible_causal(past, n):
    """[n, past + n]: new token i sees the past, the earlier new ones and itself."""
    return np.tril(np.ones((n, past + n), dtype=bool), past)


def visible_tree(parent, past):
    n = len(parent)
    see = np.zeros((n, past + n), dtype=bool)
    see[:, :past] = True
    for i in range(n):
        a = i
        while a >= 0:
            see[i, past + a] = True
            a = int(parent[a])
    return see


def attention(q, K, V, see, scale):
    """q [n, Hq, d], K, V [L, Hkv, d], see [n, L]; returns [n, Hq, d]."""
    q, K, V = (np.asarray(a, dtype=np.float64) for a in (q, K, V))
    n, Hq, d = q.shape
    G = Hq // K.shape[1]
    out = np.zeros((n, Hq, d))
    for i in range(n):
        at = np.flatnonzero(see[i])
        if len(at) == 0:
            continue
        for h in range(Hq):
            s = scale * (K[at, h // G] @ q[i, h])
            p = np.exp(s - s.max())
            out[i, h] = (p @ V[at, h // G]) / p.sum()
    return out
