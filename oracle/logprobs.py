"""Log probabilities of a row of logits, float64, by plain definition.

SpecLA guide (the draft-tree budget): the tree builder takes the top candidates of every position with
their log probabilities.  NaN logits count as -inf, +inf logits share all the weight, alternatives are
sorted by logit and then by index, and only tokens with a probability are alternatives (one whose
logarithm fp32 holds).
"""
from __future__ import annotations

import numpy as np


def logprobs(row):
    """(log probabilities of all tokens, entropy)."""
    x = np.asarray(row, dtype=np.float64).copy()
    x[np.isnan(x)] = -np.inf
    m = x.max()
    if m == -np.inf:
        return np.full(len(x), -np.inf), 0.0
    if m == np.inf:
        n = int((x == m).sum())
        return np.where(x == m, -np.log(n), -np.inf), float(np.log(n))
    with np.errstate(under="ignore"):
        w = np.exp(x - m)
    z = w.sum()
    logp = (x - m) - np.log(z)
    with np.errstate(over="ignore"):
        logp[logp.astype(np.float32) == -np.inf] = -np.inf
    away = np.where(w > 0, m - x, 0.0)
    return logp, float(np.log(z) + (w * away).sum() / z)


def alternatives(row, k):
    """(tokens [k], log probabilities [k]), -1 and -inf behind the last."""
    logp, _ = logprobs(row)
    x = np.asarray(row, dtype=np.float64)
    possible = np.flatnonzero(logp > -np.inf)
    order = possible[np.lexsort((possible, -x[possible]))][:k]
    tok, lp = np.full(k, -1, dtype=np.int64), np.full(k, -np.inf)
    tok[:len(order)], lp[:len(order)] = order, logp[order]
    return tok, lp
