"""Sparse attention over selected pages of the key/value cache, float64, by plain definition.

The score of a page for a query is the largest q.k that its channelwise limits allow.  Consecutive new
tokens and the query heads of a kv head share a selection: the best of the pages that are full at the
committed length, by the largest score of its rows, lower entries first among equals.  A row attends
to the selected pages and to every later slot that it sees anyway.

    limits     largest and smallest key of a page per channel (NaN where a key is)
    select     table entries of every selection and kv head, ascending
    visible    the visibility of a kv head's rows, given what they would see of all slots
"""
from __future__ import annotations

import numpy as np


def limits(K):
    """K [slots, d] of one page and head."""
    K = np.asarray(K, dtype=np.float64)
    return K.max(0), K.min(0)


def score(rows, hi, lo):
    """Largest over the rows [n, d]; +inf for limits that are not numbers."""
    if not (np.isfinite(hi).all() and np.isfinite(lo).all()):
        return np.inf
    rows = rows[np.isfinite(rows).all(1)]
    if len(rows) == 0:
        return -np.inf
    return max(float(np.maximum(r * hi, r * lo).sum()) for r in rows)


def selections(n, share):
    share = share or max(n, 1)
    return [(i, min(n, i + share)) for i in range(0, n, share)]


def select(q, K, page, full, top, share=1, first=0, last=0, there=None):
    """q [n, Hq, d], K [>= full * page, Hkv, d]; there [full]: the page exists.  Returns a list over
    selections of arrays [Hkv, min(top, full)]."""
    q, K = np.asarray(q, dtype=np.float64), np.asarray(K, dtype=np.float64)
    n, Hq, d = q.shape
    H = K.shape[1]
    G = Hq // H
    there = np.ones(full, dtype=bool) if there is None else there
    lim = [[limits(K[i * page:(i + 1) * page, h]) if there[i] else None for i in range(full)] for h in range(H)]
    out = []
    for i0, i1 in selections(n, share):
        sel = np.zeros((H, min(top, full)), dtype=np.int64)
        for h in range(H):
            if full <= top:
                sel[h] = np.arange(full)
                continue
            rows = q[i0:i1, h * G:(h + 1) * G].reshape(-1, d)
            kept = list(range(first)) + list(range(full - last, full))
            rest = [i for i in range(full) if i not in set(kept)]
            rank = sorted(rest, key=lambda i: (not there[i], -score(rows, *lim[h][i]) if there[i] else 0.0, i))
            sel[h] = sorted(kept + rank[:top - first - last])
        out.append(sel)
    return out


def visible(see, entries, page, full):
    """see [n, L] of a selection's rows and the entries [k] of one kv head: later slots stay as they are."""
    use = np.zeros(see.shape[1], dtype=bool)
    for i in entries:
        use[i * page:(i + 1) * page] = True
    use[full * page:] = True
    return see & use[None, :]
