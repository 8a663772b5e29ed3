"""Acceptance of a draft tree's tokens against the target's logits, float64, by plain definition.

DFlash README ("How it works"): the target's forward over the tree decides the accepted root
path.  The tree is a function of the draft's scores, so drawing from the target is lossless; the
reading taken for the given random numbers: one per depth, inverting the running sum of the
softmax weights with the children's tokens first, in id order, then the others by index.

    weights(logits, temperature)   w_j = exp((l_j - max) / T); all on the first maximum when greedy
    draw_order                     the tokens in the order their weights are summed
    accept                         (path, next token) of one tree
"""
from __future__ import annotations

import numpy as np


def weights(logits, temperature):
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    m = l.max()
    if m == -np.inf:
        return np.zeros(l.shape)
    if not temperature > 0:
        return (np.arange(len(l)) == int(np.argmax(l))).astype(np.float64)
    if m == np.inf:  # the largest logits share all the weight
        return (l == m).astype(np.float64)
    finite = l > -np.inf
    return np.where(finite, np.exp((np.where(finite, l, m) - m) / np.float64(temperature)), 0.0)


def child_tokens(parent, tokens, node, vocab):
    """[(child, token)] of a node in id order; repeated and out-of-range tokens left out."""
    seen, out = set(), []
    for c in range(node + 1, len(parent)):
        t = int(tokens[c])
        if parent[c] == node and 0 <= t < vocab and t not in seen:
            seen.add(t)
            out.append((c, t))
    return out


def accept(parent, tokens, logits, uniform, temperature):
    """logits [n, V], uniform [>= depth + 1]; returns (path, next_token)."""
    node, path = 0, []
    while True:
        path.append(node)
        w = weights(logits[node], temperature)
        kids = child_tokens(parent, tokens, node, len(w))
        if w.sum() == 0.0:
            return path, -1
        first = [t for _, t in kids]
        rest = np.setdiff1d(np.arange(len(w)), first)
        order = np.concatenate([np.array(first, dtype=np.int64), rest])
        run = np.cumsum(w[order])
        theta = (0.5 if not temperature > 0 else float(uniform[len(path) - 1])) * run[-1]
        j = int(np.searchsorted(run, theta, side="right"))  # first running sum above theta
        if j >= len(order):  # rounding at the end: the last token that has weight
            j = int(np.flatnonzero(w[order])[-1])
            if j < len(kids):
                return path, first[j]
        if j < len(kids):
            node = kids[j][0]
            continue
        return path, int(order[j])
