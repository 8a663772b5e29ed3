"""Page tables of the paged cache by plain lists: who holds which page, and where new tokens go.

    reserve    entries without a page take the lowest free ids in order of sequence and entry
    release    entries behind the kept slots give theirs back
"""
from __future__ import annotations


def entries(length, n, page, width):
    return min(width, -(-(max(length, 0) + n) // page))


def reserve(table, refs, length, new, page, depth=None):
    """table: lists of ids (changed), refs: list (changed).  Returns (missing, slots, positions)."""
    n_pages = len(refs)
    free = [p for p in range(n_pages) if refs[p] == 0]
    missing = []
    for b, row in enumerate(table):
        short = 0
        for i in range(entries(length[b], new[b], page, len(row))):
            if 0 <= row[i] < n_pages:
                continue
            if free:
                row[i] = free.pop(0)
                refs[row[i]] = 1
            else:
                short += 1
        missing.append(short)
    slots, positions, t = [], [], 0
    for b, row in enumerate(table):
        for i in range(new[b]):
            at = max(length[b], 0) + i
            k = at // page
            slots.append(row[k] * page + at % page if k < len(row) and 0 <= row[k] < n_pages else -1)
            positions.append(max(length[b], 0) + (i if depth is None else depth[t]))
            t += 1
    return missing, slots, positions


def release(table, refs, keep, page):
    for b, row in enumerate(table):
        for i in range(-(-max(keep[b], 0) // page), len(row)):
            if 0 <= row[i] < len(refs):
                refs[row[i]] = max(0, refs[row[i]] - 1)
            row[i] = -1
