"""Page operations on numpy arrays, one request and one page at a time.

State: ``kv`` [num_pages, 64, row words], ``table`` [R, W] (-1: no page),
``lens`` [R], ``counts`` [num_pages] (0: free).  Every function works in place
and returns the error bits (1: a bad index, length or entry; 2: no page left).
"""
from __future__ import annotations

import numpy as np

PAGE = 64
BAD, FULL = 1, 2


def _pages(n):
    return -(-int(n) // PAGE)


def copy(src_kv, dst_kv, src, dst):
    err = 0
    before = src_kv.copy()
    for s, d in zip(src.tolist(), dst.tolist()):
        if not (0 <= s < src_kv.shape[0] and 0 <= d < dst_kv.shape[0]):
            err |= BAD
            continue
        dst_kv[d] = before[s]
    return err


def fork(kv, table, lens, counts, parents, children):
    err = 0
    R, W = table.shape
    free = [int(p) for p in np.flatnonzero(counts == 0)]
    old_table, old_lens = table.copy(), lens.copy()
    used = 0
    for p, c in zip(parents.tolist(), children.tolist()):
        if not (0 <= p < R and 0 <= c < R) or not 0 <= old_lens[p] <= W * PAGE:
            err |= BAD
            continue
        L = int(old_lens[p])
        full, rem = divmod(L, PAGE)
        row = np.full(W, -1, table.dtype)
        page = int(old_table[p, full]) if rem else -1
        if rem and not 0 <= page < counts.size:
            err |= BAD
            page = -1
        if page >= 0:
            used += 1
            if used > len(free):
                err |= FULL
                table[c], lens[c] = row, 0
                continue
        for i in range(full):
            e = int(old_table[p, i])
            if e < -1 or e >= counts.size:
                err |= BAD
            elif e >= 0:
                row[i] = e
                counts[e] += 1
        if page >= 0:
            new = free[used - 1]
            row[full] = new
            counts[new] = 1
            kv[new, :rem] = kv[page, :rem]
        table[c], lens[c] = row, L
    return err


def alloc(table, lens, counts, new_lens):
    err = 0
    R, W = table.shape
    free = [int(p) for p in np.flatnonzero(counts == 0)]
    at = 0
    for b in range(R):
        L, N = int(lens[b]), int(new_lens[b])
        if not (0 <= L <= W * PAGE and 0 <= N <= W * PAGE):
            err |= BAD
            continue
        need = max(0, _pages(N) - _pages(L))
        if need and at + need > len(free):
            err |= FULL
        else:
            for i in range(need):
                if table[b, _pages(L) + i] != -1:
                    err |= BAD
                    continue
                table[b, _pages(L) + i] = free[at + i]
                counts[free[at + i]] = 1
        at += need
    return err


def free(table, lens, counts, new_lens, window=0, sinks=0):
    err = 0
    R, W = table.shape
    for b in range(R):
        L, N = int(lens[b]), int(new_lens[b])
        if N < 0 or N > L or L > W * PAGE:
            err |= BAD
            continue
        for i in range(W):
            seen = i < _pages(N)
            if seen and window > 0 and i * PAGE >= sinks and (i + 1) * PAGE - 1 <= N - window:
                seen = False  # its last token is behind every later query's window
            e = int(table[b, i])
            if seen or e == -1:
                continue
            table[b, i] = -1
            if not 0 <= e < counts.size or counts[e] <= 0:
                err |= BAD
            else:
                counts[e] -= 1
        lens[b] = N
    return err


def compact(kv, table, counts):
    """Returns (error bits, remap, live pages, moves)."""
    err = 0
    n = int((counts > 0).sum())
    holes = [p for p in range(n) if counts[p] == 0]
    movers = [p for p in range(n, counts.size) if counts[p] > 0]
    remap = np.where(counts > 0, np.arange(counts.size), -1).astype(np.int32)
    was_live = counts > 0
    for m, h in zip(movers, holes):
        kv[h] = kv[m]
        counts[h], counts[m] = counts[m], 0
        remap[m] = h
    for b in range(table.shape[0]):
        for i in range(table.shape[1]):
            e = int(table[b, i])
            if e == -1:
                continue
            if not 0 <= e < counts.size or not was_live[e]:
                err |= BAD
            else:
                table[b, i] = remap[e]
    return err, remap, n, len(movers)
