"""Float64 oracle of the chunk attention (a step's new rows over a paged key/value cache) and
of the page pool: pages forked, released and brought together, and their rows copied.

Written from the definitions, one row, sequence or page at a time; it shares no code with the
library.
"""

from __future__ import annotations

import math

import numpy as np


def chunk_attention(q, k_cache, v_cache, kept, lens, row_start, table, window=0, scale=None,
                    k_scale=None, v_scale=None):
    """(out, lse, weighted |v|, largest score error scale, rows written) per row and head.

    q [rows, H, D], caches [pages, page, Hkv, D].  The third result is sum_t p_t |v_t|, the
    fourth max_t scale * sum_d |q_d k_td|.  A page id outside the cache reads as zeros."""
    q = np.asarray(q, np.float64)
    N, H, D = q.shape
    P, page, Hk, _ = k_cache.shape
    scale = scale or 1.0 / math.sqrt(D)
    out, vabs = np.zeros((N, H, D)), np.zeros((N, H, D))
    lse, big = np.full((N, H), -np.inf), np.zeros((N, H))
    written = np.zeros(N, bool)
    for b in range(len(kept)):
        r0, r1 = int(row_start[b]), int(row_start[b + 1])
        T = min(max(int(lens[b]), 0), table.shape[1] * page)
        pos = np.arange(T)
        pid = np.asarray(table[b], np.int64)[pos // page]
        good = (pid >= 0) & (pid < P)
        pid = np.where(good, pid, 0)
        keys = np.where(good[:, None, None], k_cache[pid, pos % page], 0.0).astype(np.float64)
        values = np.where(good[:, None, None], v_cache[pid, pos % page], 0.0).astype(np.float64)
        if k_scale is not None:
            keys, values = keys * k_scale[:, None], values * v_scale[:, None]
        for row in range(r0, r1):
            written[row] = True
            p = max(int(kept[b]), 0) + row - r0
            lo, hi = max(0, p + 1 - window) if window else 0, min(p + 1, T)
            if hi <= lo:
                continue
            for h in range(H):
                g = h // (H // Hk)
                k, v = keys[lo:hi, g], values[lo:hi, g]
                s = scale * (k @ q[row, h])
                m = s.max()
                w = np.exp(s - m)
                lse[row, h] = m + math.log(w.sum())
                w /= w.sum()
                out[row, h] = w @ v
                vabs[row, h] = w @ np.abs(v)
                big[row, h] = scale * (np.abs(k) @ np.abs(q[row, h])).max()
    return out, lse, vabs, big, written


def _list(free_pages, span):
    first = min(max(int(span[0]), 0), len(free_pages))
    return first, min(max(int(span[1]), first), len(free_pages))


def page_fork(src_of, lens, held, table, shares, free_pages, span, page):
    """(table, lens, held, shares, span, missing, [(source, destination, rows)], bad id met)."""
    before, table = np.array(table), np.array(table)
    B, W = table.shape
    lens_out, held_out, shares = list(map(int, lens)), list(map(int, held)), np.array(shares)
    first, end = _list(free_pages, span)
    moves, missing, bad = [], 0, False
    for b in range(B):
        s = int(src_of[b])
        if held[b] > 0 or not 0 <= s < B:
            continue
        h = min(max(int(held[s]), 0), W)
        total = min(max(int(lens[s]), 0), h * page)
        full = total // page
        for j in range(full):
            table[b, j] = before[s, j]
            if 0 <= before[s, j] < len(shares):
                shares[before[s, j]] += 1
            else:
                bad = True
        lens_out[b], held_out[b] = full * page, full
        if total % page:
            if first < end:
                table[b, full] = free_pages[first]
                moves.append((int(before[s, full]), int(free_pages[first]), total % page))
                bad = bad or any(not 0 <= m < len(shares) for m in moves[-1][:2])
                first += 1
                lens_out[b], held_out[b] = total, full + 1
            else:
                missing += 1
    return table, lens_out, held_out, shares, [first, end], missing, moves, bad


def page_release(kept, held, table, shares, free_pages, span, page):
    """(held, shares, free pages, span, pages given back, bad id met)."""
    B, W = np.shape(table)
    holders = np.array(shares, np.int64) + 1
    held_out, dropped, bad = [], set(), False
    for b in range(B):
        h = min(max(int(held[b]), 0), W)
        need = min(h, -(-max(int(kept[b]), 0) // page))
        held_out.append(need)
        for j in range(need, h):
            p = int(table[b][j])
            if 0 <= p < len(holders):
                holders[p] -= 1
                dropped.add(p)
            else:
                bad = True
    back = sorted(p for p in dropped if holders[p] <= 0)
    free_pages = list(map(int, free_pages))
    first, end = _list(free_pages, span)
    front = min(len(back), first)
    for i, p in enumerate(back):
        free_pages[first - front + i if i < front else end + i - front] = p
    for p in back:
        holders[p] = 1
    return (held_out, holders - 1, free_pages, [first - front, end + len(back) - front],
            len(back), bad)


def page_compact(held, table, shares, free_pages):
    """(table, shares, free pages, span, [(source, destination)], bad id met)."""
    B, W = np.shape(table)
    P = len(shares)
    live, bad = set(), False
    for b in range(B):
        for j in range(min(max(int(held[b]), 0), W)):
            p = int(table[b][j])
            if 0 <= p < P:
                live.add(p)
            else:
                bad = True
    L = len(live)
    src = [p for p in range(L, P) if p in live]
    dst = [p for p in range(L) if p not in live]
    to = dict(zip(src, dst))
    out = np.full((B, W), -1)
    for b in range(B):
        for j in range(min(max(int(held[b]), 0), W)):
            p = int(table[b][j])
            out[b, j] = to.get(p, p)
    new = np.zeros(P, np.int64)
    for p in live:
        new[to.get(p, p)] = shares[p]
    free_pages = list(map(int, free_pages))
    free_pages[:P - L] = range(L, P)
    return out, new, free_pages, [0, P - L], list(zip(src, dst)), bad


def page_copy(cache, moves, page):
    """The cache [pages, page, ...] after (source, destination[, rows]) moves."""
    out = np.array(cache)
    for m in moves:
        rows = min(max(m[2], 0), page) if len(m) > 2 else page
        if 0 <= m[0] < len(cache) and 0 <= m[1] < len(cache):
            out[m[1], :rows] = cache[m[0], :rows]
    return out
