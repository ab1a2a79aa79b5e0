"""Float64 oracle of the paged serving steps: page tables and slots, the rows
written into the caches, and decode attention over a paged key/value cache.

Written from the definitions, one sequence, row or head at a time; it shares
no code with the library.
"""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def page_step(kept, new, held, table, free_pages, span, page, num_pages, max_rows):
    """(table, lens, held, row_start, positions, slots, span, missing, bad page met)."""
    table = np.array(table, dtype=np.int64)
    B, W = table.shape
    first = min(max(int(span[0]), 0), len(free_pages))
    end = min(max(int(span[1]), first), len(free_pages))
    free = [int(x) for x in free_pages[first:end]]
    taken = missing = 0
    lens, held_out, starts = [], [], [0]
    positions = np.full(max_rows, -1, np.int64)
    slots = np.full(max_rows, -1, np.int64)
    bad = False
    row = 0
    for b in range(B):
        k, n = max(int(kept[b]), 0), max(int(new[b]), 0)
        h = min(max(int(held[b]), 0), W)
        total = min(k + n, W * page, 2 ** 31 - 1)
        grow = max(0, math.ceil(total / page) - h)
        got = free[taken:taken + grow]
        taken += len(got)
        missing += grow - len(got)
        table[b, h:h + len(got)] = got
        h += len(got)
        held_out.append(h)
        lens.append(min(total, h * page))
        for i in range(n):
            if row < max_rows:
                pos = k + i
                positions[row] = min(pos, 2 ** 31 - 1)      # (an int32)
                if pos // page < h:
                    pid = int(table[b, pos // page])
                    if 0 <= pid < num_pages:
                        slots[row] = pid * page + pos % page
                    else:
                        bad = True
            row += 1
        starts.append(row)
    return (table, np.array(lens), np.array(held_out), np.array(starts), positions, slots,
            np.array([first + taken, end]), missing, bad)


def rotate(x, cos_sin_row, interleaved):
    """One position's rotation of x [..., d] by its table row (cosines, then sines)."""
    x = np.asarray(x, np.float64)
    half = x.shape[-1] // 2
    out = np.empty_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(cos_sin_row[i]), float(cos_sin_row[half + i])
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def rms_norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    return x / math.sqrt(float((x * x).sum()) / x.size + eps) * np.asarray(weight, np.float64)


def round_e4m3(x):
    """Nearest e4m3 value, ties to even, saturating (subnormal step 2^-9)."""
    x = np.clip(np.asarray(x, np.float64), -E4M3_MAX, E4M3_MAX)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(np.where(x == 0, 1.0, x))))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.rint(x / step) * step


def decode_attention(q, k_cache, v_cache, lens, table, window=0, scale=None, k_scale=None,
                     v_scale=None):
    """(out, lse, weighted |v|, largest score error scale) per sequence and head.

    q [B, H, D], caches [pages, page, Hkv, D].  The third result is sum_t p_t |v_t|,
    the fourth max_t scale * sum_d |q_d k_td| (what rounding errors scale with).
    A page id outside the cache reads as zeros."""
    q = np.asarray(q, np.float64)
    B, H, D = q.shape
    P, page, Hk, _ = k_cache.shape
    scale = scale or 1.0 / math.sqrt(D)
    out = np.zeros((B, H, D))
    lse = np.full((B, H), -np.inf)
    vabs = np.zeros((B, H, D))
    big = np.zeros((B, H))
    for b in range(B):
        T = min(max(int(lens[b]), 0), table.shape[1] * page)
        pos = np.arange(max(0, T - window) if window else 0, T)
        if not len(pos):
            continue
        pid = np.asarray(table[b], np.int64)[pos // page]
        good = (pid >= 0) & (pid < P)
        pid = np.where(good, pid, 0)
        for h in range(H):
            g = h // (H // Hk)
            k = np.asarray(k_cache[pid, pos % page, g], np.float64) * (
                1.0 if k_scale is None else float(k_scale[g]))
            v = np.asarray(v_cache[pid, pos % page, g], np.float64) * (
                1.0 if v_scale is None else float(v_scale[g]))
            k[~good] = 0.0
            v[~good] = 0.0
            s = scale * (k @ q[b, h])
            m = s.max()
            w = np.exp(s - m)
            lse[b, h] = m + math.log(w.sum())
            w /= w.sum()
            out[b, h] = w @ v
            vabs[b, h] = w @ np.abs(v)
            big[b, h] = scale * (np.abs(k) @ np.abs(q[b, h])).max()
    return out, lse, vabs, big
