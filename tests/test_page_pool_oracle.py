"""Pins of the page pool's and the chunk attention's oracle: worked examples and invariants."""

import numpy as np

from oracle import page_pool as O
from oracle import paged as P


def test_fork_example():
    # sequence 0 holds pages 7, 3, 5 with 10 rows of 4; slots 1 and 3 take it, the list has one page
    table = [[7, 3, 5, -1], [-1] * 4, [2, -1, -1, -1], [-1] * 4]
    t, lens, held, shares, span, missing, moves, bad = O.page_fork(
        [2, 0, 0, 0], [10, 0, 4, 0], [3, 0, 1, 0], table, [0] * 8, [9, 6, 1], [1, 2], 4)
    assert t[1].tolist() == [7, 3, 6, -1] and t[3].tolist() == [7, 3, -1, -1]
    assert t[0].tolist() == table[0] and t[2].tolist() == table[2]      # they hold pages: as before
    assert lens == [10, 10, 4, 8] and held == [3, 3, 1, 2]
    assert shares.tolist() == [0, 0, 0, 2, 0, 0, 0, 2]
    assert span == [2, 2] and missing == 1 and moves == [(5, 6, 2)] and not bad


def test_release_example():
    # page 3 is held by both sequences: one hold less; pages 7 and 5 go back in front of the list
    held, shares, free, span, n, bad = O.page_release(
        [0, 5], [3, 2], [[7, 3, 5], [2, 3, -1]], [0, 0, 0, 1, 0, 0, 0, 0], [0] * 8, [1, 1], 4)
    assert held == [0, 2] and shares.tolist() == [0] * 8 and n == 2 and not bad
    assert span == [0, 2] and free[:2] == [5, 7]
    # both end: it goes back as well, ascending, what has no room in front behind
    held, shares, free, span, n, bad = O.page_release(
        [0, 0], [3, 2], [[7, 3, 5], [2, 3, -1]], [0, 0, 0, 1, 0, 0, 0, 0], [4, 4, 4] + [0] * 5,
        [1, 2], 4)
    assert n == 4 and span == [0, 5] and free[:5] == [2, 4, 3, 5, 7]


def test_compact_example():
    table, shares, free, span, moves, bad = O.page_compact(
        [3, 2], [[7, 3, 5], [0, 3, 9]], [5, 0, 0, 1, 0, 2, 0, 3], [-1] * 8)
    assert moves == [(5, 1), (7, 2)] and span == [0, 4] and free[:4] == [4, 5, 6, 7]
    assert table.tolist() == [[2, 3, 1], [0, 3, -1]] and not bad
    assert shares.tolist() == [5, 2, 3, 1, 0, 0, 0, 0]


def test_copy_example():
    c = np.arange(12).reshape(4, 3)
    assert O.page_copy(c, [(0, 2, 2), (3, 1), (5, 0), (1, -1)], 3).tolist() == [
        [0, 1, 2], [9, 10, 11], [0, 1, 8], [9, 10, 11]]


def test_one_row_chunks_are_decode_attention():
    g = np.random.default_rng(0)
    kc, vc = g.standard_normal((9, 4, 2, 8)), g.standard_normal((9, 4, 2, 8))
    lens = [1, 7, 20]
    table = np.full((3, 5), -1)
    table[0, :1], table[1, :2], table[2, :5] = [4], [0, 8], [1, 2, 3, 5, 6]
    q = g.standard_normal((3, 4, 8))
    for window in (0, 5):
        a = O.chunk_attention(q, kc, vc, [t - 1 for t in lens], lens, [0, 1, 2, 3], table, window)
        b = P.decode_attention(q, kc, vc, lens, table, window)
        for x, y in zip(a[:4], b):
            assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


def test_chunk_rows_are_causal():
    g = np.random.default_rng(1)
    kc, vc = g.standard_normal((4, 4, 1, 8)), g.standard_normal((4, 4, 1, 8))
    table, q = np.array([[2, 0, 1, 3]]), g.standard_normal((6, 2, 8))
    out = O.chunk_attention(q, kc, vc, [5], [11], [0, 6], table)[0]
    for i in range(6):                       # row i alone, over the cache up to its position
        one = O.chunk_attention(q[i:i + 1], kc, vc, [5 + i], [6 + i], [0, 1], table)[0]
        assert np.allclose(out[i], one[0])
