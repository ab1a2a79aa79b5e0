"""Pins of the paged-step oracle (no GPU): worked examples by hand, invariants
of the page accounting, torch's double-precision attention, and e4m3 rounding
against the type's own table of values."""

import math

import numpy as np
import pytest
import torch

from oracle import paged as P


def test_page_step_by_hand():
    # pages of 4 rows; sequence 0 keeps 3 rows on 1 page and adds 3 (needs 2 pages);
    # sequence 1 is idle; sequence 2 starts from nothing and adds 5 (needs 2 pages)
    table = [[7, -1, -1], [2, 3, -1], [-1, -1, -1]]
    t, lens, held, rs, pos, slots, span, missing, bad = P.page_step(
        [3, 6, 0], [3, 0, 5], [1, 2, 0], table, [9, 5, 1, 0, 4], [1, 5], 4, 10, 10)
    assert t.tolist() == [[7, 5, -1], [2, 3, -1], [1, 0, -1]]
    assert lens.tolist() == [6, 6, 5] and held.tolist() == [2, 2, 2]
    assert rs.tolist() == [0, 3, 3, 8] and span.tolist() == [4, 5] and missing == 0
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, -1, -1]
    assert slots.tolist() == [31, 20, 21, 4, 5, 6, 7, 0, -1, -1] and not bad


def test_page_step_runs_out_of_pages():
    t, lens, held, rs, pos, slots, span, missing, _ = P.page_step(
        [0, 0], [9, 4], [0, 0], [[-1] * 3, [-1] * 3], [6, 8], [0, 2], 4, 9, 13)
    assert lens.tolist() == [8, 0] and held.tolist() == [2, 0] and missing == 2
    assert slots.tolist() == [24, 25, 26, 27, 32, 33, 34, 35, -1, -1, -1, -1, -1]
    assert pos.tolist()[-4:] == [0, 1, 2, 3] and span.tolist() == [2, 2]


@pytest.mark.parametrize("seed", range(6))
def test_page_step_invariants(seed):
    g = np.random.default_rng(seed)
    B, page, W = 9, int(g.integers(1, 9)), 12
    kept = g.integers(0, page * 6, B)
    held = -(-kept // page) + g.integers(0, 2, B)
    new = g.integers(0, page * 5, B)
    ids = g.permutation(400)
    table = np.full((B, W), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    t, lens, held2, rs, pos, slots, span, missing, bad = P.page_step(
        kept, new, held, table, ids[at:], [0, 400 - at], page, 400, int(new.sum()))
    live = slots[slots >= 0]
    assert len(set(live.tolist())) == len(live) and not bad and missing == 0
    used = t[t >= 0]
    assert len(set(used.tolist())) == len(used)            # no page twice
    assert np.array_equal(lens, kept + new) and np.array_equal(rs[1:], np.cumsum(new))
    for b in range(B):                                     # a row's slot is its table's
        for i in range(rs[b], rs[b + 1]):
            assert slots[i] == t[b, pos[i] // page] * page + pos[i] % page


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    g = np.random.default_rng(3)
    x, a = g.standard_normal((5, 32)), g.standard_normal(16)
    row = np.concatenate([np.cos(a), np.sin(a)])
    y = P.rotate(x, row, interleaved)
    z = (x[:, 0::2] + 1j * x[:, 1::2]) if interleaved else (x[:, :16] + 1j * x[:, 16:])
    w = (y[:, 0::2] + 1j * y[:, 1::2]) if interleaved else (y[:, :16] + 1j * y[:, 16:])
    np.testing.assert_allclose(w, z * np.exp(1j * a), rtol=1e-12, atol=1e-12)


def test_e4m3_rounding_matches_the_type():
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    values = np.unique(values[np.isfinite(values)])
    assert np.array_equal(P.round_e4m3(values), values)
    mid = (values[1:] + values[:-1]) / 2
    for x, lo, hi in zip(mid, values[:-1], values[1:]):
        assert P.round_e4m3(x) in (lo, hi)
        assert P.round_e4m3(x + abs(x) * 1e-9 + 1e-12) == hi
    x = np.random.default_rng(0).standard_normal(4000) * 30
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.round_e4m3(x.astype(np.float32)), want)
    assert P.round_e4m3(1e9) == 448 and P.round_e4m3(-1e9) == -448


def test_decode_attention_is_softmax_attention():
    g = np.random.default_rng(5)
    B, H, Hk, D, page = 3, 6, 2, 16, 4
    k, v = g.standard_normal((20, page, Hk, D)), g.standard_normal((20, page, Hk, D))
    table = g.permutation(20)[:18].reshape(B, 6)
    lens, q = [0, 1, 23], g.standard_normal((B, H, D))
    out, lse, vabs, big = P.decode_attention(q, k, v, lens, table)
    assert not out[0].any() and np.isinf(lse[0]).all()
    np.testing.assert_allclose(out[1], np.repeat(v[table[1, 0], 0], 3, 0), rtol=1e-14)
    kk, vv = (x[table[2]].reshape(-1, Hk, D)[:23].transpose(1, 0, 2).repeat(3, 0) for x in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[2][:, None]), torch.from_numpy(kk), torch.from_numpy(vv))
    np.testing.assert_allclose(out[2], ref[:, 0].numpy(), rtol=1e-10, atol=1e-12)
    win = P.decode_attention(q, k, v, lens, table, window=5)[0]
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[2][:, None]), torch.from_numpy(kk[:, 18:]), torch.from_numpy(vv[:, 18:]))
    np.testing.assert_allclose(win[2], ref[:, 0].numpy(), rtol=1e-10, atol=1e-12)
    s = np.einsum("hd,htd->ht", q[2], kk) / math.sqrt(D)
    np.testing.assert_allclose(lse[2], np.log(np.exp(s).sum(1)), rtol=1e-12)
    assert (vabs[2] >= np.abs(out[2]) - 1e-12).all() and (big[2] >= np.abs(s).max(1) - 1e-12).all()
