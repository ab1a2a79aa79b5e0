"""Parity of the page pool calls (fork, release, compact, copy) with the oracle: whole numbers
and copied bytes, so everything is exact."""

import numpy as np
import pytest
import torch

from oracle import page_pool as O
from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def status():
    """Whether a page id outside the pool was met since the last look."""
    torch.cuda.synchronize()
    try:
        B.mla_device_status()
    except B.MlaError:
        return True
    return False


def pool(g, batch, page, tmax, idle=0.3, spare=1, extra=9, prompts=0):
    """A pool in use: lengths, pages held, table, shares, free list and its span.  With `prompts`
    pages at most, some sequences share the first one's."""
    lens = np.where(g.random(batch) < idle, 0, g.integers(1, tmax + 1, batch))
    held = np.where(lens > 0, -(-lens // page) + g.integers(0, spare + 1, batch), 0)
    W = int(held.max()) + 2
    table = np.full((batch, W), -1)
    common = min(prompts, int(lens[0]) // page)
    shares = {}
    owner = []
    for b in range(batch):
        lead = min(common, int(held[b])) if b and g.random() < 0.6 else 0
        for j in range(int(held[b])):
            owner.append((b, j) if j >= lead else (0, j))
    pages = len(set(owner)) + extra
    ids = iter(g.permutation(pages))
    where = {}
    it = iter(owner)
    for b in range(batch):
        for j in range(int(held[b])):
            o = next(it)
            if o in where:
                shares[where[o]] = shares.get(where[o], 0) + 1
            else:
                where[o] = int(next(ids))
            table[b, j] = where[o]
    rest = [int(x) for x in ids]
    count = np.zeros(pages, np.int64)
    for p, n in shares.items():
        count[p] = n
    free = np.full(pages + 4, -1)
    first = int(g.integers(0, 4))
    free[first:first + len(rest)] = rest
    return lens, held, table, count, free, [first, first + len(rest)]


def check_fork(src, lens, held, table, shares, free, span, page, in_place=False):
    t, s = i32(table), i32(shares)
    out = None
    if in_place:
        B_, P = len(lens), len(shares)
        z = lambda n: torch.full((n,), -5, dtype=torch.int32, device=DEV)  # noqa: E731
        out = B.PageFork(z(B_), z(B_), s, z(2), z(1), z(B_), z(B_), z(B_), z(1))
    got = B.mla_page_fork(i32(src), i32(lens), i32(held), t, s, i32(free), i32(span), page,
                          out=out)
    bad = status()
    wt, wl, wh, ws, wspan, missing, moves, wbad = O.page_fork(src, lens, held, table, shares, free,
                                                             span, page)
    assert np.array_equal(t.cpu().numpy(), wt)
    assert got.cache_lens.tolist() == wl and got.held_pages.tolist() == wh
    assert np.array_equal(got.shares.cpu().numpy(), ws)
    assert got.free_span.tolist() == wspan and got.missing.tolist() == [missing]
    n = got.moves.item()
    assert n == len(moves)
    assert [got.move_src[:n].tolist(), got.move_dst[:n].tolist(), got.move_rows[:n].tolist()] == \
        [list(x) for x in zip(*moves)] or n == 0
    assert bad == wbad
    return got, moves


@pytest.mark.parametrize("batch,page,tmax", [(1, 4, 10), (2, 1, 3), (7, 16, 100), (33, 8, 700),
                                             (300, 16, 200), (1025, 3, 40), (9000, 8, 30)])
@pytest.mark.parametrize("short", [False, True])
def test_fork_matches_oracle(batch, page, tmax, short):
    g = np.random.default_rng(batch + short)
    lens, held, table, shares, free, span = pool(g, batch, page, tmax, 0.6, extra=batch + 9,
                                                 prompts=3)
    if short:
        span[1] = span[0] + int(g.integers(0, max(1, batch // 4)))
    # any source: idle ones, itself, out of range, and slots that hold pages and are passed over
    src = np.where(g.random(batch) < 0.8, g.integers(0, batch, batch), g.integers(-3, batch + 3,
                                                                                batch))
    check_fork(src, lens, held, table, shares, free, span, page)
    check_fork(src, lens, held, table, shares, free, span, page, in_place=True)


def test_fork_odd_inputs():
    # negative and large counts, a length beyond the pages held, ids outside the pool, no source
    table = np.array([[3, 9, -1, 2], [0, 1, 2, 3], [-1] * 4, [-1] * 4, [-1] * 4, [-1] * 4])
    lens, held = [11, 1000, -7, 0, 5, 0], [3, 99, 0, -2, 0, 0]
    check_fork([5, 5, 0, 1, 2, 9], lens, held, table, [0] * 6, [5, 4], [0, 2], 4)
    check_fork([5, 5, 0, 0, 0, 0], lens, held, table, [0] * 6, [5, 4], [1, 7], 4)
    check_fork([5, 5, 1, 1, 1, 1], [1, 13, 0, 0, 0, 0], held, table, [0, 2, 0, 0, 0, 1], [5, 4],
               [-3, 1], 4)
    check_fork([-1] * 6, lens, held, table, [0] * 6, [5, 4], [2, 1], 4)


def check_release(kept, held, table, shares, free, span, page, in_place=False):
    s, f = i32(shares), i32(free)
    out = None
    if in_place:
        z = lambda n: torch.full((n,), -5, dtype=torch.int32, device=DEV)  # noqa: E731
        out = B.PageRelease(z(len(held)), s, z(2), z(1))
    got = B.mla_page_release(i32(kept), i32(held), i32(table), s, f, i32(span), page, out=out)
    bad = status()
    wh, ws, wf, wspan, n, wbad = O.page_release(kept, held, table, shares, free, span, page)
    assert got.held_pages.tolist() == wh
    assert np.array_equal(got.shares.cpu().numpy(), ws)
    assert f.tolist() == wf and got.free_span.tolist() == wspan and got.released.tolist() == [n]
    assert bad == wbad


@pytest.mark.parametrize("batch,page,tmax,prompts", [
    (1, 4, 10, 0), (2, 1, 3, 2), (7, 16, 100, 3), (33, 8, 700, 20), (300, 16, 200, 5),
    (1025, 3, 40, 4), (9000, 8, 30, 2), (3, 1, 30000, 100)])
@pytest.mark.parametrize("ends", [0.0, 0.5, 1.0])
def test_release_matches_oracle(batch, page, tmax, prompts, ends):
    g = np.random.default_rng(batch + int(10 * ends))
    lens, held, table, shares, free, span = pool(g, batch, page, tmax, 0.2, prompts=prompts)
    kept = np.where(g.random(batch) < ends, 0, np.maximum(lens - g.integers(0, 2 * page, batch),
                                                          -1))
    check_release(kept, held, table, shares, free, span, page)
    check_release(kept, held, table, shares, free, span, page, in_place=True)


def test_release_odd_inputs():
    table = np.array([[3, 9, -1, 2], [0, 1, 2, 3], [5, 5, 5, 5]])
    free = [-1] * 8
    # ids outside the pool, counts out of range, a page twice without a share
    check_release([0, 0, 0], [4, 0, 0], table, [0] * 6, free, [8, 8], 4)
    check_release([-5, 1000, 3], [1, 99, 4], table, [0, 0, 0, 1, 0, 0], free, [3, 4], 4)
    check_release([0, 0, 16], [0, 4, 9], table, [0, 0, 1, 0, 0, 0], free, [-2, 3], 4)
    check_release([0, 5, 16], [0, 2, 9], table, [0, 0, 1, 0, 0, 0], free, [1, 1], 4)


def check_compact(held, table, shares, free, in_place=False):
    t, s, f = i32(table), i32(shares), i32(free)
    out = None
    if in_place:
        z = lambda n: torch.full((n,), -5, dtype=torch.int32, device=DEV)  # noqa: E731
        m = max(1, len(shares) // 2)
        out = B.PageCompact(t, s, z(2), z(m), z(m), z(1))
    got = B.mla_page_compact(i32(held), t, s, f, out=out)
    bad = status()
    wt, ws, wf, wspan, moves, wbad = O.page_compact(held, table, shares, free)
    n = got.moves.item()
    assert n == len(moves)
    assert n == 0 or [got.move_src[:n].tolist(), got.move_dst[:n].tolist()] == [
        list(x) for x in zip(*moves)]
    assert np.array_equal(got.shares.cpu().numpy(), ws)
    assert f.tolist() == wf and got.free_span.tolist() == wspan
    # (an id outside the pool stays what it is)
    assert np.array_equal(got.page_table.cpu().numpy(), wt) and bad == wbad
    return got


@pytest.mark.parametrize("batch,page,tmax,prompts,extra", [
    (1, 4, 10, 0, 0), (1, 4, 10, 0, 50), (2, 1, 3, 2, 5), (7, 16, 100, 3, 3), (33, 8, 700, 20, 900),
    (300, 16, 200, 5, 1000), (1025, 3, 40, 4, 3), (9000, 8, 30, 2, 20000), (3, 1, 30000, 100, 9)])
def test_compact_matches_oracle(batch, page, tmax, prompts, extra):
    g = np.random.default_rng(batch + extra)
    _, held, table, shares, free, _ = pool(g, batch, page, tmax, 0.2, extra=extra, prompts=prompts)
    check_compact(held, table, shares, free)
    check_compact(held, table, shares, free, in_place=True)


def test_compact_odd_inputs():
    table = np.array([[3, 9, -1, 2], [0, 1, 2, 3], [5, 5, 5, 5]])
    check_compact([4, -1, 0], table, [7, 0, 1, 2, 3, 4], [-1] * 6)
    check_compact([0, 0, 9], table, [0, 0, 0, 0, 0, 3], [-1] * 7)
    check_compact([0, 0, 0], table, [0] * 6, [-1] * 6)
    check_compact([0], np.array([[0]]), [0], [-1])
    check_compact([1], np.array([[0]]), [0], [-1])


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("counted", [False, True])
def test_copy_matches_oracle(page, partial, counted):
    g, gen = np.random.default_rng(page), torch.Generator(DEV).manual_seed(page)
    P, n = 37, 14
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    wide = r(P, page, 2, 3, 96)
    caches = [
        r(P, page, 512).to(BF16), r(P, page, 64).to(BF16),              # latents and RoPE keys
        r(P, page, 576).to(BF16)[..., :512],                            # one packed cache's part
        r(P, page, 4, 128).to(BF16), r(P, 4, page, 128).to(BF16).transpose(1, 2),
        r(P, page, 5, 80), r(P, 3, page, 48).to(torch.float8_e4m3fn).transpose(1, 2),
        r(page, P, 2, 64).transpose(0, 1),                              # pages interleaved
        wide[:, :, 0], wide[:, :, 1],                                   # keys and values in one
        r(P, page, 1, 8).to(BF16), r(P, page, 7, 1024).to(BF16),
    ]
    perm = g.permutation(P)
    src, dst = perm[:n], perm[n:2 * n]
    rows = g.integers(-1, page + 2, n) if partial else None
    live = 9 if counted else n
    before = [c.clone() for c in caches]
    B.mla_page_copy(caches, i32(src), i32(dst), i32([live]) if counted else None,
                    i32(rows) if partial else None)
    assert not status()
    for i, (b, c) in enumerate(zip(before, caches)):
        moves = [(src[m], dst[m]) + ((rows[m],) if partial else ()) for m in range(live)]
        assert np.array_equal(bits(c), bits(torch.as_tensor(O.page_copy(
            b.view(torch.uint8).cpu().numpy() if b.is_contiguous() else
            b.contiguous().view(torch.uint8).cpu().numpy(), moves, page)))), i


def test_copy_odd_moves():
    c = torch.arange(6 * 4 * 16, device=DEV, dtype=torch.float32).view(6, 4, 16)
    before = c.clone()
    # pages outside the pool are passed over and reported; counts below zero and beyond the list
    B.mla_page_copy([c], i32([6, 0, -1, 2]), i32([1, 9, 3, 4]))
    assert status()
    before[4] = before[2]
    assert torch.equal(c, before)
    B.mla_page_copy([c], i32([0]), i32([1]), i32([-4]))
    B.mla_page_copy([c], i32([]), i32([]))
    assert not status() and torch.equal(c, before)
    B.mla_page_copy([c], i32([0]), i32([1]), i32([2 ** 31 - 1]))
    before[1] = before[0]
    assert not status() and torch.equal(c, before)


def test_copy_many_views_and_pages():
    gen = torch.Generator(DEV).manual_seed(3)
    caches = [torch.randn(300, 16, 2, 64, generator=gen, device=DEV).to(BF16) for _ in range(128)]
    before = [c.clone() for c in caches]
    src, dst = i32(range(150)), i32(range(299, 149, -1))
    B.mla_page_copy(caches, src, dst)
    assert not status()
    for b, c in zip(before, caches):
        b[dst.long()] = b[src.long()]
        assert torch.equal(b, c)
    with pytest.raises(B.MlaError, match="views"):
        B.mla_page_copy(caches + [caches[0].clone()], src, dst)
