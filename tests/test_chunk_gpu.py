"""Parity of the chunk attention (a step's new rows over a paged key/value cache) with the
float64 oracle, at the lengths, masks, layouts and contents where it can go wrong.

Tolerances, derived from the roundings the kernels make:
* an output stored in type t is off by at most half a step, u(t) of its size (bf16 2^-8, fp32
  2^-24);
* a score is a sum of D products accumulated in fp32, each addition off by at most 2^-23 (the
  tensor cores may cut off instead of rounding): ds = (D + 4) * 2^-23 * max_t scale * sum |q k|
  (beside an e4m3 cache queries are fp16 relative to their head's largest element, 2^-24 * scale
  * |q|max * sum |k|, folded in by doubling);
* a weight exp(s - m) is off by 2 ds (its own and the maximum's), by the exponential's 2^-21, and
  by its rounding before the second product, 2^-8 (bf16) or 2^-11 (fp16 beside an e4m3 cache;
  none for fp32); sums over n positions add n * 2^-23.  The weighted sum's error is all of that
  times sum p |v|, and the sum of the weights carries the same relative error, which doubles it.
"""

import numpy as np
import pytest
import torch

from oracle import page_pool as O
from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3, BF16, FP32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def npy(t):
    return t.detach().to(torch.float64).cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def randn(gen, *shape, dtype=FP32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)


def case(kept, new, H, Hk, D, page, dtype=BF16, cache=None, by_head=False, seed=0, spread=1.0,
         lens=None, pad=0, poison=True, width=None):
    """A step's queries and caches; cache rows behind each sequence hold NaN, pages are shuffled,
    tables hold -1 behind a sequence's pages."""
    cache = cache or dtype
    g, gen = np.random.default_rng(seed), torch.Generator(DEV).manual_seed(seed)
    lens = lens or [max(k, 0) + n for k, n in zip(kept, new)]
    used = [max(0, -(-t // page)) for t in lens]
    W = width or max(max(used), 1)
    used = [min(u, W) for u in used]
    pages = sum(used) + 2
    ids = g.permutation(pages)
    table = np.full((len(lens), W), -1)
    shape = (pages, Hk, page, D) if by_head else (pages, page, Hk, D)
    kc, vc = (randn(gen, *shape, scale=s * (60.0 if cache == E4M3 else 1.0)).clamp(
        -448.0, 448.0).to(cache) for s in (spread, 1.0))
    if by_head:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    live = np.zeros((pages, page), bool)
    at = 0
    for b, t in enumerate(lens):
        t = min(max(t, 0), W * page)
        table[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
        pos = np.arange(t)
        live[table[b, pos // page], pos % page] = True
    if poison:
        dead = torch.tensor(~live, device=DEV)
        for c in (kc, vc):
            if cache == E4M3:
                c.view(torch.uint8)[dead] = 0x7F
            else:
                c[dead] = float("nan")
    ks = vs = None
    if cache == E4M3:
        ks, vs = (torch.rand(Hk, generator=gen, device=DEV) * 0.01 + 0.01 for _ in range(2))
    starts = np.concatenate([[0], np.cumsum(new)])
    q = randn(gen, int(starts[-1]) + pad, H, D, dtype=dtype)
    return dict(q=q, k_cache=kc, v_cache=vc, kept_lens=i32(kept), cache_lens=i32(lens),
                row_start=i32(starts), page_table=i32(table), k_scale=ks, v_scale=vs)


def oracle(c, window=0, scale=None):
    sc = lambda x: None if x is None else npy(x)  # noqa: E731
    ints = [c[n].cpu().numpy() for n in ("kept_lens", "cache_lens", "row_start", "page_table")]
    return O.chunk_attention(npy(c["q"]), npy(c["k_cache"]), npy(c["v_cache"]), *ints, window,
                             scale, sc(c["k_scale"]), sc(c["v_scale"]))


def run(c, **kw):
    """Outputs over a background that shows what was written, and the status word."""
    N, H, D = c["q"].shape
    out = torch.full((N, H, D), 7.0, dtype=c["q"].dtype, device=DEV)
    lse = torch.full((N, H), 7.0, device=DEV)
    B.mla_chunk_attention(**c, **kw, out=out, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def check(c, out, lse, window=0, scale=None, what="", want=None):
    q, cache = c["q"], c["k_cache"].dtype
    D = q.shape[-1]
    want, want_lse, vabs, big, written = want or oracle(c, window, scale)
    out, lse = npy(out), npy(lse)
    assert (out[~written] == 7.0).all() and (lse[~written] == 7.0).all(), what + " other rows"
    n = int(max(1, c["cache_lens"].max().item()))
    ds = (D + 4) * 2.0 ** -23 * big * (2 if cache == E4M3 else 1)
    weights = {FP32: 0.0, BF16: 2.0 ** -8, E4M3: 2.0 ** -11}[cache]
    rel = 2 * (2 * ds + 2.0 ** -21 + weights + n * 2.0 ** -23)[..., None]
    tol = U[q.dtype] * np.abs(want) * (1 + 2.0 ** -7) + rel * vabs + 1e-30
    bad = ~(np.abs(out - want) <= tol) & written[:, None, None]
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(out - want)[bad])} at {np.argwhere(bad)[0]}: got "
                           f"{out[bad][0]}, want {want[bad][0]}, tolerance {tol[bad][0]}")
    fin = np.isfinite(want_lse)
    assert (lse[~fin & written[:, None]] == -np.inf).all(), what + " empty rows"
    tol = 2 * ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(fin, want_lse, 0))
    bad = ~(np.abs(lse - np.where(fin, want_lse, 0)) <= tol) & fin & written[:, None]
    assert not bad.any(), f"{what} lse: {bad.sum()} off at {np.argwhere(bad)[0]}"


KEPT = [0, 0, 0, 1, 15, 63, 64, 65, 127, 128, 129, 250, 255, 0, 300]
NEW = [1, 2, 0, 3, 16, 1, 64, 7, 1, 5, 130, 9, 2, 33, 0]

CASES = [
    # kept, new, H, Hk, D, page, dtype, cache, by_head, window
    ([0], [1], 1, 1, 64, 16, BF16, BF16, False, 0),
    ([56], [5], 16, 8, 64, 16, BF16, BF16, False, 0),
    (KEPT, NEW, 8, 2, 128, 64, BF16, BF16, False, 0),
    (KEPT, NEW, 8, 2, 128, 16, BF16, E4M3, True, 0),
    (KEPT, NEW, 6, 2, 64, 8, FP32, FP32, False, 0),
    (KEPT, NEW, 4, 4, 64, 24, BF16, BF16, True, 50),
    (KEPT, NEW, 4, 2, 80, 7, BF16, BF16, False, 64),
    (KEPT, NEW, 5, 1, 96, 1, BF16, E4M3, False, 17),
    (KEPT, NEW, 5, 1, 40, 5, FP32, FP32, True, 33),
    (KEPT, NEW, 2, 2, 112, 20, BF16, BF16, False, 129),
    (KEPT, NEW, 4, 1, 192, 32, BF16, BF16, False, 0),
    (KEPT, NEW, 3, 1, 256, 128, BF16, BF16, True, 0),
    (KEPT, NEW, 4, 2, 256, 64, BF16, E4M3, False, 100),
    (KEPT, NEW, 3, 3, 8, 16, BF16, BF16, False, 0),
    (KEPT, NEW, 7, 1, 16, 16, BF16, E4M3, False, 0),
    (KEPT, NEW, 3, 3, 4, 16, FP32, FP32, False, 0),
    (KEPT, NEW, 2, 1, 136, 48, BF16, BF16, False, 0),
    (KEPT, NEW, 2, 1, 208, 6, BF16, E4M3, True, 0),
    ([1000, 3], [300, 2], 12, 1, 128, 64, BF16, BF16, False, 0),
    ([1000, 3], [30, 2], 160, 1, 64, 32, BF16, BF16, False, 0),
    ([1000, 3], [30, 2], 33, 3, 192, 16, BF16, BF16, True, 0),
    ([1000, 3], [30, 2], 17, 1, 200, 16, FP32, FP32, False, 100),
    ([20000], [4], 8, 1, 128, 64, BF16, BF16, True, 0),
    ([15000], [3], 4, 2, 64, 128, BF16, E4M3, False, 0),
    ([9000, 4000], [2, 40], 2, 1, 128, 100, FP32, FP32, False, 0),
    ([5000], [100], 4, 1, 96, 64, BF16, BF16, False, 700),
    ([3, 0, 1, 9] * 40, [1, 0, 2, 4] * 40, 4, 2, 64, 16, BF16, BF16, False, 0),
    ([0, 5, 0], [0, 0, 0], 8, 2, 128, 16, BF16, BF16, False, 0),
]


@pytest.mark.parametrize("kept,new,H,Hk,D,page,dtype,cache,by_head,window", CASES)
def test_chunk_matches_oracle(kept, new, H, Hk, D, page, dtype, cache, by_head, window):
    c = case(kept, new, H, Hk, D, page, dtype, cache, by_head, seed=len(kept) + D, pad=3)
    out, lse = run(c, window=window)
    B.mla_device_status()
    check(c, out, lse, window)
    again, lse2 = run(c, window=window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)    # the same bits each time


def test_chunk_scale_and_sharp_scores():
    for cache in (BF16, E4M3, FP32):
        c = case([0, 700], [200, 3], 4, 2, 64, 16, FP32 if cache == FP32 else BF16, cache, seed=5,
                 spread=4.0)
        out, lse = run(c, scale=0.5)
        check(c, out, lse, scale=0.5, what=str(cache))


def test_chunk_lengths_that_do_not_match_the_rows():
    # the free list ran out (fewer cached rows than the step's last positions), a window that
    # ends behind the cached rows, no cached rows, counts out of range
    kept, new = [100, 300, 40, -5, 0, 2 ** 31 - 1], [30, 9, 5, 20, 3, 4]
    lens = [110, 200, 0, -3, 2, 150]
    for window in (0, 50):
        for dtype, cache in ((BF16, BF16), (BF16, E4M3), (FP32, FP32)):
            c = case(kept, new, 6, 2, 64, 16, dtype, cache, seed=6, lens=lens, pad=2)
            out, lse = run(c, window=window)
            B.mla_device_status()
            check(c, out, lse, window, what=f"{cache} {window}")
            assert not out[139 - 100:].isnan().any()


def test_chunk_rows_outside_every_sequence():
    c = case([50, 60, 70], [4, 5, 6], 4, 2, 64, 16, seed=7, pad=10)
    c["row_start"] = i32([3, 7, 7, 18])      # rows 0-2 and 18 on belong to nobody
    out, lse = run(c)
    check(c, out, lse)
    c["row_start"] = i32([5, 2, 9, 4000])    # descending, and beyond the rows
    out, lse = run(c)
    want = list(oracle({**c, "row_start": i32([0, 0, 0, 0])}))
    third = oracle({**c, "row_start": i32([9, 9, 9, 25])})
    second = oracle({**c, "row_start": i32([2, 2, 9, 9])})
    for i in range(5):
        want[i] = np.where(third[4].reshape([-1] + [1] * (want[i].ndim - 1)), third[i], want[i])
        want[i] = np.where(second[4].reshape([-1] + [1] * (want[i].ndim - 1)), second[i], want[i])
    check(c, out, lse, want=want)
    B.mla_device_status()


def hit(c, which, b, t, h, d, value):
    page = c["k_cache"].shape[1]
    cache = c[which]
    at = (c["page_table"][b, t // page].item(), t % page, h, d)
    if cache.dtype == E4M3:
        cache.view(torch.uint8)[at] = value
    else:
        cache[at] = value


@pytest.mark.parametrize("dtype,cache,page,D", [(BF16, BF16, 16, 128), (BF16, BF16, 5, 64),
                                                (BF16, E4M3, 16, 128), (FP32, FP32, 16, 64),
                                                (BF16, BF16, 8, 256), (BF16, E4M3, 3, 192)])
@pytest.mark.parametrize("rows", [6, 150])
def test_chunk_hidden_values_may_be_anything(dtype, cache, page, D, rows):
    """NaN and infinities at positions that some rows see and others do not: those others'
    results are what they were, and the seen ones' columns are not finite."""
    kept, window = 200, 120
    c = case([kept, 7], [rows, 2], 4, 2, D, page, dtype, cache, seed=8)
    clean, clean_lse = run(c, window=window)
    mid = kept + rows // 2
    nan, inf = (0x7F, None) if cache == E4M3 else (float("nan"), float("inf"))
    hit(c, "v_cache", 0, mid, 0, 3, nan)                  # rows from rows // 2 on see it
    if inf:
        hit(c, "v_cache", 0, mid, 1, 5, inf)
        hit(c, "v_cache", 0, kept + rows - 1, 0, 9, -inf)  # the last row alone
    hit(c, "v_cache", 0, kept - window + 2, 1, 7, nan)    # the first rows' window alone
    hit(c, "k_cache", 0, kept + rows - 1, 1, 0, nan)      # a key: the last row's heads of one
    out, lse = run(c, window=window)
    B.mla_device_status()
    o, z = npy(out), npy(clean)
    pos = kept + np.arange(rows)
    bad = np.zeros(o.shape, bool)
    sees = lambda t: (pos >= t) & (pos < t + window)      # noqa: E731
    bad[:rows, :2, 3] |= sees(mid)[:, None]
    if inf:
        bad[:rows, 2:, 5] |= sees(mid)[:, None]
        assert (o[:rows, 2:, 5][sees(mid)][:-1] == np.inf).all()
        bad[rows - 1, :2, 9] = True
        assert (o[rows - 1, :2, 9] == -np.inf).all()
    bad[:rows, 2:, 7] |= sees(kept - window + 2)[:, None]
    bad[rows - 1, 2:] = True
    assert not np.isfinite(o[bad]).any()
    assert np.array_equal(o[~bad], z[~bad])
    keep = np.ones(lse.shape, bool)
    keep[rows - 1, 2:] = False
    assert np.array_equal(npy(lse)[keep], npy(clean_lse)[keep])
    assert np.isnan(npy(lse)[~keep]).all()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (BF16, E4M3), (FP32, FP32)])
def test_chunk_infinite_scores(dtype, cache):
    c = case([140, 0], [5, 40], 2, 1, 64, 16, dtype, cache, seed=12)
    big = 448.0 if cache == E4M3 else float("inf")
    c["q"][:, :, 0] = -1.0 if cache != E4M3 else -float("inf")
    for t in range(150):                                  # every score of sequence 0: -inf
        if t < 145:
            c["k_cache"][c["page_table"][0, t // 16].item(), t % 16, 0, 0] = big
    out, lse = run(c)
    o = npy(out)
    if cache == E4M3:                                     # -inf * 448 + ...: -inf as well
        assert (npy(lse)[:5] == -np.inf).all() and not o[:5].any()
    else:
        assert not o[:5].any() and (npy(lse)[:5] == -np.inf).all()
    c = case([140], [5], 2, 1, 64, 16, dtype, cache, seed=13)
    c["q"][2, 1, 4] = float("nan")                        # a query: its head alone
    out, lse = run(c)
    o = npy(out)
    assert np.isnan(o[2, 1]).all() and np.isnan(npy(lse)[2, 1])
    o[2, 1] = 0
    assert np.isfinite(o).all()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (FP32, FP32)])
def test_chunk_scores_of_any_finite_size(dtype, cache):
    # scores of 2^21 to 2^40: sums round, but weights of equal scores stay equal and finite
    for scale in (2.0 ** 21, 2.0 ** 33, 2.0 ** 40):
        c = case([300], [4], 2, 1, 64, 16, dtype, cache, seed=14)
        c["q"].zero_()
        c["q"][:, :, 0] = scale
        live = c["page_table"][0].long()
        c["k_cache"][live] = 0.0
        c["k_cache"][live, :, :, 0] = 1.0                 # all the same ...
        hit(c, "k_cache", 0, 100, 0, 0, 2.0)              # ... but one, which takes it all
        out, lse = run(c, scale=1.0)
        v = npy(c["v_cache"][live[100 // 16], 100 % 16, 0])
        assert np.allclose(npy(out), v, rtol=2.0 ** -7, atol=0)
        assert np.allclose(npy(lse), 2 * scale, rtol=2.0 ** -20)
        hit(c, "k_cache", 0, 100, 0, 0, 1.0)              # none: the average of the values
        out, lse = run(c, scale=1.0)
        got = npy(out)
        assert np.isfinite(got).all() and np.isfinite(npy(lse)).all()
        vals = npy(c["v_cache"][live].flatten(0, 1)[:301, 0])
        assert np.abs(got[0, 0] - vals.mean(0)).max() <= 2.0 ** -7 * np.abs(vals).max()


def test_chunk_odd_scales():
    c = case([130], [4], 8, 4, 64, 16, BF16, E4M3, seed=15)
    c["k_scale"].copy_(torch.tensor([float("nan"), float("inf"), 0.0, -0.02], device=DEV))
    c["v_scale"].copy_(torch.tensor([0.01, 0.01, -0.5, 0.0], device=DEV))
    out, lse = run(c)
    o = npy(out)
    assert np.isnan(o[:, :4]).all() and np.isnan(npy(lse)[:, :4]).all()
    # a zero scale: the average; a negative one: the signs turned
    want, want_lse, vabs, _, _ = oracle({**c, "k_scale": torch.nan_to_num(c["k_scale"], posinf=1.0)})
    assert np.abs(o[:, 4:6] - want[:, 4:6]).max() <= 2.0 ** -6 * vabs[:, 4:6].max()
    assert np.abs(npy(lse)[:, 4:] - want_lse[:, 4:]).max() <= 1e-3
    assert not o[:, 6:].any()


@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
@pytest.mark.parametrize("page", [16, 3])
def test_chunk_table_capacity_and_bad_pages(cache, page):
    dtype = FP32 if cache == FP32 else BF16
    c = case([190, 60, 85], [10, 4, 5], 4, 2, 64, page, dtype, cache, seed=16, width=80 // page)
    out, lse = run(c)                                     # 200 and 90 count as what the table holds
    B.mla_device_status()
    check(c, out, lse)
    c["page_table"][1, 2] = c["k_cache"].shape[0]         # reads as zeros, reported
    c["page_table"][2, 0] = -7
    out, lse = run(c)
    check(c, out, lse)
    with pytest.raises(B.MlaError, match="page id"):
        B.mla_device_status()


@pytest.mark.parametrize("batch,idle", [(257, 0.2), (2100, 0.5), (5000, 0.995), (300, 1.0)])
def test_chunk_many_sequences(batch, idle):
    g = np.random.default_rng(batch)
    new = np.where(g.random(batch) < idle, 0, g.integers(1, 5, batch))
    kept = np.where(new > 0, g.integers(0, 60, batch), 0)
    if idle < 1:
        kept[[3, batch - 2]], new[[3, batch - 2]] = [900, 1500], [40, 9]
    c = case(kept.tolist(), new.tolist(), 4, 2, 64, 16, seed=batch, pad=1)
    out, lse = run(c)
    check(c, out, lse)
    again, lse2 = run(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_chunk_many_heads_and_units():
    for H, Hk, n in ((96, 96, 5), (256, 2, 7), (300, 1, 3), (2, 1, 700)):
        c = case([120, 4], [n, 1], H, Hk, 64, 32, seed=H)
        out, lse = run(c)
        check(c, out, lse, what=str((H, Hk)))


def test_chunk_single_rows_are_decode_attention():
    """One row per sequence: what the decode attention gives, within both calls' roundings."""
    lens = [1, 2, 63, 64, 65, 128, 129, 500, 2000]
    for cache in (BF16, E4M3):
        c = case([t - 1 for t in lens], [1] * len(lens), 8, 2, 128, 16, BF16, cache, seed=17)
        out, lse = run(c)
        d, dl = B.mla_decode_attention(c["q"], c["k_cache"], c["v_cache"], c["cache_lens"],
                                       c["page_table"], k_scale=c["k_scale"],
                                       v_scale=c["v_scale"], return_lse=True)
        torch.cuda.synchronize()
        check(c, out, lse)
        check(c, d, dl)


def test_chunk_strided_inputs():
    c = case([100, 37], [20, 3], 8, 2, 128, 16, seed=18)
    pages = c["k_cache"].shape[0]
    qkv = torch.randn(23, 12, 128, device=DEV).to(BF16)
    both = torch.full((pages, 2, 16, 3, 136), float("nan"), dtype=BF16, device=DEV)
    both[:, 0, :, :2, :128] = c["k_cache"]
    both[:, 1, :, :2, :128] = c["v_cache"]
    want = run({**c, "q": qkv[:, :8].contiguous()})
    got = run({**c, "q": qkv[:, :8], "k_cache": both[:, 0, :, :2, :128],
               "v_cache": both[:, 1, :, :2, :128]})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cache", [E4M3, BF16])
def test_chunk_offsets_beyond_32_bits(cache):
    # caches of more than 2^32 elements; the sequences use pages at both ends
    page, Hk, D = 64, 1, 128
    pages = 540000
    size = 1 if cache == E4M3 else 2
    if torch.cuda.mem_get_info()[0] < (12 * size) << 30:
        pytest.skip("needs the memory")
    kind = torch.uint8 if cache == E4M3 else cache
    kc, vc = (torch.empty(pages, page, Hk, D, dtype=kind, device=DEV) for _ in range(2))
    kept, new = [120, 196], [10, 4]
    table = i32([[539999, 0, 539990, 1], [524288, 524287, 530001, 2]])
    small = case(kept, new, 4, Hk, D, page, BF16, cache, seed=1)
    for c, s in ((kc, small["k_cache"]), (vc, small["v_cache"])):
        for b in range(2):
            n = -(-(kept[b] + new[b]) // page)
            x = s[small["page_table"][b, :n].long()]
            c[table[b, :n].long()] = x.view(torch.uint8) if cache == E4M3 else x
    want = run(small)
    got = run({**small, "k_cache": kc.view(cache), "v_cache": vc.view(cache), "page_table": table})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # (rows one by one as well: pages of 4 rows)
    if cache == BF16:
        t4 = (table.long()[:, :, None] * 16 + torch.arange(16, device=DEV)).flatten(1).int()
        got = run({**small, "k_cache": kc.view(-1, 4, Hk, D), "v_cache": vc.view(-1, 4, Hk, D),
                   "page_table": t4.contiguous()})
        check(small, *got)
    del kc, vc
    torch.cuda.empty_cache()


def test_chunk_graph_follows_lengths_and_tables():
    c = case([480, 0, 77, 20], [20, 300, 3, 5], 8, 2, 128, 16, seed=21, poison=False)
    call = B.PreparedChunkAttention(**c, return_lse=True)
    call.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for kept, new in (([480, 0, 77, 20], [20, 300, 3, 5]), ([3, 100, 0, 9], [1, 8, 0, 40]),
                      ([0, 0, 0, 0], [0, 0, 0, 0]), ([490, 299, 79, 24], [1, 1, 1, 1])):
        c["kept_lens"].copy_(i32(kept))
        c["cache_lens"].copy_(i32([k + n for k, n in zip(kept, new)]))
        c["row_start"].copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        call.out.fill_(7.0)
        call.lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(c, call.out, call.lse, what=str(new))
    # (the second step's last sequence is longer than its pages: zeros, and reported)
    with pytest.raises(B.MlaError, match="page id"):
        B.mla_device_status()


def test_chunk_graphs_sharing_a_workspace_and_streams():
    cs = [case([3000, 200], [9, 100], 8, 2, 128, 16, seed=41),
          case([50, 1000, 700], [3, 1, 90], 4, 1, 64, 16, FP32, FP32, seed=42),
          case([2000, 5], [30, 1], 8, 1, 128, 16, BF16, E4M3, seed=43)]
    want = [oracle(c) for c in cs]
    need = [B.mla_chunk_workspace_bytes(c["q"].shape[1], c["k_cache"].shape[2], c["q"].shape[2],
                                        c["page_table"].shape[0], c["q"].shape[0], 16,
                                        c["page_table"].shape[1], c["q"].dtype,
                                        c["k_cache"].dtype) for c in cs]
    ws = torch.full((max(need),), 0x7F, dtype=torch.uint8, device=DEV)   # (any contents will do)
    calls = [B.PreparedChunkAttention(**c, return_lse=True, workspace=ws) for c in cs]
    graphs = []
    for call in calls:
        call.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call.run()
    for i in (0, 1, 2, 1, 0, 2, 2, 0):                                   # one after the other
        calls[i].out.fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        check(cs[i], calls[i].out, calls[i].lse, want=want[i])
    streams = [torch.cuda.Stream() for _ in cs]                          # side by side
    for _ in range(4):
        got = [B.mla_chunk_attention(**c, return_lse=True, stream=s.cuda_stream)
               for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        for c, g, w in zip(cs, got, want):
            check(c, *g, want=w)
    call, other = calls[0], torch.cuda.Stream()
    for stream in (None, other.cuda_stream, 0):
        call.out.fill_(7.0)
        torch.cuda.synchronize()
        call.run(stream)
        torch.cuda.synchronize()
        check(cs[0], call.out, call.lse, want=want[0])


def test_chunk_small_workspace_is_refused_and_no_rows_are_no_work():
    c = case([100], [4], 4, 2, 64, 16, seed=50)
    with pytest.raises(B.MlaError, match="workspace"):
        B.mla_chunk_attention(**c, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    empty = {**c, "q": c["q"][:0], "row_start": i32([0, 0])}
    out, lse = B.mla_chunk_attention(**empty, return_lse=True)
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    with pytest.raises(B.MlaError, match="overlaps"):
        B.mla_chunk_attention(**c, out=c["q"])
    B.mla_device_status()
