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
