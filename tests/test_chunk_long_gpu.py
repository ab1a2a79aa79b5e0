"""The chunk attention over long caches, cut into parts: every stretch of the cache is seen in
columns of the output of its own, so that one lost, doubled or taken from another place shows."""

import numpy as np
import pytest
import torch

from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from test_chunk_gpu import BF16, DEV, E4M3, FP32, case, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def mark(c):
    """Values that are zero but for one column per stretch of positions: 1 or 2 there.  A stretch
    is 64 positions (half a tile, or one) or as many more as let two stretches share a column, so a
    tile that is lost takes a twelfth of its column or more at the sizes below, and a column's
    tolerance, relative to the values it weighs, is below a twentieth of it: 2 (2^-8 + n 2^-23) and
    2^-8 for the output in bf16, n = 131072 at most."""
    v, page, D = c["v_cache"], c["v_cache"].shape[1], c["v_cache"].shape[3]
    fp32 = torch.zeros(v.shape, device=DEV)
    for b, T in enumerate(c["cache_lens"].tolist()):
        size = 64 * -(-T // (64 * 2 * D))
        t = torch.arange(T, device=DEV)
        at = t // size
        pages = c["page_table"][b].long()[t // page]
        for h in range(v.shape[2]):
            fp32[pages, t % page, h, (at + 7 * h) % D] = (1.0 + at // D)
    dead = v.view(torch.uint8) == 0x7F if v.dtype == E4M3 else v.isnan()
    v.copy_(fp32.to(v.dtype))
    if v.dtype == E4M3:
        v.view(torch.uint8)[dead] = 0x7F
    else:
        v[dead] = float("nan")


@pytest.mark.parametrize("kept,new,H,Hk,D,page,dtype,cache,by_head,window", [
    ([20000], [4], 8, 1, 128, 64, BF16, BF16, True, 0),
    ([131056], [16], 8, 2, 128, 64, BF16, BF16, False, 0),
    ([30000, 7000, 12], [3, 40, 2], 6, 2, 80, 20, BF16, BF16, False, 0),
    ([9001], [130], 4, 2, 64, 16, BF16, BF16, False, 0),
    ([20003], [5], 4, 1, 192, 32, BF16, BF16, False, 0),
    ([6000, 9000], [150, 1], 2, 1, 256, 128, BF16, BF16, True, 0),
    ([15000], [3], 4, 2, 64, 128, BF16, E4M3, False, 0),
    ([40000, 100], [2, 30], 8, 1, 128, 64, BF16, E4M3, True, 0),
    ([12000], [20], 4, 1, 256, 24, BF16, E4M3, False, 0),
    ([9000, 4000], [2, 40], 2, 1, 128, 100, FP32, FP32, False, 0),
    ([33000], [6], 5, 1, 80, 24, FP32, FP32, True, 0),
    ([5000], [100], 4, 1, 96, 64, BF16, BF16, False, 700),
    ([50000], [9], 8, 1, 128, 16, BF16, BF16, False, 30000),
    ([3000] * 300, [1] * 300, 2, 1, 64, 64, BF16, BF16, False, 0),
])
def test_chunk_every_part_counts(kept, new, H, Hk, D, page, dtype, cache, by_head, window):
    c = case(kept, new, H, Hk, D, page, dtype, cache, by_head, seed=len(kept) + D)
    mark(c)
    out, lse = run(c, window=window)
    check(c, out, lse, window)


def test_chunk_a_lost_tile_would_fail():
    """The oracle with one tile's values taken away is outside the tolerance."""
    c = case([20000], [4], 8, 1, 128, 64, BF16, BF16, seed=1)
    mark(c)
    out, lse = run(c)
    page = c["k_cache"].shape[1]
    for tile in (0, 77, 155):
        less = {**c, "v_cache": c["v_cache"].clone()}
        t = torch.arange(128 * tile, 128 * tile + 128, device=DEV)
        less["v_cache"][c["page_table"][0].long()[t // page], t % page] = 0.0
        with pytest.raises(AssertionError, match="off, worst"):
            check(less, out, lse)
