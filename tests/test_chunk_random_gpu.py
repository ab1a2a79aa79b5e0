"""The chunk attention at random geometries, lengths, page sizes, windows and layouts against the
float64 oracle, with the same tolerances as at the chosen ones; repeated calls give the same bits."""

import numpy as np
import pytest
import torch

from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from test_chunk_gpu import BF16, E4M3, FP32, case, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def shape(g):
    dtype, cache, unit = [(BF16, BF16, 8), (BF16, E4M3, 16), (FP32, FP32, 4)][g.integers(3)]
    D = unit * int(g.integers(1, 256 // unit + 1))
    if g.random() < 0.3:
        D = int(g.choice([64, 80, 128, 192, 256]))
    Hk, group = int(g.integers(1, 5)), int(g.choice([1, 2, 3, 5, 8, 16]))
    page = int(g.choice([1, 2, 3, 8, 12, 16, 24, 40, 64, 128, 256]))
    batch = int(g.integers(1, 12))
    kept = [int(2 ** g.uniform(0, 11.3)) * int(g.random() > 0.2) for _ in range(batch)]
    new = [int(2 ** g.uniform(0, 8.2)) * int(g.random() > 0.25) for _ in range(batch)]
    # (what the oracle has to compute, bounded)
    while sum((k + n) * n for k, n in zip(kept, new)) * Hk * group * D > 2e8:
        kept, new = [k // 2 for k in kept], [n // 2 for n in new]
    new[0] = max(new[0], 1)
    need = max(1, max(-(-(k + n) // page) for k, n in zip(kept, new)))
    width = None if g.random() < 0.5 else need + int(g.integers(0, 200))
    window = int(g.choice([0, 0, 1, 5, 100, 129, 1000]))
    return (kept, new, Hk * group, Hk, D, page, dtype, cache, g.random() > 0.6, width,
            int(g.choice([0, 0, 4])), window)


@pytest.mark.parametrize("seed", range(60))
def test_chunk_random_shapes(seed):
    g = np.random.default_rng(7000 + seed)
    kept, new, H, Hk, D, page, dtype, cache, by_head, width, pad, window = shape(g)
    c = case(kept, new, H, Hk, D, page, dtype, cache, by_head, seed=seed, pad=pad, width=width)
    out, lse = run(c, window=window)
    again, lse_again = run(c, window=window)
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
    assert torch.equal(lse, lse_again)
    B.mla_device_status()
    check(c, out, lse, window)
