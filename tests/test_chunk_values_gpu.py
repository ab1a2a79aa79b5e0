"""The chunk attention at values where it can go wrong: queries, key scales and scores of any size,
infinities and values that are no numbers.

Tolerances are those of the parity tests (derived there): what changes here are the inputs."""

import numpy as np
import pytest
import torch

from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from test_chunk_gpu import BF16, DEV, E4M3, FP32, case, check, hit, npy, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def scaled(c, factor):
    """The case with its queries times `factor`, subnormal ones among them."""
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.randn(c["q"].shape, generator=g, device=DEV).clamp(-3.0, 3.0)
    c["q"] = (x.double() * factor).to(BF16)
    assert c["q"].isfinite().all() and (c["q"] != 0).any()
    return c


@pytest.mark.parametrize("D,page", [(64, 16), (128, 5), (192, 16)])
@pytest.mark.parametrize("factor", [2.0 ** -133, 1e-39, 2.0 ** -128, 2.0 ** -126, 1e-30, 1e-10,
                                    1e10, 1e30])
def test_chunk_e4m3_queries_of_any_size(D, page, factor):
    c = scaled(case([140, 0, 60], [5, 40, 200], 4, 2, D, page, BF16, E4M3, seed=60, spread=0.01),
               factor)
    # with key scales that bring the scores back to a few units ...
    size = min(max(10.0 / factor, 1e-37), 1e38)
    c["k_scale"].copy_(torch.tensor([size, -0.75 * size], device=DEV))
    out, lse = run(c)
    check(c, out, lse)
    # ... and with ones that leave them small: every position weighs the same
    if factor < 1:
        c["k_scale"].fill_(0.01)
        out, lse = run(c)
        check(c, out, lse)


@pytest.mark.parametrize("factor", [2.0 ** -133, 2.0 ** -100, 2.0 ** -40, 2.0 ** -27, 1.0])
@pytest.mark.parametrize("scales", [(0.0, -0.0), (1e-37, 1e-44), (1e-30, -1e-41)])
def test_chunk_e4m3_score_scales_that_vanish(factor, scales):
    # scores too small to tell positions apart: hidden ones stay hidden, the others weigh the same
    for window in (0, 50):
        c = scaled(case([140, 0, 60], [5, 40, 200], 4, 2, 64, 16, BF16, E4M3, seed=61), factor)
        c["k_scale"].copy_(torch.tensor(scales, device=DEV))
        out, lse = run(c, window=window)
        check(c, out, lse, window)


def test_chunk_e4m3_large_queries_under_small_key_scales():
    for D in (64, 192):
        c = scaled(case([140, 0, 60], [5, 40, 200], 4, 2, D, 16, BF16, E4M3, seed=66, spread=0.01),
                   1e38)
        c["k_scale"].copy_(torch.tensor([1e-37, -8e-38], device=DEV))
        out, lse = run(c)
        check(c, out, lse)


def test_chunk_e4m3_key_scale_of_no_number_and_rows_that_see_nothing():
    # fewer cached rows than the step's last positions, a window that ends behind them
    for bad in (float("nan"), float("inf")):
        c = case([100, 100], [30, 300], 4, 2, 64, 16, BF16, E4M3, seed=62, lens=[110, 330])
        c["k_scale"][0] = bad
        out, lse = run(c, window=5)
        pos = np.concatenate([100 + np.arange(30), 100 + np.arange(300)])
        T = np.array([110] * 30 + [330] * 300)
        sees = pos + 1 - 5 < T
        assert 0 < sees[:30].sum() < 30 and 0 < sees[30:].sum() < 300
        o, z = npy(out), npy(lse)
        assert np.isnan(o[sees, :2]).all() and np.isnan(z[sees, :2]).all()
        assert not o[~sees].any() and (z[~sees] == -np.inf).all()
        c["k_scale"][0] = 1.0
        want, want_lse = run(c, window=5)
        assert torch.equal(out[:, 2:], want[:, 2:]) and torch.equal(lse[:, 2:], want_lse[:, 2:])


@pytest.mark.parametrize("dtype,cache", [(FP32, FP32), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("kept", [140, 9000])
def test_chunk_scores_all_minus_infinity_over_values_of_no_number(dtype, cache, kept):
    # zeros and -inf, whatever the values: short, and cut between thread blocks
    c = case([kept], [5], 2, 1, 64, 16, dtype, cache, seed=63)
    live = c["page_table"][0].long()
    c["q"][:, :, 0] = -float("inf")
    k = c["k_cache"].view(torch.uint8) if cache == E4M3 else c["k_cache"]
    k[live, :, :, 0] = 0x7E if cache == E4M3 else 2.0
    for t in (3, 70, kept - 1, kept):
        hit(c, "v_cache", 0, t, 0, 7, 0x7F if cache == E4M3 else float("nan"))
        if cache != E4M3:
            hit(c, "v_cache", 0, t, 0, 9, float("inf"))
    out, lse = run(c)
    assert not npy(out).any() and (npy(lse) == -np.inf).all()


@pytest.mark.parametrize("dtype,cache", [(FP32, FP32), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("t", [10, 70, 100, 120, 139])
def test_chunk_values_of_no_number_under_weights_of_zero(dtype, cache, t):
    """A seen value that is no number shows whatever its weight, in tiles that every row sees
    whole and in those at an edge; a hidden one does not."""
    c = case([100], [40], 2, 1, 64, 16, dtype, cache, seed=64)
    live = c["page_table"][0].long()
    c["q"].zero_()
    c["q"][:, :, 0] = 1.0
    if cache == E4M3:
        c["k_cache"].view(torch.uint8)[live, :, :, 0] = 0x38      # 1.0
        c["k_scale"].fill_(1.0)
    else:
        c["k_cache"][live, :, :, 0] = 0.0
    # the position's score is 400 below the others' (a weight of 2^-577)
    low = {FP32: -400.0, BF16: -400.0, E4M3: 0xFE}[cache]         # -448
    hit(c, "k_cache", 0, t, 0, 0, low)
    clean, clean_lse = run(c, scale=1.0)
    check(c, clean, clean_lse, scale=1.0)
    hit(c, "v_cache", 0, t, 0, 7, 0x7F if cache == E4M3 else float("nan"))
    if cache != E4M3:
        hit(c, "v_cache", 0, t, 0, 9, float("inf"))
    out, lse = run(c, scale=1.0)
    sees = 100 + np.arange(40) >= t
    o, z = npy(out), npy(clean)
    assert np.isnan(o[sees][:, :, 7]).all()
    z[sees, :, 7] = o[sees, :, 7]
    if cache != E4M3:
        assert not np.isfinite(o[sees][:, :, 9]).any()
        z[sees, :, 9] = o[sees, :, 9]
    assert np.array_equal(o, z, equal_nan=True)
    assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dtype,cache", [(FP32, FP32), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("kept,low", [(200, 150), (9000, 4500), (9000, 8900)])
def test_chunk_values_of_no_number_under_scores_of_minus_infinity(dtype, cache, kept, low):
    """... also where all that a thread block sees of a row has such scores."""
    c = case([kept], [5], 2, 1, 64, 16, dtype, cache, seed=67)
    live = c["page_table"][0].long()
    c["q"].zero_()
    c["q"][:, :, 0] = -2.0 ** 120                         # times the keys: beyond fp32
    if cache == E4M3:
        c["k_cache"].view(torch.uint8)[live, :, :, 0] = 0x7E
        c["k_scale"].fill_(64.0)
    else:
        c["k_cache"][live] = 0.0
        c["k_cache"][live, :, :, 0] = 2.0 ** 20
    for t in range(low, kept + 5):                        # finite from here on
        hit(c, "k_cache", 0, t, 0, 0, 0 if cache == E4M3 else 0.0)
    clean, clean_lse = run(c, scale=1.0)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
    vals = npy(c["v_cache"][live].flatten(0, 1)[:, 0]) * (
        npy(c["v_scale"])[0] if cache == E4M3 else 1.0)
    for i in range(5):
        v = vals[low:kept + 1 + i]
        assert np.abs(npy(clean)[i] - v.mean(0)).max() <= 2.0 ** -7 * np.abs(v).max()
    for t in (3, low - 1):
        hit(c, "v_cache", 0, t, 0, t % 64, 0x7F if cache == E4M3 else float("nan"))
    out, lse = run(c, scale=1.0)
    o, z = npy(out), npy(clean)
    for t in (3, low - 1):
        assert np.isnan(o[:, :, t % 64]).all()
        z[:, :, t % 64] = np.nan
    assert np.array_equal(o, z, equal_nan=True) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dtype,cache", [(FP32, FP32), (BF16, BF16), (BF16, E4M3)])
@pytest.mark.parametrize("kept", [300, 9000])
def test_chunk_equal_scores_of_any_size_weigh_the_same(dtype, cache, kept):
    # (products of the score and its scale that fp32 has to round)
    for scale in (1.1, 3.3e5, 2.0 ** 21, 1.37e9, 2.0 ** 33, 3.3e11):
        c = case([kept], [4], 2, 1, 64, 16, dtype, cache, seed=65)
        live = c["page_table"][0].long()
        c["q"].zero_()
        c["q"][:, :, 0] = 1.3
        if cache == E4M3:
            c["k_scale"].fill_(0.7)
            c["k_cache"].view(torch.uint8)[live, :, :, 0] = 0x3B  # 1.375
        else:
            c["k_cache"][live] = 0.0
            c["k_cache"][live, :, :, 0] = 1.1
        out, lse = run(c, scale=scale)
        vals = npy(c["v_cache"][live].flatten(0, 1)[:kept + 4, 0])
        if cache == E4M3:
            vals = vals * npy(c["v_scale"])[0]
        # every weight is the same number, rounded the same way (bf16 2^-8, fp16 2^-11), which
        # leaves the sums, the quotient and the output (fp32 2^-24, bf16 2^-8)
        tol = {FP32: 2.0 ** -22, BF16: 2.0 ** -7 * (1 + 2.0 ** -7),
               E4M3: (2.0 ** -8 + 2.0 ** -11) * (1 + 2.0 ** -7)}[cache]
        got = npy(out)
        for i in range(4):
            v = vals[:kept + 1 + i]
            bound = tol * np.abs(v.mean(0)) + 2 * (kept + 4) * 2.0 ** -23 * np.abs(v).mean(0)
            assert (np.abs(got[i] - v.mean(0)) <= bound).all(), (scale, i)
