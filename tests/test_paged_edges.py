"""The paged-step kernels at the ends of what their documentation allows: the
largest tables, values and scales that are not numbers, scores beyond what the
weights' type holds, long runs of idle slots, streams, and a draft loop whose
slots are not all in use.  Tolerances as in test_paged_gpu."""

import numpy as np
import pytest
import torch

from oracle import paged as P
from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from test_paged_gpu import (BF16, DEV, E4M3, EDGES, FP32, _check_decode, _check_page_step, _decode_case,
                            _page_case, i32, near, npy)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def _graph_us(call, reps=20):
    """Device time of one run among others in a captured graph, the least of ten replays."""
    call.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(reps):
            call.run()
    best = float("inf")
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / reps)
    return best


# ------------------------------------------------------------------------------ page step

def test_page_step_largest_table():
    """A table of 2^31 - 2^15 pages, all taken in one step: the list position of the last
    pages plus a grid's stride passes 2^31."""
    batch, width = 65535, 32768
    if torch.cuda.mem_get_info()[0] < 28 << 30:
        pytest.skip("needs 28 GB")
    full = torch.full((batch,), width, dtype=torch.int32, device=DEV)
    none = torch.zeros(batch, dtype=torch.int32, device=DEV)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(batch * width, dtype=torch.int32, device=DEV)
    out = B.mla_page_step(none, full, none, table, free, i32([0, batch * width]), 1, 2 ** 31 - 1, 0)
    torch.cuda.synchronize()
    assert out.missing.item() == 0 and out.free_span.tolist() == [batch * width] * 2
    assert torch.equal(table.view(-1), free)
    assert torch.equal(out.cache_lens, full) and torch.equal(out.held_pages, full)
    assert out.row_start[-1].item() == batch * width


@pytest.mark.parametrize("batch,page,tmax,newmax,short", [
    (257, 16, 90, 30, True), (1024, 8, 40, 40, False), (1025, 8, 40, 40, True),
    (1025, 16, 300, 3, False), (2047, 16, 300, 1, True), (4095, 16, 60, 3, False),
    (4096, 7, 60, 4, True), (4097, 16, 60, 2, False)])
def test_page_step_forms(batch, page, tmax, newmax, short):
    c = _page_case(batch, batch, page, tmax, newmax, short)
    total = int(c["new"].sum())
    for rows in (total, 4 * batch + 1, 4 * batch, total // 2):
        _check_page_step(c, rows)


@pytest.mark.parametrize("batch", [300, 1024, 4096, 5000, 65535])
@pytest.mark.parametrize("live", [{0: 3, -1: 3}, {0: 1, 1: 1, -2: 5, -1: 2}, {-1: 7}, {5: 2, 40: 3}])
def test_page_step_long_runs_of_idle_slots(batch, live):
    c = _page_case(batch, batch, 4, 9, 0)
    for b, n in live.items():
        c["new"][b] = n
    c["table"] = np.concatenate([c["table"], np.full((batch, 3), -1)], 1)
    top = c["num_pages"]
    c["free"], c["span"], c["num_pages"] = np.arange(top, top + 20), [1, 19], top + 20
    _check_page_step(c, sum(live.values()) + 2)


def test_page_step_idle_slots_between_live_ones_cost_little():
    # (one by one they cost the thread whose rows span them 0.06 us each)
    def us(last):
        batch = 65535
        kept = torch.full((batch,), 10, dtype=torch.int32, device=DEV)
        new = torch.zeros(batch, dtype=torch.int32, device=DEV)
        new[[0, last]] = 3
        held = torch.ones(batch, dtype=torch.int32, device=DEV)
        table = torch.arange(batch, dtype=torch.int32, device=DEV).view(batch, 1)
        return _graph_us(B.PreparedPageStep(kept, new, held, table, i32([7]), i32([0, 1]), 16,
                                            batch, 6), 5)
    apart, together = us(65534), us(1)
    assert apart < 3 * together + 20, (apart, together)


# -------------------------------------------------------------------------------- streams

def _busy():
    """Tens of milliseconds of copies on the current stream."""
    a = torch.empty(1 << 30, dtype=torch.uint8, device=DEV)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    for _ in range(100):
        b.copy_(a)


def test_outputs_made_on_one_stream_and_run_on_another():
    # what the constructor's stream still does with the buffers comes before the run
    gen = torch.Generator(DEV).manual_seed(1)
    q = torch.randn(3, 4, 192, generator=gen, device=DEV).to(BF16)
    kv = torch.randn(3, 576, generator=gen, device=DEV).to(BF16)
    cs = torch.cat([torch.ones(9, 32, device=DEV), torch.zeros(9, 32, device=DEV)], 1)
    pos, slots = i32([0, 4, 8]), torch.tensor([5, 1, 0], device=DEV)
    ckv, kr = (torch.zeros(8, w, dtype=BF16, device=DEV) for w in (512, 64))
    kc, vc = (torch.zeros(2, 4, 2, 192, dtype=BF16, device=DEV) for _ in "kv")
    other = torch.cuda.Stream()
    for _ in range(2):
        _busy()
        lat = B.PreparedAppendLatent(q, kv, cs, pos, slots, ckv, kr)
        put = B.PreparedAppendKV(q, q[:, :2], q[:, 2:], None, pos, slots, kc, vc)
        lat.run(other.cuda_stream)
        put.run(other.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(lat.q_nope, q[..., :128]) and torch.equal(lat.q_rope, q[..., 128:])
        assert torch.equal(put.q_out, q)


def test_handle_zero_is_the_default_stream():
    # a call on handle 0 allocates (and zeroes) on the stream that its kernel runs on
    assert B._stream_object(0, torch.device(DEV, 0)).cuda_stream == 0
    gen = torch.Generator(DEV).manual_seed(2)
    k = torch.randn(3, 2, 64, generator=gen, device=DEV).to(BF16)
    q = torch.randn(3, 4, 64, generator=gen, device=DEV).to(BF16)
    kc, vc = (torch.zeros(2, 4, 2, 64, dtype=BF16, device=DEV) for _ in "kv")
    pos, slots = i32([0, 4, 8]), torch.tensor([5, 1, 0], device=DEV)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        out = B.mla_append_kv(q, k, k, None, pos, slots, kc, vc, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, q)


# ----------------------------------------------------------------------- decode attention

@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("lens", [[300, 41, 1, 0], [9000]])
def test_decode_key_scale_that_is_no_number(lens, scale):
    c = _decode_case(lens, 9, 3, 64, 16, BF16, E4M3, seed=15)
    want, want_lse = B.mla_decode_attention(**c, return_lse=True)
    c["k_scale"][1] = scale
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    others = [0, 1, 2, 6, 7, 8]
    assert torch.equal(out[:, others], want[:, others])
    assert torch.equal(lse[:, others], want_lse[:, others])
    for b, t in enumerate(lens):
        if t:
            assert torch.isnan(out[b, 3:6]).all() and torch.isnan(lse[b, 3:6]).all()
        else:
            assert not out[b].any() and (lse[b] == float("-inf")).all()


@pytest.mark.parametrize("dtype,lens,H,Hk,D", [
    (BF16, [300, 41], 4, 1, 64), (FP32, [300, 41], 4, 1, 64), (BF16, [700, 20000], 32, 2, 128),
    (BF16, [300, 41], 12, 1, 256)])
def test_decode_infinite_values(dtype, lens, H, Hk, D):
    c = _decode_case(lens, H, Hk, D, 16, dtype, dtype, seed=15)
    want = B.mla_decode_attention(**c)
    inf, group = float("inf"), H // Hk
    put = {0: {3: [(5, inf)], 9: [(7, -inf)], 33: [(2, inf), (8, inf)], 20: [(8, inf), (9, -inf)]},
           1: {0: [(40, inf)], 1: [(0, -inf)], 2: [(31, inf)], 3: [(32, -inf)]}}
    for b, cols in put.items():
        for d, values in cols.items():
            for t, x in values:
                c["v_cache"][c["page_table"][b, t // 16], t % 16, 0, d] = x
    out = B.mla_decode_attention(**c)
    torch.cuda.synchronize()
    for b, cols in put.items():
        for d in range(D):
            got = out[b, :group, d]
            if d not in cols:
                assert torch.equal(got, want[b, :group, d])
            elif len({x for _, x in cols[d]}) == 2:
                assert torch.isnan(got).all()
            else:
                assert (got == cols[d][0][1]).all(), (b, d, got)
    assert torch.equal(out[:, group:], want[:, group:])


@pytest.mark.parametrize("power", [0, 12, 17, 18, 20, 22, 24, 28, 33, 60])
@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
def test_decode_scores_of_any_size(cache, power):
    # finite scores give finite results, and a key above all others its value
    dtype = FP32 if cache == FP32 else BF16
    lens, D = [300, 41, 3000], 64
    c = _decode_case(lens, 8, 2, D, 16, dtype, cache, seed=15)
    scale = 2.0 ** power
    out, lse = B.mla_decode_attention(**c, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse, scale=scale)
    # every other score is at most half of this key's
    c["q"].fill_(1.0)
    k = torch.nan_to_num(c["k_cache"].float(), nan=0.0).clamp(-2.0, 2.0)
    at = [17, 40, 2999]
    for b, t in enumerate(at):
        k[c["page_table"][b, t // 16], t % 16] = 4.0
    c["k_cache"] = k.to(cache)
    if cache == E4M3:
        c["k_scale"].fill_(0.5)
    out, lse = B.mla_decode_attention(**c, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    for b, t in enumerate(at):
        v = npy(c["v_cache"][c["page_table"][b, t // 16], t % 16])
        top = 4.0 * D * scale
        if cache == E4M3:
            v, top = v * npy(c["v_scale"])[:, None], top * 0.5
        # (the others weigh less than 3000 e^-64 of it; fp32: two roundings of the result)
        u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -22
        v = np.repeat(v, 4, 0)
        near(out[b], v, np.abs(v) * (u + 2.0 ** -20) + 1e-20, f"{power} {b}")
        assert (np.abs(npy(lse[b]) - top) <= top * 2.0 ** -21).all()


@pytest.mark.parametrize("batch,lens", [
    (1024, {0: 700, 1023: 500}), (4096, {0: 40, 4095: 3}), (65535, {0: 100, 65534: 70}),
    (2048, {0: 20064, 2047: 25000}), (4500, {31: 5, 32: 9, 64: 1, 97: 33, 4480: 2}), (300, {299: 1}), (300, {0: 1})])
@pytest.mark.parametrize("cache,H,Hk,D", [(BF16, 4, 2, 128), (FP32, 2, 1, 16)])
def test_decode_long_runs_of_idle_slots(batch, lens, cache, H, Hk, D):
    all_lens = [0] * batch
    for b, t in lens.items():
        all_lens[b] = t
    c = _decode_case(all_lens, H, Hk, D, 16, cache, cache, seed=batch)
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    rows = sorted(lens)
    live = dict(c, q=c["q"][rows], cache_lens=c["cache_lens"][rows],
                page_table=c["page_table"][rows].contiguous())
    _check_decode(live, out[rows], lse[rows])
    rest = torch.ones(batch, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert not out[rest].any() and (lse[rest] == float("-inf")).all()


def test_decode_idle_slots_between_live_ones_cost_little():
    # (one by one they cost the thread block whose share spans them 0.1 us each)
    def us(last):
        lens = [0] * 4096
        lens[0], lens[last] = 20064, 25000
        c = _decode_case(lens, 8, 2, 128, 16, BF16, BF16, seed=1)
        return _graph_us(B.PreparedDecodeAttention(**c))
    apart, together = us(4095), us(1)
    assert apart < 3 * together + 20, (apart, together)


@pytest.mark.parametrize("lens,H,Hk,D,cache", [
    (EDGES, 8, 2, 128, BF16), (EDGES, 40, 2, 64, E4M3), (EDGES, 20, 2, 64, FP32),
    ([30001, 0, 700], 36, 2, 128, BF16), ([3, 0, 1, 9] * 200, 4, 2, 64, BF16)])
def test_decode_in_place(lens, H, Hk, D, cache):
    c = _decode_case(lens, H, Hk, D, 16, FP32 if cache == FP32 else BF16, cache, seed=7)
    want = B.mla_decode_attention(**c)
    for _ in range(3):
        q = c["q"].clone()
        got = B.mla_decode_attention(**dict(c, q=q), out=q)
        torch.cuda.synchronize()
        assert got is q and torch.equal(got, want)


@pytest.mark.parametrize("lens,H,Hk,D,page,cache,window", [
    (EDGES, 8, 4, 80, 16, BF16, 0), (EDGES, 8, 8, 40, 16, BF16, 0), (EDGES, 4, 2, 96, 7, BF16, 33),
    (EDGES, 12, 4, 112, 64, BF16, 0), (EDGES, 6, 2, 80, 16, BF16, 0), (EDGES, 3, 3, 80, 16, BF16, 0),
    (EDGES, 8, 4, 64, 16, E4M3, 0), (EDGES, 16, 2, 128, 16, E4M3, 0), (EDGES, 8, 2, 64, 8, BF16, 9),
    (EDGES, 36, 4, 96, 24, E4M3, 0), (EDGES, 4, 4, 16, 16, E4M3, 20),
    ([700, 5, 2000, 0], 36, 4, 200, 16, BF16, 0), ([700, 5, 2000, 0], 36, 4, 168, 16, BF16, 0),
    ([700, 5, 2000, 0], 8, 4, 192, 16, E4M3, 0), ([700, 5, 2000, 0], 72, 4, 208, 16, E4M3, 0),
    ([9000, 1, 4000], 8, 4, 8, 16, BF16, 0), ([30, 0, 64, 7] * 90, 8, 4, 80, 16, BF16, 0),
])
def test_decode_several_heads_to_a_tile_of_a_large_pool(lens, H, Hk, D, page, cache, window):
    # heads side by side that are no whole lines, in a pool and tables beyond 256 MB
    size = 1 if cache == E4M3 else 2
    pages = -(-(256 << 20) // (2 * D * size * Hk * page)) + 1
    c = _decode_case(lens, H, Hk, D, page, BF16, cache, seed=len(lens) + D,
                     width=-(-pages // len(lens)))
    large = dict(c)
    for name in ("k_cache", "v_cache"):
        small = c[name].view(torch.uint8)
        pool = torch.full((pages, *small.shape[1:]), 0x7F, dtype=torch.uint8, device=DEV)
        if cache == BF16:
            pool.view(BF16).fill_(float("nan"))
        pool[:small.shape[0]] = small
        large[name] = pool.view(cache)
    out, lse = B.mla_decode_attention(**large, window=window, return_lse=True)
    torch.cuda.synchronize()
    B.mla_device_status()
    narrow = dict(c, page_table=c["page_table"][:, :max(-(-max(lens) // page), 1)].contiguous())
    _check_decode(narrow, out, lse, window)


@pytest.mark.parametrize("D,cache", [(80, BF16), (64, BF16), (64, E4M3)])
def test_decode_goes_by_the_pool_where_the_tables_are_wider(D, cache):
    # a table for the longest context over a small pool: the same bits as one that fits
    lens = np.random.default_rng(3).integers(1500, 2100, 16).tolist()
    c = _decode_case(lens, 16, 8, D, 16, BF16, cache, seed=1, width=16384)
    wide = B.mla_decode_attention(**c, return_lse=True)
    c["page_table"] = c["page_table"][:, :2100 // 16 + 1].contiguous()
    fit = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, *fit)
    assert torch.equal(wide[0], fit[0]) and torch.equal(wide[1], fit[1])


# ------------------------------------------------------------------- a draft loop, idle slots

@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
def test_draft_loop_with_idle_slots_in_a_graph(cache):
    """page step -> K/V append -> queries by sequence -> decode attention, captured once; at
    every step the rows that the page table names are the ones appended so far, and the
    attention is theirs."""
    H, Hk, D, page, Bn, W = 8, 2, 64, 8, 5, 4
    pages, dtype = Bn * W, FP32 if cache == FP32 else BF16
    g, gen = np.random.default_rng(51), torch.Generator(DEV).manual_seed(51)
    a = g.uniform(-3, 3, (W * page, D // 2))
    cs = torch.tensor(np.concatenate([np.cos(a), np.sin(a)], 1), dtype=FP32, device=DEV)
    ks = vs = None
    if cache == E4M3:
        ks, vs = (torch.tensor([0.02, 0.03], device=DEV) for _ in "kv")
    kc, vc = (torch.zeros(pages, page, Hk, D, dtype=FP32, device=DEV).to(cache) for _ in "kv")
    table = i32(np.full((Bn, W), -1))
    kept, new, held = (i32([0] * Bn) for _ in range(3))
    free, span = i32(g.permutation(pages)), i32([0, pages])
    qkv = torch.zeros(Bn, H + 2 * Hk, D, dtype=dtype, device=DEV)
    step = B.PreparedPageStep(kept, new, held, table, free, span, page, pages, Bn)
    put = B.PreparedAppendKV(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], cs, step.out.positions,
                             step.out.slots, kc, vc, k_scale=ks, v_scale=vs)
    q = torch.zeros(Bn, H, D, dtype=dtype, device=DEV)
    att = B.PreparedDecodeAttention(q, kc, vc, step.out.cache_lens, table, k_scale=ks, v_scale=vs,
                                    return_lse=True)

    def one():
        step.run()
        put.run()
        # the step's rows are packed: sequence b's is row_start[b]
        rows = step.out.row_start[:Bn].clamp_max(Bn - 1).long()
        torch.index_select(put.q_out, 0, rows, out=q)
        att.run()
        kept.copy_(step.out.cache_lens)
        held.copy_(step.out.held_pages)
        span.copy_(step.out.free_span)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one()
    hist = [[] for _ in range(Bn)]                     # (rotated k, v), [Hk, D] in 64 bits
    u = {BF16: 2.0 ** -8, FP32: 2.0 ** -24, E4M3: 2.0 ** -4}[cache]
    for i in range(24):
        live = [b for b in range(Bn) if (i + 2 * b) % 5 != 0 and not (b == 2 and i < 9) and b != 4]
        new.copy_(i32([int(b in live) for b in range(Bn)]))
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert step.out.missing.item() == 0
        x = npy(qkv)
        for row, b in enumerate(live):
            turn = npy(cs)[len(hist[b])]
            want_q = P.rotate(x[row, :H], turn, False)
            near(q[b], want_q, np.abs(want_q) * {BF16: 2.0 ** -8, FP32: 2.0 ** -23}[dtype]
                 + 2.0 ** -20, f"q of {b} at step {i}")
            hist[b].append((P.rotate(x[row, H:H + Hk], turn, False), x[row, H + Hk:]))
        lens = step.out.cache_lens.tolist()
        assert lens == [len(h) for h in hist]
        tab = table.cpu().numpy()
        for b in range(Bn):
            pos = np.arange(lens[b])
            for c, scale, part in ((kc, ks, 0), (vc, vs, 1)):
                got = npy(c)[tab[b, pos // page], pos % page]
                want = np.array([h[part] for h in hist[b]]).reshape(-1, Hk, D)
                sc = 1.0 if scale is None else npy(scale)[:, None]
                # (half a step of the cache's type, e4m3's smallest, and the rotation in fp32)
                tol = np.abs(want) * (u + 2.0 ** -20) + 2.0 ** -20
                if cache == E4M3:
                    tol = np.maximum(tol, 2.0 ** -10 * sc) + 2.0 ** -20
                    assert (np.abs(want) < 448 * sc).all()
                assert (np.abs(got * sc - want) <= tol).all(), (i, b, part)
        _check_decode(dict(q=q, k_cache=kc, v_cache=vc, cache_lens=step.out.cache_lens,
                           page_table=table, k_scale=ks, v_scale=vs), att.out, att.lse,
                      what=f"step {i}")
    assert lens[4] == 0 and 0 < lens[2] < lens[0]
    B.mla_device_status()
