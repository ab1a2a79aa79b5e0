"""Parity of the paged-step kernels with the float64 oracle: page tables and
slots (exact), the appends, and decode attention, at the sizes and contents
where they can go wrong; then the operators together, as a serving loop runs
them.

Tolerances, derived from the roundings the kernels make:
* a value stored in type t is off by at most half a step, u(t) of its size
  (bf16 2^-8, fp32 2^-24, e4m3 2^-4, and 2^-10 below e4m3's normal range);
* a rotation in fp32 takes three roundings of terms |a| + |b|: 3 * 2^-24 of that;
* the norm sums r squares (each addition 2^-24), so its factor is off by at
  most (r / 2 + 4) * 2^-24;
* attention: a score is a sum of D products accumulated in fp32, off by at
  most ds = (D + 4) * 2^-24 * max_t scale * sum |q k| (for an e4m3 cache, q is
  also held in fp16 relative to its largest element: 2^-24 * scale * |q|max *
  sum |k|, folded in by doubling); a weight exp(s - m) is then off by 2 ds (its
  own and the maximum's) plus the exponential's 2^-21 and the rounding of the
  weights before the second product, 2^-16 (bf16: kept as two bf16 parts) or
  2^-11 (fp16 beside an e4m3 cache); sums over n positions add n * 2^-24; the
  weighted sum's error is all of that times sum p |v|, on top of u(t) |out|.
  The sum of the weights carries the same relative error, which doubles it.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import paged as P
from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib
from parity_util import compare

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
E4M3 = torch.float8_e4m3fn
BF16, FP32 = torch.bfloat16, torch.float32


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


def near(got, want, tol, what=""):
    got, want = npy(got), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.abs(got - want)[bad].max()} at {np.argwhere(bad)[0]}: "
                           f"got {got[bad][0]}, want {want[bad][0]}")


# ------------------------------------------------------------------------------ page step

def _page_case(seed, batch, page, tmax, newmax, short=False, extra=1):
    g = np.random.default_rng(seed)
    kept = g.integers(0, tmax + 1, batch)
    new = g.integers(0, newmax + 1, batch)
    width = (tmax + newmax) // page + 2
    held = np.minimum(width, -(-kept // page) + g.integers(0, 1 + extra, batch))
    grow = np.maximum(0, -(-(kept + new) // page) - held)
    free = int(grow.sum() // 2 if short else grow.sum() + 3)
    num_pages = int(held.sum()) + free + 4
    ids = g.permutation(num_pages)
    table = np.full((batch, width), -1)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    lst = np.concatenate([[0, 0], ids[at:at + free], [1]])
    return dict(kept=kept, new=new, held=held, table=table, free=lst, span=[2, 2 + free],
                page=page, num_pages=num_pages)


def _run_page_step(c, max_rows):
    table = i32(c["table"])
    args = [i32(c["kept"]), i32(c["new"]), i32(c["held"]), table, i32(c["free"]), i32(c["span"])]
    out = B.mla_page_step(*args, c["page"], c["num_pages"], max_rows)
    torch.cuda.synchronize()
    return args, table, out


def _check_page_step(c, max_rows, expect_bad=False):
    args, table, out = _run_page_step(c, max_rows)
    want = P.page_step(c["kept"], c["new"], c["held"], c["table"], c["free"], c["span"], c["page"],
                       c["num_pages"], max_rows)
    got = [table, out.cache_lens, out.held_pages, out.row_start, out.positions, out.slots,
           out.free_span]
    for name, a, b in zip(("table", "lens", "held", "row_start", "positions", "slots", "span"),
                          got, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    assert out.missing.item() == want[7]
    if expect_bad:
        assert want[8]
        with pytest.raises(B.MlaError, match="page id"):
            B.mla_device_status()
    else:
        assert not want[8]
        B.mla_device_status()
    return args, table, out


@pytest.mark.parametrize("batch,page,tmax,newmax,short", [
    (1, 1, 3, 5, False), (1, 64, 0, 1, False), (3, 16, 40, 0, False), (32, 64, 900, 8, False),
    (33, 7, 50, 90, False), (100, 24, 300, 33, True), (511, 8, 40, 9, False),
    (2047, 16, 20, 5, False), (2048, 16, 20, 5, True), (2049, 16, 20, 5, False),
    (5000, 4, 9, 3, False), (2, 32, 100, 30000, False), (1, 16, 5, 40001, False),
])
def test_page_step_matches_oracle(batch, page, tmax, newmax, short):
    for seed in range(2):
        c = _page_case(seed, batch, page, tmax, newmax, short)
        total = int(c["new"].sum())
        for rows in (total + 5, total, max(0, total - 3)):
            _check_page_step(c, rows)


def test_page_step_largest_batch():
    _check_page_step(_page_case(1, 65535, 4, 6, 2), 65000)


def test_page_step_odd_inputs():
    c = _page_case(4, 6, 8, 30, 9)
    width = c["table"].shape[1]
    c["kept"] = np.array([-5, 10, 0, 1000, 3, 2 ** 31 - 1])     # negative, past the table
    c["new"] = np.array([4, -7, 0, 12, 3, 9])
    c["held"] = np.array([0, 2, -3, width + 9, 0, 0])
    _check_page_step(c, 60)
    c["span"] = [5, 3]                                          # an empty list
    _check_page_step(c, 60)
    c["span"] = [-4, 10 ** 6]                                   # clamped to the capacity
    c["free"] = np.arange(12)[::-1].copy()
    c["num_pages"] = 10 ** 9
    _check_page_step(c, 60)


def test_page_step_huge_counts_saturate():
    c = _page_case(7, 5, 16, 20, 9)
    c["new"] = np.array([2 ** 31 - 1] * 5)
    args, table, out = _run_page_step(c, 4000)
    assert out.row_start.tolist() == [0] + [2 ** 31 - 1] * 5
    assert out.positions.tolist() == [int(c["kept"][0]) + i for i in range(4000)]
    B.mla_device_status()


def test_page_step_reports_ids_outside_the_pool():
    c = _page_case(5, 4, 8, 30, 9)
    c["kept"][:] = 4
    c["new"][:] = 3
    c["held"][:] = 1
    c["table"][1, 0] = c["num_pages"]
    c["table"][2, 0] = -1
    _check_page_step(c, 20, expect_bad=True)


def test_page_step_repeats_and_no_free_list():
    c = _page_case(9, 8, 16, 50, 20)
    args, table, out = _run_page_step(c, 200)
    first = [t.clone() for t in (table, *out)]
    B.mla_page_step(*args, c["page"], c["num_pages"], 200, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (table, *out)))
    c["free"], c["span"] = np.zeros(0), [0, 0]
    _check_page_step(c, 200)
    B.mla_page_step(args[0], args[1], args[2], table, args[4], args[5], c["page"], c["num_pages"],
                    0)                                          # no rows wanted
    B.mla_device_status()


# -------------------------------------------------------------------------------- appends

def _table(rows, rope, g):
    a = g.uniform(-3, 3, (rows, rope // 2))
    return torch.tensor(np.concatenate([np.cos(a), np.sin(a)], 1), dtype=FP32, device=DEV)


def _randn(gen, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _slots(g, rows, cache_rows, table_rows):
    """Distinct slots; a few skipped rows, and rows outside the cache or the table."""
    slots = g.permutation(cache_rows)[:rows].astype(np.int64)
    pos = g.integers(0, table_rows, rows)
    if rows > 6:
        slots[[1, 4]] = [-1, cache_rows]
        pos[[2, 5, 6]] = [-1, table_rows, -2 ** 31]
    return pos, slots


def _rot_tol(x, out, dtype, cs):
    """u(t) |out| plus the fp32 rotation's error, 3 * 2^-24 of |a| + |b|."""
    return U[dtype] * np.abs(out) * (1 + 2.0 ** -8) + 2.0 ** -22 * np.abs(x).max(
        -1, keepdims=True) + 1e-30


@pytest.mark.parametrize("rows,H,r,n,rope,dtype,inter,norm,pad", [
    (1, 1, 64, 16, 16, BF16, True, True, 0), (5, 4, 512, 128, 64, BF16, True, True, 0),
    (7, 4, 512, 128, 64, FP32, False, True, 8), (33, 128, 512, 128, 64, BF16, False, True, 16),
    (64, 32, 512, 192, 64, BF16, True, False, 0), (9, 3, 1024, 512, 128, FP32, True, True, 4),
    (9, 5, 8, 8, 32, BF16, False, True, 0), (700, 16, 256, 64, 64, BF16, True, True, 0),
    (3001, 7, 512, 40, 48, BF16, False, True, 0),
])
def test_append_latent_matches_oracle(rows, H, r, n, rope, dtype, inter, norm, pad):
    g, gen = np.random.default_rng(rows), torch.Generator(DEV).manual_seed(rows)
    cs = _table(50, rope, g)
    pages, page = rows // 16 + 3, 16
    pos, slots = _slots(g, rows, pages * page, 50)
    q = _randn(gen, rows, H, n + rope, dtype=dtype)
    # rows of a wider projection: a stride beyond the row
    kv = _randn(gen, rows, r + rope + pad, dtype=dtype, scale=2.0)[:, :r + rope]
    w = _randn(gen, r, dtype=dtype) if norm else None
    packed = _randn(gen, pages, page, r + rope, dtype=dtype)     # one cache for both parts
    c_kv, k_rope = packed[..., :r], packed[..., r:]
    old = packed.clone()
    qn0, qr0 = _randn(gen, rows, H, n, dtype=dtype), _randn(gen, rows, H, rope, dtype=dtype)
    qn, qr = qn0.clone(), qr0.clone()
    got = B.mla_append_latent(q, kv, cs, i32(pos), torch.tensor(slots, device=DEV), c_kv, k_rope,
                              norm_weight=w, eps=1e-5, interleaved=inter, q_nope=qn, q_rope=qr)
    torch.cuda.synchronize()
    assert got[0] is qn and got[1] is qr
    want = npy(old).reshape(-1, r + rope)
    tol = np.zeros_like(want)
    for i in range(rows):
        if not 0 <= pos[i] < 50:
            assert torch.equal(qn[i], qn0[i]) and torch.equal(qr[i], qr0[i])
            continue
        t = npy(cs)[pos[i]]
        assert torch.equal(qn[i], q[i, :, :n])                   # copied bit for bit
        x = npy(q[i, :, n:])
        y = P.rotate(x, t, inter)
        near(qr[i], y, _rot_tol(x, y, dtype, t), "q_rope")
        if not 0 <= slots[i] < pages * page:
            continue
        x = npy(kv[i, r:])
        want[slots[i], r:] = P.rotate(x, t, inter)
        tol[slots[i], r:] = _rot_tol(x, want[slots[i], r:], dtype, t)
        x = npy(kv[i, :r])
        want[slots[i], :r] = P.rms_norm(x, npy(w), 1e-5) if norm else x
        if norm:
            tol[slots[i], :r] = np.abs(want[slots[i], :r]) * (U[dtype] + (r / 2 + 8) * 2.0 ** -24)
    near(packed.view(-1, r + rope), want, tol, "cache")


def test_append_latent_without_queries():
    gen, g = torch.Generator(DEV).manual_seed(1), np.random.default_rng(1)
    cs, kv = _table(9, 64, g), _randn(gen, 4, 576, dtype=BF16)
    pos, slots = i32([0, 3, 8, 1]), torch.tensor([5, 1, 0, 7], device=DEV)
    a = [torch.zeros(8, w, dtype=BF16, device=DEV) for w in (512, 64)]
    b = [torch.zeros(8, w, dtype=BF16, device=DEV) for w in (512, 64)]
    assert B.mla_append_latent(None, kv, cs, pos, slots, *a) == (None, None)
    B.mla_append_latent(_randn(gen, 4, 6, 192, dtype=BF16), kv, cs, pos, slots, *b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and a[0][5].any()


@pytest.mark.parametrize("rows,H,Hk,D,rope,dtype,cache,inter,page,by_head", [
    (1, 1, 1, 64, 64, BF16, BF16, False, 1, False), (5, 8, 2, 128, 128, BF16, BF16, False, 16, False),
    (9, 8, 2, 128, 128, BF16, E4M3, False, 16, True), (9, 6, 3, 80, 48, BF16, BF16, True, 24, False),
    (17, 8, 8, 256, 128, FP32, FP32, True, 8, True), (40, 5, 1, 8, 0, BF16, BF16, False, 64, False),
    (40, 5, 1, 4, 0, FP32, FP32, False, 7, False), (33, 12, 4, 112, 112, BF16, E4M3, True, 32, False),
    (2000, 32, 8, 128, 64, BF16, BF16, False, 64, False), (501, 7, 7, 96, 96, FP32, FP32, False, 16, True),
    (300, 64, 8, 192, 192, BF16, E4M3, False, 128, False),
])
def test_append_kv_matches_oracle(rows, H, Hk, D, rope, dtype, cache, inter, page, by_head):
    g, gen = np.random.default_rng(rows), torch.Generator(DEV).manual_seed(rows)
    cs = _table(40, rope, g) if rope else None
    pages = rows // page + 9
    pos, slots = _slots(g, rows, pages * page, 40)
    if not rope:
        pos = np.where(pos >= 0, pos, -1)
    qkv = _randn(gen, rows, H + 2 * Hk, D, dtype=dtype, scale=3.0)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    ks = vs = None
    if cache == E4M3:
        ks, vs = (torch.rand(Hk, generator=gen, device=DEV) * 0.02 + 0.005 for _ in range(2))
        if rows > 6:
            v[3, 0, :4] = torch.tensor([1e4, -1e4, 1e-5, float("nan")])   # saturates, vanishes, NaN
    shape = (pages, Hk, page, D) if by_head else (pages, page, Hk, D)
    kc, vc = (_randn(gen, *shape, dtype=FP32, scale=30.0).to(cache) for _ in range(2))
    if by_head:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    want_k, want_v = npy(kc), npy(vc)
    q0 = _randn(gen, rows, H, D, dtype=dtype)
    out = q0.clone()
    got = B.mla_append_kv(q, k, v, cs, i32(pos), torch.tensor(slots, device=DEV), kc, vc,
                          interleaved=inter, k_scale=ks, v_scale=vs, q_out=out)
    torch.cuda.synchronize()
    assert got is out
    tol_k, tol_v = np.zeros_like(want_k), np.zeros_like(want_v)

    def turned(x, i):
        y = x.copy()
        if rope:
            y[:, :rope] = P.rotate(x[:, :rope], npy(cs)[pos[i]], inter)
        return y

    for i in range(rows):
        if pos[i] < 0 or (rope and pos[i] >= 40):
            assert torch.equal(out[i], q0[i])
            continue
        x = npy(q[i])
        y = turned(x, i)
        near(out[i], y, _rot_tol(x, y, dtype, None), "q")
        assert torch.equal(out[i][:, rope:], q[i][:, rope:])
        if not 0 <= slots[i] < pages * page:
            continue
        at = (slots[i] // page, slots[i] % page)
        x = npy(k[i])
        y = turned(x, i)
        z = npy(v[i])
        if cache == E4M3:
            # (k: within half a step, or the fp32 error next to a border; v: the very value)
            sk = npy(ks)[:, None]
            want_k[at] = np.clip(y / sk, -448, 448)
            tol_k[at] = np.maximum(np.abs(want_k[at]) * (U[E4M3] + 2.0 ** -20), 2.0 ** -10) + \
                2.0 ** -22 * np.abs(x).max() / sk
            z32 = np.divide(z.astype(np.float32), vs.cpu().numpy()[:, None])
            want_v[at] = P.round_e4m3(z32)
        else:
            want_k[at], want_v[at] = y, z
            tol_k[at] = _rot_tol(x, y, dtype, None)
    near(kc, want_k, tol_k, "k")
    nan = np.isnan(want_v)
    assert np.array_equal(np.isnan(npy(vc)), nan)
    assert np.array_equal(npy(vc)[~nan], want_v[~nan])


def test_append_kv_in_place_and_without_queries():
    g, gen = np.random.default_rng(2), torch.Generator(DEV).manual_seed(2)
    cs = _table(9, 64, g)
    q, k, v = (_randn(gen, 3, h, 64, dtype=BF16) for h in (4, 2, 2))
    pos, slots = i32([1, 8, 0]), torch.tensor([3, 0, 5], device=DEV)
    caches = [torch.zeros(2, 4, 2, 64, dtype=BF16, device=DEV) for _ in range(4)]
    want = B.mla_append_kv(q, k, v, cs, pos, slots, *caches[:2])
    assert B.mla_append_kv(None, k, v, cs, pos, slots, *caches[2:]) is None
    got = B.mla_append_kv(q, k, v, cs, pos, slots, *caches[:2], q_out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q, want)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    with pytest.raises(B.MlaError, match="overlaps"):
        buf = torch.zeros(5, 4, 64, dtype=BF16, device=DEV)
        B.mla_append_kv(buf[:3], k, v, cs, pos, slots, *caches[:2], q_out=buf[2:])


# ----------------------------------------------------------------------- decode attention

def _decode_case(lens, H, Hk, D, page, dtype, cache, by_head=False, seed=0, spread=1.0,
                 poison=True, extra_pages=2, width=None):
    """Caches whose unread rows hold NaN, shuffled pages, -1 behind each sequence's table."""
    g, gen = np.random.default_rng(seed), torch.Generator(DEV).manual_seed(seed)
    used = [max(0, -(-t // page)) for t in lens]
    W = width or max(max(used), 1)
    used = [min(u, W) for u in used]
    pages = sum(used) + extra_pages
    ids = g.permutation(pages)
    table = np.full((len(lens), W), -1)
    shape = (pages, Hk, page, D) if by_head else (pages, page, Hk, D)
    most = 448.0 if cache == E4M3 else 1e30      # (torch's own cast turns larger values into NaN)
    kc, vc = (_randn(gen, *shape, dtype=FP32, scale=s).clamp(-most, most).to(cache)
              for s in ((60.0 if cache == E4M3 else 1.0) * spread, 60.0 if cache == E4M3 else 1.0))
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
    q = _randn(gen, len(lens), H, D, dtype=dtype)
    return dict(q=q, k_cache=kc, v_cache=vc, cache_lens=i32(lens), page_table=i32(table),
                k_scale=ks, v_scale=vs)


def _check_decode(c, out, lse, window=0, scale=None, what=""):
    q, cache = c["q"], c["k_cache"].dtype
    D = q.shape[-1]
    sc = lambda x: None if x is None else npy(x)  # noqa: E731
    want, want_lse, vabs, big = P.decode_attention(
        npy(q), npy(c["k_cache"]), npy(c["v_cache"]), c["cache_lens"].cpu().numpy(),
        c["page_table"].cpu().numpy(), window, scale, sc(c["k_scale"]), sc(c["v_scale"]))
    n = int(max(1, c["cache_lens"].max().item()))
    ds = (D + 4) * 2.0 ** -24 * big * (2 if cache == E4M3 else 1)
    weights = {FP32: 0.0, BF16: 2.0 ** -16, E4M3: 2.0 ** -11}[cache]
    rel = 2 * (2 * ds + 2.0 ** -21 + weights + n * 2.0 ** -24)[..., None]
    near(out, want, U[q.dtype] * np.abs(want) * (1 + 2.0 ** -7) + rel * vabs + 1e-30, what + " out")
    fin = np.isfinite(want_lse)
    assert np.array_equal(np.isfinite(npy(lse)), fin), what
    assert (npy(lse)[~fin] == -np.inf).all()
    tol = (2 * ds + 2.0 ** -20 + n * 2.0 ** -24) + 2.0 ** -22 * np.abs(np.where(fin, want_lse, 0))
    assert (np.abs(npy(lse) - np.where(fin, want_lse, 0))[fin] <= tol[fin]).all(), what + " lse"


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]

DECODE = [
    # lens, H, Hk, D, page, dtype, cache, by_head, window
    (EDGES, 8, 2, 128, 64, BF16, BF16, False, 0),
    (EDGES, 8, 2, 128, 16, BF16, E4M3, True, 0),
    (EDGES, 6, 2, 64, 8, FP32, FP32, False, 0),
    (EDGES, 8, 8, 64, 24, BF16, BF16, True, 50),
    (EDGES, 4, 4, 80, 7, BF16, BF16, False, 64),
    (EDGES, 10, 2, 96, 1, BF16, E4M3, False, 17),
    (EDGES, 5, 1, 40, 5, FP32, FP32, True, 33),
    ([1], 1, 1, 64, 16, BF16, BF16, False, 0),
    ([61], 16, 8, 64, 16, BF16, BF16, False, 0),
    ([700, -3, 0, 5000, 1], 32, 4, 128, 64, BF16, BF16, False, 0),
    ([700, 5, 2000], 12, 1, 112, 32, BF16, BF16, False, 0),
    ([700, 5, 2000], 48, 2, 128, 32, BF16, E4M3, False, 1000),
    ([700, 5, 2000], 33, 3, 192, 16, BF16, BF16, True, 0),
    ([700, 5, 2000], 18, 1, 256, 64, BF16, BF16, False, 0),
    ([700, 5, 2000], 16, 2, 256, 64, BF16, E4M3, False, 0),
    ([700, 5, 2000], 17, 1, 192, 64, BF16, E4M3, False, 0),
    ([900, 3], 40, 2, 256, 16, FP32, FP32, False, 0),
    ([900, 3], 9, 1, 192, 16, FP32, FP32, True, 100),
    ([900, 3], 3, 3, 4, 16, FP32, FP32, False, 0),
    ([900, 3], 3, 3, 8, 16, BF16, BF16, False, 0),
    ([900, 3], 7, 1, 16, 16, BF16, E4M3, False, 0),
    ([40000], 8, 1, 128, 64, BF16, BF16, True, 0),
    ([30001], 4, 1, 64, 128, BF16, E4M3, False, 0),
    ([9000, 10000], 2, 1, 128, 100, FP32, FP32, False, 0),
    ([3, 0, 1, 9] * 80, 4, 2, 64, 16, BF16, BF16, False, 0),
    ([0, 0, 0], 8, 2, 128, 16, BF16, BF16, False, 0),
]


@pytest.mark.parametrize("lens,H,Hk,D,page,dtype,cache,by_head,window", DECODE)
def test_decode_matches_oracle(lens, H, Hk, D, page, dtype, cache, by_head, window):
    c = _decode_case(lens, H, Hk, D, page, dtype, cache, by_head, seed=len(lens) + D)
    out, lse = B.mla_decode_attention(**c, window=window, return_lse=True)
    torch.cuda.synchronize()
    B.mla_device_status()
    _check_decode(c, out, lse, window)
    again, lse2 = B.mla_decode_attention(**c, window=window, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)    # the same bits each time


@pytest.mark.parametrize("lens,H,Hk,D,page,cache,window", [
    (EDGES, 8, 4, 80, 16, BF16, 0), (EDGES, 8, 8, 40, 16, BF16, 0), (EDGES, 4, 2, 96, 7, BF16, 33),
    (EDGES, 12, 4, 112, 64, BF16, 0), (EDGES, 6, 2, 80, 16, BF16, 0), (EDGES, 3, 3, 80, 16, BF16, 0),
    (EDGES, 8, 4, 64, 16, E4M3, 0), (EDGES, 16, 2, 128, 16, E4M3, 0), (EDGES, 8, 2, 64, 8, BF16, 9),
    (EDGES, 36, 4, 96, 24, E4M3, 0), (EDGES, 4, 4, 16, 16, E4M3, 20),
    ([700, 5, 2000, 0], 36, 4, 200, 16, BF16, 0), ([700, 5, 2000, 0], 36, 4, 168, 16, BF16, 0),
    ([700, 5, 2000, 0], 8, 4, 192, 16, E4M3, 0), ([700, 5, 2000, 0], 72, 4, 208, 16, E4M3, 0),
    ([9000, 1, 4000], 8, 4, 8, 16, BF16, 0), ([30, 0, 64, 7] * 90, 8, 4, 80, 16, BF16, 0),
])
def test_decode_several_heads_to_a_tile(lens, H, Hk, D, page, cache, window):
    # heads side by side that are no whole lines, and a table of a cache beyond 256 MB
    size = 1 if cache == E4M3 else 2
    width = -(-(256 << 20) // (2 * D * size * Hk * len(lens) * page)) + 1
    c = _decode_case(lens, H, Hk, D, page, BF16, cache, seed=len(lens) + D, width=width)
    out, lse = B.mla_decode_attention(**c, window=window, return_lse=True)
    torch.cuda.synchronize()
    B.mla_device_status()
    narrow = dict(c, page_table=c["page_table"][:, :max(-(-max(lens) // page), 1)].contiguous())
    _check_decode(narrow, out, lse, window)
    one, one_lse = B.mla_decode_attention(**narrow, window=window, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(narrow, one, one_lse, window)


@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
def test_decode_sharp_scores_and_scale(cache):
    dtype = FP32 if cache == FP32 else BF16
    c = _decode_case([500, 77], 8, 2, 64, 16, dtype, cache, seed=3, spread=12.0)
    out, lse = B.mla_decode_attention(**c, scale=0.3, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse, scale=0.3)


@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
def test_decode_one_heavy_position_among_many_light_ones(cache):
    # one key far above 20000 equal ones whose summed weight still counts
    dtype = FP32 if cache == FP32 else BF16
    c = _decode_case([20001], 2, 1, 64, 16, dtype, cache, seed=4)
    c["q"].zero_()
    c["q"][..., 0] = 8.0
    kc = c["k_cache"].float()
    kc[torch.isnan(kc)] = 0.0
    kc[..., 1:] = 0.0
    kc[..., 0] = 0.0
    pos = 777
    pid = c["page_table"][0, pos // 16].item()
    big = 9.0 if cache != E4M3 else 256.0                        # exact in the type
    kc[pid, pos % 16, 0, 0] = big
    c["k_cache"] = kc.to(cache)
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse)


@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
def test_decode_reads_nothing_before_the_window(cache):
    dtype = FP32 if cache == FP32 else BF16
    c = _decode_case([300, 41, 16], 6, 2, 64, 16, dtype, cache, seed=14)
    window = 37
    table = c["page_table"]
    for b, t in enumerate([300, 41, 16]):
        lo = max(0, t - window)
        for pos in range(lo):                       # rows before it hold NaN
            pid = table[b, pos // 16].item()
            for x in (c["k_cache"], c["v_cache"]):
                if cache == E4M3:
                    x.view(torch.uint8)[pid, pos % 16] = 0x7F
                else:
                    x[pid, pos % 16] = float("nan")
        table[b, :lo // 16] = -1                    # and whole pages have no id
    out, lse = B.mla_decode_attention(**c, window=window, return_lse=True)
    torch.cuda.synchronize()
    B.mla_device_status()
    _check_decode(c, out, lse, window)


def test_decode_odd_scales():
    # a negative key scale, a zero one, and none at all
    c = _decode_case([300, 41], 9, 3, 64, 16, BF16, E4M3, seed=15)
    c["k_scale"].copy_(torch.tensor([-0.02, 0.0, 0.01], device=DEV))
    c["v_scale"].copy_(torch.tensor([0.01, -0.5, 0.0], device=DEV))
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse)
    with pytest.raises(ValueError, match="positive"):
        B.mla_decode_attention(**c, scale=-1.0)
    c["k_scale"] = c["v_scale"] = None
    out, lse = B.mla_decode_attention(**c, scale=1e-4, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse, scale=1e-4)


def test_decode_many_sequences():
    # more sequences than threads of a CTA, and than CTAs
    g = np.random.default_rng(5)
    lens = g.integers(0, 40, 3000)
    lens[[7, 2999]] = [1500, 700]
    c = _decode_case(lens.tolist(), 4, 2, 64, 16, BF16, BF16, seed=16)
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse)


def test_decode_graphs_sharing_a_workspace():
    a = _decode_case([3000, 200], 8, 2, 128, 16, BF16, BF16, seed=41)
    b = _decode_case([50, 1000, 700], 4, 1, 64, 16, FP32, FP32, seed=42)
    need = [B.mla_decode_workspace_bytes(8, 2, 128, 2, 16, a["page_table"].shape[1]),
            B.mla_decode_workspace_bytes(4, 1, 64, 3, 16, b["page_table"].shape[1], FP32)]
    assert min(need) > 0
    ws = torch.full((max(need),), 0x7F, dtype=torch.uint8, device=DEV)   # (any contents will do)
    calls = [B.PreparedDecodeAttention(**x, return_lse=True, workspace=ws) for x in (a, b)]
    graphs = []
    for call in calls:
        call.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call.run()
    for i in (0, 1, 1, 0, 1, 0):                                        # one after the other
        calls[i].out.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        _check_decode((a, b)[i], calls[i].out, calls[i].lse)


def test_calls_on_the_default_stream_handle_and_a_second_stream():
    c = _decode_case([700, 33], 8, 2, 64, 16, BF16, BF16, seed=70)
    want = B.mla_decode_attention(**c, return_lse=True)
    got = B.mla_decode_attention(**c, return_lse=True, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    call = B.PreparedDecodeAttention(**c, return_lse=True)
    other = torch.cuda.Stream()
    for stream in (None, other.cuda_stream, 0, other.cuda_stream):
        call.out.zero_()
        torch.cuda.synchronize()
        call.run(stream)
        torch.cuda.synchronize()
        assert torch.equal(call.out, want[0])
    with pytest.raises(B.MlaError, match="aligned"):
        lens = i32([0, 700, 33])[1:]
        B.mla_decode_attention(**{**c, "cache_lens": lens})


def test_direct_calls_inside_a_capture():
    c = _page_case(71, 6, 8, 30, 9)
    args = [i32(c["kept"]), i32(c["new"]), i32(c["held"]), i32(c["table"]), i32(c["free"]),
            i32(c["span"])]
    rows = 64
    g, gen = np.random.default_rng(3), torch.Generator(DEV).manual_seed(3)
    cs = _table(64, 64, g)
    kv, q = _randn(gen, rows, 576, dtype=BF16), _randn(gen, rows, 4, 192, dtype=BF16)
    ckv, kr = (torch.zeros(c["num_pages"], 8, w, dtype=BF16, device=DEV) for w in (512, 64))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        st = B.mla_page_step(*args, c["page"], c["num_pages"], rows)
        qn, qr = B.mla_append_latent(q, kv, cs, st.positions, st.slots, ckv, kr)
    for _ in range(2):
        ckv.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = P.page_step(c["kept"], c["new"], c["held"], c["table"], c["free"], c["span"],
                           c["page"], c["num_pages"], rows)
        assert np.array_equal(st.slots.cpu().numpy(), want[5])
        live = [(i, s) for i, s in enumerate(want[5]) if s >= 0]
        flat = ckv.view(-1, 512)
        assert len(live) and all(torch.equal(flat[s], kv[i, :512]) for i, s in live)
        assert flat.abs().sum(1).count_nonzero().item() == len(live)
        n = int(want[3][-1])
        assert torch.equal(qn[:n], q[:n, :, :128]) and not qn[n:].any()


def test_steps_on_several_streams():
    cases = [_page_case(60 + i, 40, 8, 60, 9) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for c, s in zip(cases, streams):
        args = [i32(c["kept"]), i32(c["new"]), i32(c["held"]), i32(c["table"]), i32(c["free"]),
                i32(c["span"])]
        torch.cuda.synchronize()
        outs.append((args, B.mla_page_step(*args, c["page"], c["num_pages"], 300,
                                           stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for c, (args, out) in zip(cases, outs):
        want = P.page_step(c["kept"], c["new"], c["held"], c["table"], c["free"], c["span"],
                           c["page"], c["num_pages"], 300)
        assert np.array_equal(args[3].cpu().numpy(), want[0])
        assert np.array_equal(out.slots.cpu().numpy(), want[5])


def test_decode_strided_inputs():
    c = _decode_case([100, 37], 8, 2, 128, 16, BF16, BF16, seed=8)
    pages = c["k_cache"].shape[0]
    qkv = torch.randn(2, 12, 128, device=DEV).to(BF16)
    both = torch.full((pages, 2, 16, 3, 136), float("nan"), dtype=BF16, device=DEV)
    both[:, 0, :, :2, :128] = c["k_cache"]
    both[:, 1, :, :2, :128] = c["v_cache"]
    want = B.mla_decode_attention(**{**c, "q": qkv[:, :8].contiguous()}, return_lse=True)
    got = B.mla_decode_attention(**{**c, "q": qkv[:, :8], "k_cache": both[:, 0, :, :2, :128],
                                    "v_cache": both[:, 1, :, :2, :128]}, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cache", [BF16, E4M3, FP32])
def test_decode_table_capacity_and_bad_pages(cache):
    dtype = FP32 if cache == FP32 else BF16
    c = _decode_case([200, 64, 90], 4, 2, 64, 16, dtype, cache, seed=6, width=5)
    out, lse = B.mla_decode_attention(**c, return_lse=True)     # 200 and 90 count as 80
    torch.cuda.synchronize()
    B.mla_device_status()
    _check_decode(c, out, lse)
    c["page_table"][1, 2] = c["k_cache"].shape[0]               # reads as zeros, reported
    c["page_table"][2, 0] = -7
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    _check_decode(c, out, lse)
    with pytest.raises(B.MlaError, match="page id"):
        B.mla_device_status()


@pytest.mark.parametrize("cache", [BF16, FP32])
def test_decode_infinite_and_nan_inputs(cache):
    c = _decode_case([40, 33, 20], 2, 1, 64, 8, cache, cache, seed=12)
    at = lambda b, t: (c["page_table"][b, t // 8].item(), t % 8, 0)  # noqa: E731
    c["q"][0, :, 0] = 1.0
    c["k_cache"][at(0, 5)] = 0.0
    c["k_cache"][at(0, 5) + (0,)] = float("-inf")               # a score of -inf: weight 0
    c["v_cache"][at(1, 9) + (3,)] = float("nan")                # a live NaN stays in its column
    c["q"][2, :, 0] = 1.0
    for t in range(20):                                         # every score -inf
        c["k_cache"][at(2, t)] = 0.0
        c["k_cache"][at(2, t) + (0,)] = float("-inf")
    out, lse = B.mla_decode_attention(**c, return_lse=True)
    torch.cuda.synchronize()
    o = npy(out)
    assert np.isfinite(o[0]).all()
    assert np.isnan(o[1, :, 3]).all() and np.isfinite(np.delete(o[1], 3, 1)).all()
    assert not o[2].any() and (npy(lse)[2] == -np.inf).all()


def test_decode_offsets_beyond_32_bits():
    # 8-bit caches of 4.4e9 elements each; the sequences use pages at both ends
    pages, page, Hk, D = 540000, 64, 1, 128
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    kc, vc = (torch.empty(pages, page, Hk, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    lens = [130, 200]
    table = i32([[539999, 0, 539990, 1], [524288, 524287, 530001, 2]])
    small = _decode_case(lens, 4, Hk, D, page, BF16, E4M3, seed=1)
    for c, s in ((kc, small["k_cache"]), (vc, small["v_cache"])):
        for b in range(2):
            n = -(-lens[b] // page)
            c[table[b, :n].long()] = s[small["page_table"][b, :n].long()].view(torch.uint8)
    want = B.mla_decode_attention(**small, return_lse=True)
    got = B.mla_decode_attention(small["q"], kc.view(E4M3), vc.view(E4M3), small["cache_lens"],
                                 table, k_scale=small["k_scale"], v_scale=small["v_scale"],
                                 return_lse=True)
    torch.cuda.synchronize()
    B.mla_device_status()
    near(got[0], npy(want[0]), 2.0 ** -7 * np.abs(npy(want[0])) + 1e-3)
    assert torch.allclose(got[1], want[1], atol=1e-4)
    # and an append there
    k = torch.randn(2, Hk, D, device=DEV).to(BF16)
    slots = torch.tensor([539999 * 64 + 63, 530001 * 64], device=DEV)
    B.mla_append_kv(None, k, k, None, i32([1, 2]), slots, kc.view(E4M3), vc.view(E4M3))
    torch.cuda.synchronize()
    assert torch.equal(kc.view(E4M3)[539999, 63].float(), k[0].to(E4M3).float())
    assert torch.equal(vc.view(E4M3)[530001, 0].float(), k[1].to(E4M3).float())


def test_decode_graph_follows_lengths_and_tables():
    c = _decode_case([500, 300, 0, 20], 8, 2, 128, 16, BF16, BF16, seed=21, poison=False)
    call = B.PreparedDecodeAttention(**c, return_lse=True)
    call.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run()
    for lens in ([500, 300, 0, 20], [1, 299, 0, 3], [0, 0, 0, 0], [480, 17, 0, 16]):
        c["cache_lens"].copy_(i32(lens))
        c["page_table"].copy_(torch.where(c["page_table"] >= 0, c["page_table"].flip(1).clamp_min(0),
                                          c["page_table"]))
        graph.replay()
        torch.cuda.synchronize()
        _check_decode(c, call.out, call.lse, what=str(lens))
    B.mla_device_status()


def test_decode_concurrent_streams():
    cs = [_decode_case([3000, 77 + i], 8, 2, 128, 16, BF16, BF16, seed=30 + i) for i in range(3)]
    want = [B.mla_decode_attention(**c, return_lse=True) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [B.mla_decode_attention(**c, return_lse=True, stream=s.cuda_stream)
               for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(got, want):
            assert torch.equal(a, b) and torch.equal(la, lb)


# --------------------------------------------------------------------- a serving loop of both

def _dense_latent(hist, n):
    return np.stack([x for x in hist[:n]])


def test_verify_steps_over_a_growing_paged_cache():
    """page step -> latent append -> verify attention, with rejections between the steps."""
    H, r, n, v, rope, page, L = 4, 512, 128, 128, 64, 64, 4
    g, gen = np.random.default_rng(40), torch.Generator(DEV).manual_seed(40)
    Bn, W, pages = 3, 6, 20
    cs = _table(W * page, rope, g)
    w = _randn(gen, r, dtype=BF16)
    W_UK = _randn(gen, H, n, r, dtype=BF16, scale=512 ** -0.5)
    W_UV = _randn(gen, H, r, v, dtype=BF16, scale=512 ** -0.5)
    c_kv = torch.full((pages, page, r), float("nan"), dtype=BF16, device=DEV)
    k_rope = torch.full((pages, page, rope), float("nan"), dtype=BF16, device=DEV)
    table = i32(np.full((Bn, W), -1))
    free = i32(g.permutation(pages))
    kept, held, span = i32([0] * Bn), i32([0] * Bn), i32([0, pages])
    hist = [[] for _ in range(Bn)]                               # (c, k) rows per sequence, rounded

    def rows_of(new, max_rows):
        """One page step and append; returns the step, and the row tensors."""
        st = B.mla_page_step(kept, i32(new), held, table, free, span, page, pages, max_rows)
        q = _randn(gen, max_rows, H, n + rope, dtype=BF16)
        kv = _randn(gen, max_rows, r + rope, dtype=BF16)
        qn, qr = B.mla_append_latent(q, kv, cs, st.positions, st.slots, c_kv, k_rope,
                                     norm_weight=w)
        torch.cuda.synchronize()
        assert st.missing.item() == 0
        pos = st.positions.cpu().numpy()
        starts = st.row_start.tolist()
        for b in range(Bn):
            for i in range(starts[b], starts[b + 1]):
                slot = st.slots[i].item()
                got = (c_kv.view(-1, r)[slot], k_rope.view(-1, rope)[slot])
                near(got[0], P.rms_norm(npy(kv[i, :r]), npy(w), 1e-6),
                     np.abs(P.rms_norm(npy(kv[i, :r]), npy(w), 1e-6)) * (2.0 ** -8 + 2.0 ** -14))
                hist[b].append((npy(got[0]), npy(got[1])))
                assert len(hist[b]) == pos[i] + 1
        return st, qn, qr

    st, _, _ = rows_of([130, 64, 1], 200)                        # prompts, with padding rows
    for step in range(3):
        kept, held, span = st.cache_lens, st.held_pages, st.free_span
        if step:                                                 # reject some of the last rows
            drop = [step, 0, 3]
            kept = kept - i32(drop)
            hist = [h[:len(h) - d] for h, d in zip(hist, drop)]
        st, qn, qr = rows_of([L] * Bn, Bn * L)
        lens = st.cache_lens.tolist()
        assert lens == [len(h) for h in hist]
        qn, qr = qn.view(Bn, L, H, n), qr.view(Bn, L, H, rope)
        out, _ = B.mla_verify_attention(qn, qr, c_kv, k_rope, W_UK, W_UV, lens, page_table=table,
                                        cache_lens_dev=st.cache_lens, mode="absorbed")
        torch.cuda.synchronize()
        B.mla_device_status()
        T = max(lens)
        dense = [np.zeros((Bn, T, x)) for x in (r, rope)]
        for b in range(Bn):
            for t, (c, k) in enumerate(hist[b]):
                dense[0][b, t], dense[1][b, t] = c, k
        want = oracle.absorbed(npy(qn), npy(qr), dense[0], dense[1], npy(W_UK), npy(W_UV), lens)
        compare(out, want, BF16, f"step {step}")


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_draft_loop_in_a_graph(cache):
    """page step -> K/V append -> decode attention, captured once and replayed."""
    H, Hk, D, page, Bn, W = 8, 2, 64, 8, 4, 5
    pages = Bn * W
    g, gen = np.random.default_rng(50), torch.Generator(DEV).manual_seed(50)
    cs = _table(W * page, D, g)
    ks, vs = (None, None) if cache == BF16 else (torch.full((Hk,), 0.02, device=DEV) for _ in "kv")
    kc, vc = (torch.zeros(pages, page, Hk, D, dtype=FP32, device=DEV).to(cache) for _ in "kv")
    table = i32(np.full((Bn, W), -1))
    kept, new, held = i32([0] * Bn), i32([1, 1, 0, 1]), i32([0] * Bn)
    free, span = i32(g.permutation(pages)), i32([0, pages])
    qkv = torch.zeros(Bn, H + 2 * Hk, D, dtype=BF16, device=DEV)
    step = B.PreparedPageStep(kept, new, held, table, free, span, page, pages, Bn)
    put = B.PreparedAppendKV(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], cs, step.out.positions,
                             step.out.slots, kc, vc, k_scale=ks, v_scale=vs)
    att = B.PreparedDecodeAttention(put.q_out, kc, vc, step.out.cache_lens, table, k_scale=ks,
                                    v_scale=vs, return_lse=True)

    def one():
        step.run()
        put.run()
        att.run()
        kept.copy_(step.out.cache_lens)
        held.copy_(step.out.held_pages)
        span.copy_(step.out.free_span)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    hist = [[] for _ in range(Bn)]
    for i in range(20):
        # sequence 2 is idle at first; the rows of a step are those of the live sequences
        live = [0, 1, 3] if i < 9 else [0, 1, 2, 3]
        new.copy_(i32([1 if b in live else 0 for b in range(Bn)]))
        qkv.copy_(_randn(gen, *qkv.shape, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        assert step.out.missing.item() == 0
        lens = step.out.cache_lens.tolist()
        for row, b in enumerate(live):
            hist[b].append(row)
        assert lens == [len(h) for h in hist]
        # (with a sequence idle, rows and sequences part ways: the query rows are gathered
        # by the caller; here only full steps line up)
        if len(live) == Bn:
            c = dict(q=put.q_out, k_cache=kc, v_cache=vc, cache_lens=step.out.cache_lens,
                     page_table=table, k_scale=ks, v_scale=vs)
            _check_decode(c, att.out, att.lse, what=f"step {i}")
    B.mla_device_status()
