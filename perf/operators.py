"""The paged-cache operators as they are measured: building page tables and slots, writing the
rows of a step into the caches, and attention of one new token over a paged key/value cache.

``run`` computes each operator with elementary torch operations, or, where ``own`` is true, with
the library's calls.  ``exact`` computes it in 64 bits from its definition.

Sequence lengths come from the case alone, so ``work`` knows them; page ids, keys, values and
queries come from the seed.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    return [
        # a verify step of 32 served sequences: up to 8 rows each, 64-row pages, idle slots
        dict(name="pages_step_b32", op="pages", batch=32, tmax=32768, new=8, page=64, short=False),
        # chunked prompts of many sequences at once, small pages
        dict(name="pages_prompts_b4096", op="pages", batch=4096, tmax=8192, new=512, page=16,
             short=False),
        # the rows of a verify step of 32 sequences, 8 rows each, 128 heads
        dict(name="latent_step_256", op="latent", rows=256, pad=0, heads=128, rank=512, nope=128,
             rope=64, dtype="bf16", page=64, interleaved=True),
        # a prompt's rows into the latent cache, 32 heads of the 512/192/256 geometry
        dict(name="latent_prompt_8191", op="latent", rows=8191, pad=5, heads=32, rank=512,
             nope=192, rope=64, dtype="bf16", page=64, interleaved=True),
        # one decode step of 64 drafted sequences into an 8-bit cache
        dict(name="kv_step_64_e4m3", op="kv", rows=64, pad=3, heads=32, kv_heads=8, dim=128,
             rope=128, dtype="bf16", cache="e4m3", page=64, by_head=False, interleaved=False),
        # a drafter's prompt rows, pages laid out head by head
        dict(name="kv_prompt_16383", op="kv", rows=16383, pad=0, heads=32, kv_heads=8, dim=128,
             rope=128, dtype="bf16", cache="bf16", page=64, by_head=True, interleaved=False),
        # the first draft tokens of one short sequence: latency
        dict(name="attn_one_61", op="attn", batch=1, tmin=61, tmax=61, idle=False, heads=16,
             kv_heads=8, dim=64, dtype="bf16", cache="bf16", page=16, by_head=False, window=0),
        # an ordinary draft step: 16 slots, some idle, one with a single token
        dict(name="attn_step_b16", op="attn", batch=16, tmin=200, tmax=4099, idle=True, heads=32,
             kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64, by_head=False, window=0),
        # batched paged serving: 32 sequences of 1024 to 32768 positions
        dict(name="attn_serving_b32", op="attn", batch=32, tmin=1024, tmax=32768, idle=False,
             heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64, by_head=False,
             window=0),
        # one long context: the work is split along the cache
        dict(name="attn_long_131072", op="attn", batch=1, tmin=131072, tmax=131072, idle=False,
             heads=32, kv_heads=4, dim=128, dtype="bf16", cache="bf16", page=64, by_head=True,
             window=0),
        # many sequences over an 8-bit cache
        dict(name="attn_e4m3_b64", op="attn", batch=64, tmin=1, tmax=16384, idle=False, heads=64,
             kv_heads=8, dim=128, dtype="bf16", cache="e4m3", page=64, by_head=False, window=0),
        # 32-bit cache, an odd group of 5 heads of 80, a sliding window, small pages
        dict(name="attn_fp32_window", op="attn", batch=8, tmin=100, tmax=4000, idle=True,
             heads=20, kv_heads=4, dim=80, dtype="fp32", cache="fp32", page=24, by_head=False,
             window=1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["pages", "latent", "kv", "attn", "attn", "attn"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "pages":
        batch, new = _log_int(rng, 1, 4096), _log_int(rng, 1, 512)
        return dict(op=op, batch=batch, tmax=_log_int(rng, 1, 8192), new=new, page=page,
                    short=rng.random() < 0.25)
    if op == "latent":
        heads = rng.choice([4, 16, 32, 64, 128])
        nope, rank = rng.choice([(128, 512), (192, 512), (256, 512), (64, 256)])
        rows = _log_int(rng, 1, 8191 * 32 // max(heads, 32) * 3 // 4)
        return dict(op=op, rows=rows, pad=rng.randint(0, rows // 4), heads=heads, rank=rank,
                    nope=nope, rope=64, dtype=rng.choice(["bf16", "bf16", "fp32"]), page=page,
                    interleaved=rng.random() < 0.5)
    dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"),
                               ("fp32", "fp32")])
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 112, 128, 192, 256])
    by_head = rng.random() < 0.4
    if op == "kv":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
        rows = _log_int(rng, 1, min(16383, 16383 * 32 * 128 // (2 * dim * max(heads, 32))))
        rope = rng.choice([dim, dim, dim // 2 // 16 * 16, 0])
        return dict(op=op, rows=rows, pad=rng.randint(0, rows // 4), heads=heads,
                    kv_heads=kv_heads, dim=dim, rope=rope, dtype=dtype, cache=cache, page=page,
                    by_head=by_head, interleaved=rng.random() < 0.5)
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    # positions of the whole batch, bounded by a third of the largest listed case's bytes
    most = 700_000_000 // (2 * kv_heads * dim * BYTES[cache])
    batch = _log_int(rng, 1, 64)
    tmax = _log_int(rng, 1, min(32768, max(1, most // batch)))
    return dict(op=op, batch=batch, tmin=rng.randint(1, tmax), tmax=tmax, idle=rng.random() < 0.3,
                heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, cache=cache, page=page,
                by_head=by_head, window=rng.choice([0, 0, 0, _log_int(rng, 1, tmax)]))


# ------------------------------------------------------------------------------ inputs

def _lens(case):
    """Cache lengths of an attention case, the new token included."""
    r = random.Random("%d %d %d" % (case["batch"], case["tmin"], case["tmax"]))
    t = [r.randint(case["tmin"], case["tmax"]) for _ in range(case["batch"])]
    if case["idle"]:
        for b in range(0, len(t), 5):
            t[b] = 0
        t[-1] = 1
    return t


def _visible(case):
    w = case["window"]
    return [min(t, w) if w else t for t in _lens(case)]


def _counts(case):
    """(kept lengths, new rows, pages held) of a page case, and the table's width."""
    r = random.Random("%d %d %d %d" % (case["batch"], case["tmax"], case["new"], case["page"]))
    page, width = case["page"], (case["tmax"] + case["new"]) // case["page"] + 2
    kept = [r.randint(0, case["tmax"]) for _ in range(case["batch"])]
    new = [r.randint(0, case["new"]) for _ in range(case["batch"])]
    # a rollback leaves a page or two more than the kept rows need
    held = [min(width, -(-t // page) + (r.randint(0, 1) if t else 0)) for t in kept]
    return kept, new, held, width


def _table(pos_count, rope, dev):
    """cos | sin of position * 10000^(-2i/rope), the angles in 64 bits."""
    f = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev),
                  -2.0 * torch.arange(rope // 2, dtype=torch.float64, device=dev) / max(rope, 1))
    a = torch.arange(pos_count, dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _cache(g, pages, page, heads, dim, kind, by_head, spread):
    """A cache as [pages, page, heads, dim]; by_head lays each page out head by head."""
    shape = (pages, heads, page, dim) if by_head else (pages, page, heads, dim)
    x = torch.randn(shape, generator=g, device=g.device)
    if kind == "e4m3":
        x = (x * spread).clamp_(-E4M3_MAX, E4M3_MAX)
    x = x.to(DTYPES[kind])
    return x.transpose(1, 2) if by_head else x


def _randn(g, *shape, dtype):
    return torch.randn(shape, generator=g, device=g.device).to(DTYPES[dtype])


def _rows_in_cache(g, case, rows):
    """Positions and slots of the rows: consecutive rows of sequences in shuffled pages, the
    padding behind them -1.  Returns (positions, slots, pages, positions in the table)."""
    page, pages, dev = case["page"], -(-rows // case["page"]) + 4, g.device
    perm = torch.randperm(pages, generator=g, device=dev)
    i = torch.arange(rows, device=dev)
    slots = perm[i // page] * page + i % page
    positions = (i * 7 + 3) % 8192
    live = rows - case["pad"]
    slots[live:] = -1
    positions[live:] = -1
    return positions.to(torch.int32), slots, pages, 8192


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = _prepare(case, g, dev)
    s["op"] = case["op"]
    if own:
        from mla_attention_speculative_gb300 import binding as B
        if case["op"] == "pages":
            s["call"] = B.PreparedPageStep(
                s["kept"], s["new"], s["held"], s["page_table"], s["free_pages"], s["free_span"],
                s["page"], s["num_pages"], s["max_rows"])
        elif case["op"] == "latent":
            s["call"] = B.PreparedAppendLatent(
                s["q"], s["kv"], s["cos_sin"], s["positions"], s["slots"], s["c_kv"], s["k_rope"],
                norm_weight=s["weight"], eps=s["eps"], interleaved=s["interleaved"],
                q_nope=s["q_nope"], q_rope=s["q_rope"])
        elif case["op"] == "kv":
            s["call"] = B.PreparedAppendKV(
                s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], s["slots"], s["k_cache"],
                s["v_cache"], interleaved=s["interleaved"], k_scale=s["k_scale"],
                v_scale=s["v_scale"], q_out=s["q_out"])
        else:
            s["call"] = B.PreparedDecodeAttention(
                s["q"], s["k_cache"], s["v_cache"], s["lens"], s["page_table"],
                window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
    return s


def _prepare(case, g, dev):
    if case["op"] == "pages":
        kept, new, held, width = _counts(case)
        page, B = case["page"], case["batch"]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        grow = sum(max(0, -(-(k + n) // page) - h) for k, n, h in zip(kept, new, held))
        free = max(1, grow // 2) if case["short"] else grow + 7
        num_pages = sum(held) + free + 5
        ids = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
        h = i32(held)
        col = torch.arange(width, device=dev)
        first = torch.cumsum(h, 0) - h
        at = (first[:, None] + col).clamp_max(num_pages - 1)
        table = torch.where(col < h[:, None], ids[at], -1).to(torch.int32)
        # the list's first entries went to earlier steps
        free_pages = torch.cat([ids[:3], ids[sum(held):sum(held) + free]]).contiguous()
        rows = sum(new)
        return dict(kept=i32(kept), new=i32(new), held=h, page_table=table.contiguous(),
                    free_pages=free_pages, free_span=i32([3, 3 + free]), page=page,
                    num_pages=num_pages, max_rows=rows + max(1, rows // 16))
    if case["op"] == "latent":
        N, H, n, r, d = (case[k] for k in ("rows", "heads", "nope", "rank", "rope"))
        dt = case["dtype"]
        positions, slots, pages, table = _rows_in_cache(g, case, N)
        return dict(q=_randn(g, N, H, n + d, dtype=dt), kv=_randn(g, N, r + d, dtype=dt),
                    weight=(1 + 0.1 * torch.randn(r, generator=g, device=dev)).to(DTYPES[dt]),
                    eps=1e-6, cos_sin=_table(table, d, dev), positions=positions, slots=slots,
                    interleaved=case["interleaved"], live=N - case["pad"],
                    c_kv=_randn(g, pages, case["page"], r, dtype=dt),
                    k_rope=_randn(g, pages, case["page"], d, dtype=dt),
                    q_nope=_randn(g, N, H, n, dtype=dt), q_rope=_randn(g, N, H, d, dtype=dt))
    H, Hk, D, dt, kind = (case[k] for k in ("heads", "kv_heads", "dim", "dtype", "cache"))
    k_scale = v_scale = None
    if kind == "e4m3":
        k_scale = 0.01 * (1 + torch.rand(Hk, generator=g, device=dev))
        v_scale = 0.01 * (1 + torch.rand(Hk, generator=g, device=dev))
    if case["op"] == "kv":
        N, d = case["rows"], case["rope"]
        positions, slots, pages, table = _rows_in_cache(g, case, N)
        # q, k and v are views of one projection's rows, as the layer before leaves them
        qkv = _randn(g, N, H + 2 * Hk, D, dtype=dt)
        cache = lambda: _cache(g, pages, case["page"], Hk, D, kind, case["by_head"], 60.0)  # noqa: E731
        return dict(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], k_scale=k_scale,
                    v_scale=v_scale, cos_sin=_table(table, d, dev) if d else None, rope=d,
                    positions=positions, slots=slots, live=N - case["pad"], k_cache=cache(),
                    v_cache=cache(), interleaved=case["interleaved"],
                    q_out=_randn(g, N, H, D, dtype=dt))
    lens, page = _lens(case), case["page"]
    used = [-(-t // page) for t in lens]
    pages, width = sum(used) + 3, max(used) + 1
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    u = torch.tensor(used, device=dev)
    col = torch.arange(width, device=dev)
    first = torch.cumsum(u, 0) - u
    at = (first[:, None] + col).clamp_max(pages - 1)
    table = torch.where(col < u[:, None], ids[at], -1).to(torch.int32).contiguous()
    return dict(q=_randn(g, case["batch"], H, D, dtype=dt),
                k_cache=_cache(g, pages, page, Hk, D, kind, case["by_head"], 60.0),
                v_cache=_cache(g, pages, page, Hk, D, kind, case["by_head"], 60.0),
                k_scale=k_scale, v_scale=v_scale, page_table=table, window=case["window"],
                lens=torch.tensor(lens, dtype=torch.int32, device=dev))


# ----------------------------------------------------------------------------- one pass

def run(s):
    if own:
        s["call"].run()
        if s["op"] == "pages":
            o = s["call"].out
            return dict(page_table=s["page_table"], cache_lens=o.cache_lens, held=o.held_pages,
                        row_start=o.row_start, positions=o.positions, slots=o.slots,
                        free_span=o.free_span, missing=o.missing)
        if s["op"] == "latent":
            return dict(q_nope=s["q_nope"], q_rope=s["q_rope"], c_kv=s["c_kv"],
                        k_rope=s["k_rope"])
        if s["op"] == "kv":
            return dict(q=s["q_out"], k=s["k_cache"], v=s["v_cache"])
        return dict(out=s["call"].out, lse=s["call"].lse)
    return _PLAIN[s["op"]](s)


def _plain_pages(s):
    page, table, width = s["page"], s["page_table"], s["page_table"].shape[1]
    kept, held = s["kept"].long(), s["held"].long()
    total = (kept + s["new"]).clamp_max(width * page)
    grow = ((total + page - 1) // page - held).clamp_min(0)
    base = torch.cumsum(grow, 0) - grow
    have = (s["free_span"][1] - s["free_span"][0]).long()
    got = torch.minimum(grow, (have - base).clamp_min(0))
    held_out = held + got
    lens = torch.minimum(total, held_out * page)
    col = torch.arange(width, device=table.device)
    take = (s["free_span"][0] + base[:, None] + col - held[:, None])
    fresh = (col >= held[:, None]) & (col < held_out[:, None])
    ids = s["free_pages"][take.clamp(0, s["free_pages"].numel() - 1)]
    table.copy_(torch.where(fresh, ids, table))
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device=table.device),
                        torch.cumsum(s["new"], 0)])
    row = torch.arange(s["max_rows"], device=table.device)
    seq = (torch.searchsorted(starts, row, right=True) - 1).clamp_max(kept.numel() - 1)
    live = row < starts[-1]
    pos = kept[seq] + row - starts[seq]
    home = table.long()[seq, (pos // page).clamp_max(width - 1)]
    slots = torch.where(live & (pos < lens[seq]), home * page + pos % page, -1)
    taken, want = got.sum(), grow.sum()
    i32 = torch.int32
    return dict(page_table=table, cache_lens=lens.to(i32), held=held_out.to(i32),
                row_start=starts.to(i32), positions=torch.where(live, pos, -1).to(i32),
                slots=slots, missing=(want - taken).to(i32).reshape(1),
                free_span=torch.stack([s["free_span"][0] + taken, s["free_span"][1]]).to(i32))


def _rotate(x, cos_sin, positions, interleaved):
    """The rotation of x [rows, heads, d] in 32 bits."""
    half = x.shape[-1] // 2
    t = cos_sin[positions.long()]
    cos, sin = t[:, None, :half], t[:, None, half:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(x.shape)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_latent(s):
    n, (r, live) = s["q_nope"].shape[-1], (s["c_kv"].shape[-1], s["live"])
    page = s["c_kv"].shape[1]
    pos, slots = s["positions"][:live], s["slots"][:live]
    q, kv = s["q"][:live].float(), s["kv"][:live].float()
    dt = s["q"].dtype
    s["q_nope"][:live] = s["q"][:live, :, :n]
    s["q_rope"][:live] = _rotate(q[..., n:], s["cos_sin"], pos, s["interleaved"]).to(dt)
    c = kv[:, :r]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    s["c_kv"][slots // page, slots % page] = c.to(dt)
    k = _rotate(kv[:, None, r:], s["cos_sin"], pos, s["interleaved"])[:, 0]
    s["k_rope"][slots // page, slots % page] = k.to(dt)
    return dict(q_nope=s["q_nope"], q_rope=s["q_rope"], c_kv=s["c_kv"], k_rope=s["k_rope"])


def _put(cache, slots, x, scale):
    page = cache.shape[1]
    if scale is not None:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    x = x.to(cache.dtype)
    if cache.element_size() == 1:  # indexed as bytes
        cache.view(torch.uint8)[slots // page, slots % page] = x.view(torch.uint8)
    else:
        cache[slots // page, slots % page] = x


def _plain_kv(s):
    live, d = s["live"], s["rope"]
    pos, slots = s["positions"][:live], s["slots"][:live]
    q, k, v = (s[x][:live].float() for x in ("q", "k", "v"))
    if d:
        turn = lambda x: torch.cat([_rotate(x[..., :d], s["cos_sin"], pos, s["interleaved"]),  # noqa: E731
                                    x[..., d:]], -1)
        q, k = turn(q), turn(k)
    s["q_out"][:live] = q.to(s["q"].dtype)
    _put(s["k_cache"], slots, k, s["k_scale"])
    _put(s["v_cache"], slots, v, s["v_scale"])
    return dict(q=s["q_out"], k=s["k_cache"], v=s["v_cache"])


def _gathered(cache, table, scale):
    """[batch, heads, positions, dim] in 32 bits."""
    t = table.long().clamp_min(0)
    x = cache.view(torch.uint8)[t].view(cache.dtype) if cache.element_size() == 1 else cache[t]
    x = x.flatten(1, 2).float().transpose(1, 2)
    return x if scale is None else x * scale[:, None, None]


def _plain_attn(s):
    q, lens = s["q"], s["lens"]
    B, H, D = q.shape
    k = _gathered(s["k_cache"], s["page_table"], s["k_scale"])
    Hk, T = k.shape[1], k.shape[2]
    qs = q.float().view(B, Hk, H // Hk, D) / math.sqrt(D)
    scores = torch.matmul(qs, k.transpose(2, 3))
    pos = torch.arange(T, device=q.device)
    seen = pos < lens[:, None]
    if s["window"]:
        seen &= pos >= lens[:, None] - s["window"]
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["page_table"], s["v_scale"])
    # positions behind a sequence may hold anything
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return dict(out=o.view(B, H, D).to(q.dtype), lse=(top + total.log()).view(B, H))


_PLAIN = {"pages": _plain_pages, "latent": _plain_latent, "kv": _plain_kv, "attn": _plain_attn}


# ------------------------------------------------------------------------ work and truth

def work(case):
    if case["op"] == "pages":
        kept, new, held, _ = _counts(case)
        rows, page = sum(new), case["page"]
        grow = sum(max(0, -(-(k + n) // page) - h) for k, n, h in zip(kept, new, held))
        # three counts in, three out; a new page's id read and written; a held page read where
        # rows go into it; a position and a slot per row
        return dict(bytes=case["batch"] * 4 * 6 + grow * 8 + case["batch"] * 4
                    + (rows + max(1, rows // 16)) * 12, flops=0)
    if case["op"] == "latent":
        live, b = case["rows"] - case["pad"], BYTES[case["dtype"]]
        q = case["heads"] * (case["nope"] + case["rope"])
        kv = case["rank"] + case["rope"]
        return dict(bytes=live * ((q + kv) * b * 2 + 12 + case["rope"] * 4), flops=live * (
            3 * case["heads"] * case["rope"] + 4 * case["rank"]))
    if case["op"] == "kv":
        live, b = case["rows"] - case["pad"], BYTES[case["dtype"]]
        kv = 2 * case["kv_heads"] * case["dim"]
        return dict(bytes=live * (case["heads"] * case["dim"] * b * 2 + kv * (
            b + BYTES[case["cache"]]) + 12 + case["rope"] * 4), flops=live * 3 * case["rope"] * (
                case["heads"] + case["kv_heads"]))
    seen = sum(_visible(case))
    row = case["kv_heads"] * case["dim"] * BYTES[case["cache"]]
    out = case["batch"] * case["heads"] * (2 * case["dim"] * BYTES[case["dtype"]] + 4)
    return dict(bytes=seen * (2 * row) + 4 * -(-seen // case["page"]) + out,
                flops=4 * seen * case["heads"] * case["dim"])


def _spin64(x, angles, interleaved):
    """Complex rotation of x [rows, heads, d] by table angles given as cos + i sin."""
    half = x.shape[-1] // 2
    z = torch.complex(*((x[..., 0::2], x[..., 1::2]) if interleaved
                        else (x[..., :half], x[..., half:])))
    z = z * angles[:, None]
    y = torch.empty_like(x)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = z.real, z.imag
    else:
        y[..., :half], y[..., half:] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] == "pages":
        return None
    dev = torch.device("cuda")
    s = _prepare(case, torch.Generator(device=dev).manual_seed(int(seed)), dev)
    d64 = torch.float64
    if case["op"] in ("latent", "kv"):
        keep = case["rows"] - case["pad"]
        half = case["rope"] // 2
        rows = s["positions"][:keep].long()
        angles = None
        if half:
            t = s["cos_sin"].to(d64)[rows]
            angles = torch.complex(t[:, :half].contiguous(), t[:, half:].contiguous())
        flat = s["slots"][:keep]

        def written(cache, x):
            pages, page = cache.shape[:2]
            y = cache.to(d64).reshape(pages * page, *cache.shape[2:])
            y[flat] = x
            return y.view(cache.shape)

        def upto(old, x):
            return torch.cat([x, old[keep:].to(d64)])

        if case["op"] == "latent":
            n, r = case["nope"], case["rank"]
            q, kv = s["q"][:keep].to(d64), s["kv"][:keep].to(d64)
            c = kv[:, :r] / torch.sqrt(kv[:, :r].square().sum(1, keepdim=True) / r + s["eps"])
            return dict(
                q_nope=upto(s["q_nope"], q[..., :n]),
                q_rope=upto(s["q_rope"], _spin64(q[..., n:], angles, case["interleaved"])),
                c_kv=written(s["c_kv"], c * s["weight"].to(d64)),
                k_rope=written(s["k_rope"],
                               _spin64(kv[:, None, r:], angles, case["interleaved"])[:, 0]))
        q, k, v = (s[x][:keep].to(d64) for x in ("q", "k", "v"))
        if half:
            q, k = q.clone(), k.clone()
            for x in (q, k):
                x[..., :2 * half] = _spin64(x[..., :2 * half], angles, case["interleaved"])
        if s["k_scale"] is not None:
            k, v = k / s["k_scale"].to(d64)[:, None], v / s["v_scale"].to(d64)[:, None]
            k, v = k.clamp(-E4M3_MAX, E4M3_MAX), v.clamp(-E4M3_MAX, E4M3_MAX)
        return dict(q=upto(s["q_out"], q), k=written(s["k_cache"], k),
                    v=written(s["v_cache"], v))
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(case["batch"], H, D, dtype=d64, device=dev)
    lse = torch.full((case["batch"], H), -math.inf, dtype=d64, device=dev)
    for b, t in enumerate(_lens(case)):
        at = torch.arange(max(0, t - case["window"]) if case["window"] else 0, t, device=dev)
        if not at.numel():
            continue
        page, row = s["page_table"][b].long()[at // case["page"]], at % case["page"]
        for h in range(Hk):
            k, v = s["k_cache"][page, row, h].to(d64), s["v_cache"][page, row, h].to(d64)
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].to(d64), v * s["v_scale"][h].to(d64)
            mine = slice(h * H // Hk, (h + 1) * H // Hk)
            x = s["q"][b, mine].to(d64) @ k.T * D ** -0.5
            lse[b, mine] = torch.logsumexp(x, 1)
            out[b, mine] = torch.exp(x - lse[b, mine][:, None]) @ v
    return dict(out=out, lse=lse)
