"""Further paged-cache operators as they are measured: attention of a step's new rows over a
paged key/value cache, and the pages themselves forked, copied, released and compacted.

``run`` computes each operator with elementary torch operations, or, where ``own`` is true, with
the library's calls.  ``exact`` computes it in 64 bits from its definition.

Lengths, and which sequences fork or end, come from the case alone, so ``work`` knows them; page
ids, keys, values and queries come from the seed.
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
        # a short prompt's last draft rows, one sequence: latency
        dict(name="chunk_one_5", op="chunk", batch=1, kmin=56, kmax=56, nmin=5, nmax=5, idle=False,
             pad=0, heads=16, kv_heads=8, dim=64, dtype="bf16", cache="bf16", page=16,
             by_head=False, window=0),
        # the draft rows of 16 served sequences, some slots idle, a padded step
        dict(name="chunk_verify_b16", op="chunk", batch=16, kmin=200, kmax=4099, nmin=1, nmax=8,
             idle=True, pad=9, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64,
             by_head=False, window=0),
        # a whole prompt
        dict(name="chunk_prompt_8192", op="chunk", batch=1, kmin=0, kmax=0, nmin=8192, nmax=8192,
             idle=False, pad=0, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="bf16", page=64,
             by_head=False, window=0),
        # prompts in chunks beside sequences that add a row or two, an 8-bit cache
        dict(name="chunk_mixed_e4m3", op="chunk", batch=24, kmin=0, kmax=8192, nmin=1, nmax=512,
             idle=True, pad=37, heads=64, kv_heads=8, dim=128, dtype="bf16", cache="e4m3", page=64,
             by_head=False, window=0),
        # 16 rows over one long context: the work is split along the cache
        dict(name="chunk_long_131072", op="chunk", batch=1, kmin=131056, kmax=131056, nmin=16,
             nmax=16, idle=False, pad=0, heads=32, kv_heads=4, dim=128, dtype="bf16", cache="bf16",
             page=64, by_head=True, window=0),
        # 32-bit cache, an odd group of 5 heads of 80, a sliding window, small pages
        dict(name="chunk_fp32_window", op="chunk", batch=8, kmin=0, kmax=4000, nmin=1, nmax=129,
             idle=True, pad=3, heads=20, kv_heads=4, dim=80, dtype="fp32", cache="fp32", page=24,
             by_head=False, window=1000),
        # four prompts sampled eight times each: seven idle slots take a prompt's pages
        dict(name="fork_samples_b32", op="fork", batch=32, parents=4, tmax=32768, heads=8, dim=128,
             cache="bf16", page=64, by_head=False, layers=2, short=False),
        # many short prompts forked at once, small pages head by head
        dict(name="fork_b1024", op="fork", batch=1024, parents=128, tmax=4096, heads=8, dim=128,
             cache="bf16", page=16, by_head=True, layers=4, short=False),
        # a verify step's rejections: a page here and there comes back
        dict(name="release_step_b32", op="release", batch=32, tmax=8192, end=0.0, cut=16,
             shared=0.0, page=64),
        # many sequences end at once, half of them sharing a prompt's pages
        dict(name="release_b4096", op="release", batch=4096, tmax=4096, end=0.5, cut=64,
             shared=0.5, page=16),
        # a small pool brought together
        dict(name="compact_256", op="compact", num_pages=256, batch=16, live=0.4, shared=0.0,
             heads=8, dim=128, cache="bf16", page=16, by_head=False, layers=1),
        # half of a pool of 2 x 512 MB in use, scattered
        dict(name="compact_4096", op="compact", num_pages=4096, batch=128, live=0.5, shared=0.25,
             heads=8, dim=128, cache="bf16", page=64, by_head=False, layers=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "fork", "release", "compact"])
    if op == "chunk":
        dtype, cache = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"),
                                   ("fp32", "fp32")])
        kv_heads = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 96, 112, 128, 192, 256])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        batch = _log_int(rng, 1, 32)
        # operations and cached bytes of the whole batch, within the largest listed cases'
        flops = 2e11 if dtype == "bf16" else 1e10
        kmax = _log_int(rng, 1, min(65536, 200_000_000 // (2 * kv_heads * dim * BYTES[cache]
                                                           * batch)))
        most = max(1, int(flops / (4.0 * heads * dim * batch * (kmax + 1024))))
        nmax = _log_int(rng, 1, min(1024, most))
        return dict(op=op, batch=batch, kmin=rng.randint(0, kmax), kmax=kmax,
                    nmin=rng.randint(1, nmax), nmax=nmax, idle=rng.random() < 0.3,
                    pad=rng.choice([0, 0, _log_int(rng, 1, 64)]), heads=heads, kv_heads=kv_heads,
                    dim=dim, dtype=dtype, cache=cache,
                    page=rng.choice([8, 16, 20, 24, 32, 64, 128]), by_head=rng.random() < 0.4,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, kmax + nmax)]))
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "release":
        return dict(op=op, batch=_log_int(rng, 1, 4096), tmax=_log_int(rng, 1, 4096),
                    end=rng.choice([0.0, 0.1, 0.5]), cut=_log_int(rng, 1, 64),
                    shared=rng.choice([0.0, 0.5]), page=max(page, 16))
    kind = dict(heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 80, 96, 128, 256]),
                cache=rng.choice(["bf16", "bf16", "fp32"]), page=page,
                by_head=rng.random() < 0.4)
    row = kind["heads"] * kind["dim"] * BYTES[kind["cache"]]
    if op == "fork":
        batch = _log_int(rng, 2, 512)
        # bytes of the pool, below a listed case's
        most = max(1, 400_000_000 // (2 * row * max(1, batch // 4)))
        return dict(op=op, batch=batch, parents=max(1, batch // rng.choice([2, 4, 8])),
                    tmax=_log_int(rng, 1, min(8192, most)), layers=rng.choice([1, 2]),
                    short=rng.random() < 0.2, **kind)
    num_pages = _log_int(rng, 2, min(4096, 300_000_000 // (row * page)))
    return dict(op=op, num_pages=num_pages, batch=_log_int(rng, 1, min(128, num_pages)),
                live=rng.uniform(0.05, 0.95), shared=rng.choice([0.0, 0.25]), layers=1, **kind)


# ------------------------------------------------------------------------------ inputs

def _seeded(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _steps(case):
    """(kept lengths, new rows) of a chunk case; idle slots have neither."""
    r = _seeded(case)
    kept = [r.randint(case["kmin"], case["kmax"]) for _ in range(case["batch"])]
    new = [r.randint(case["nmin"], case["nmax"]) for _ in range(case["batch"])]
    if case["idle"]:
        for b in range(0, case["batch"], 5):
            kept[b] = new[b] = 0
        new[-1] = 1
    return kept, new


def _pages_of(case, lens):
    return [-(-t // case["page"]) for t in lens]


def _forks(case):
    """(lengths, source of each slot or -1) of a fork case: the parents lie among idle slots."""
    r = _seeded(case)
    batch, parents = case["batch"], min(case["parents"], case["batch"] - 1)
    at = sorted(r.sample(range(batch), parents))
    lens = [0] * batch
    for b in at:
        lens[b] = r.randint(max(1, case["tmax"] // 4), case["tmax"])
    src = [-1] * batch
    for b in range(batch):
        if not lens[b]:
            src[b] = at[r.randrange(parents)]
    return lens, src


def _cuts(case):
    """(lengths, kept lengths, pages held, pages of a shared prompt) of a release case."""
    r = _seeded(case)
    page, batch = case["page"], case["batch"]
    lens = [r.randint(1, case["tmax"]) for _ in range(batch)]
    kept = [0 if r.random() < case["end"] else max(0, t - r.randint(0, case["cut"])) for t in lens]
    held = [-(-t // page) + r.randint(0, 1) for t in lens]
    prompt = max(1, case["tmax"] // page // 4) if case["shared"] else 0
    sharing = [bool(prompt) and r.random() < case["shared"] for _ in range(batch)]
    return kept, held, prompt, sharing


def _live(case):
    """Pages held by each sequence, and those of the first one that others share."""
    r = _seeded(case)
    n = max(1, int(case["num_pages"] * case["live"]))
    batch = min(case["batch"], n)
    cuts = sorted(r.sample(range(1, n), batch - 1)) if batch > 1 else []
    held = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    sharers = [b for b in range(1, batch) if r.random() < case["shared"]]
    return held, sharers


def _randn(g, shape, dtype):
    """Normal values drawn in pieces, so that a large tensor needs no 32-bit copy beside it."""
    x = torch.empty(shape, dtype=DTYPES[dtype], device=g.device)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - i)
        y = torch.randn(n, generator=g, device=g.device)
        if dtype == "e4m3":
            y = (y * 60.0).clamp_(-E4M3_MAX, E4M3_MAX)
        flat[i:i + n] = y.to(DTYPES[dtype])
    return x


def _cache(g, case, pages, heads):
    """A cache as [pages, page, heads, dim]; by_head lays each page out head by head."""
    if case["by_head"]:
        return _randn(g, (pages, heads, case["page"], case["dim"]), case["cache"]).transpose(1, 2)
    return _randn(g, (pages, case["page"], heads, case["dim"]), case["cache"])


def _table(held, ids, width, dev):
    """A table whose rows take `held` ids each, -1 behind them."""
    h = torch.tensor(held, device=dev)
    col = torch.arange(width, device=dev)
    at = (torch.cumsum(h, 0) - h)[:, None] + col
    return torch.where(col < h[:, None], ids[at.clamp_max(ids.numel() - 1)],
                       -1).to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = _prepare(case, g, dev)
    s["op"] = case["op"]
    if own:
        from mla_attention_speculative_gb300 import binding as B
        if case["op"] == "chunk":
            s["call"] = B.PreparedChunkAttention(
                s["q"], s["k_cache"], s["v_cache"], s["kept"], s["lens"], s["row_start"],
                s["page_table"], window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                out=s["out"], lse=s["lse"])
        elif case["op"] == "fork":
            s["call"] = B.PreparedPageFork(
                s["src"], s["lens"], s["held"], s["page_table"], s["shares"], s["free_pages"],
                s["free_span"], s["page"])
            o = s["call"].out
            s["copy"] = B.PreparedPageCopy(s["caches"], o.move_src, o.move_dst, o.moves,
                                           o.move_rows)
        elif case["op"] == "release":
            s["call"] = B.PreparedPageRelease(
                s["kept"], s["held"], s["page_table"], s["shares"], s["free_pages"],
                s["free_span"], s["page"])
        else:
            s["call"] = B.PreparedPageCompact(s["held"], s["page_table"], s["shares"],
                                              s["free_pages"])
            o = s["call"].out
            s["copy"] = B.PreparedPageCopy(s["caches"], o.move_src, o.move_dst, o.moves)
    return s


def _prepare(case, g, dev):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=g, device=dev).to(torch.int32)  # noqa: E731
    if case["op"] == "chunk":
        H, Hk, D = (case[k] for k in ("heads", "kv_heads", "dim"))
        kept, new = _steps(case)
        lens = [k + n for k, n in zip(kept, new)]
        used = _pages_of(case, lens)
        pages, starts = sum(used) + 3, [0]
        for n in new:
            starts.append(starts[-1] + n)
        rows = starts[-1] + case["pad"]
        k_scale = v_scale = None
        if case["cache"] == "e4m3":
            k_scale = 0.01 * (1 + torch.rand(Hk, generator=g, device=dev))
            v_scale = 0.01 * (1 + torch.rand(Hk, generator=g, device=dev))
        # queries are a view of one projection's rows; rows behind the step keep what out holds
        qkv = _randn(g, (rows, H + 2 * Hk, D), case["dtype"])
        return dict(q=qkv[:, :H], k_cache=_cache(g, case, pages, Hk),
                    v_cache=_cache(g, case, pages, Hk), k_scale=k_scale, v_scale=v_scale,
                    kept=i32(kept), lens=i32(lens), row_start=i32(starts), window=case["window"],
                    page_table=_table(used, perm(pages), max(used) + 1, dev),
                    out=_randn(g, (rows, H, D), case["dtype"]),
                    lse=torch.randn((rows, H), generator=g, device=dev), steps=(kept, new))
    if case["op"] == "fork":
        lens, src = _forks(case)
        held = _pages_of(case, lens)
        wants = sum(1 for s in src if s >= 0 and lens[s] % case["page"])
        free = max(1, wants // 2) if case["short"] else wants + 5
        pages = sum(held) + free + 3
        ids = perm(pages)
        listed_pages = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        listed_pages[3:3 + free] = ids[sum(held):sum(held) + free]
        return dict(src=i32(src), lens=i32(lens), held=i32(held), page=case["page"],
                    page_table=_table(held, ids, max(held) + 2, dev), free_pages=listed_pages,
                    free_span=i32([3, 3 + free]),
                    shares=torch.zeros(pages, dtype=torch.int32, device=dev),
                    caches=[_cache(g, case, pages, case["heads"])
                            for _ in range(2 * case["layers"])])
    if case["op"] == "release":
        kept, held, prompt, sharing = _cuts(case)
        own_pages = [max(0, h - prompt) if s else h for h, s in zip(held, sharing)]
        pages = prompt + sum(own_pages) + 9
        ids = perm(pages)
        # a sharing sequence's first pages are the prompt's
        h, o = torch.tensor(held, device=dev), torch.tensor(own_pages, device=dev)
        col = torch.arange(max(held) + 1, device=dev)
        lead = (h - o)[:, None]
        at = (prompt + torch.cumsum(o, 0) - o)[:, None] + col - lead
        pick = torch.where(col < lead, col, at).clamp(0, pages - 1)
        table = torch.where(col < h[:, None], ids[pick], -1).to(torch.int32).contiguous()
        shares = torch.zeros(pages, dtype=torch.int32, device=dev)
        for j in range(prompt):
            holders = sum(1 for x, s in zip(held, sharing) if s and x > j)
            shares[ids[j].long()] = max(0, holders - 1)
        free = ids[pages - 9:]
        listed_pages = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        listed_pages[pages - 12:pages - 3] = free
        return dict(kept=i32(kept), held=i32(held), page_table=table, shares=shares,
                    free_pages=listed_pages, free_span=i32([pages - 12, pages - 3]),
                    page=case["page"])
    held, sharers = _live(case)
    pages = case["num_pages"]
    ids = perm(pages)
    width = max(held) + held[0] + 1
    table = _table(held, ids, width, dev)
    shares = torch.zeros(pages, dtype=torch.int32, device=dev)
    # sharers hold the first sequence's pages in front of their own
    for b in sharers:
        table[b] = torch.cat([table[0, :held[0]], table[b, :width - held[0]]])
    if sharers:
        shares[ids[:held[0]].long()] = len(sharers)
    total = [h + held[0] if b in set(sharers) else h for b, h in enumerate(held)]
    return dict(held=i32(total), page_table=table, shares=shares,
                free_pages=torch.full((pages,), -1, dtype=torch.int32, device=dev),
                caches=[_cache(g, case, pages, case["heads"]) for _ in range(2 * case["layers"])])


# ----------------------------------------------------------------------------- one pass

def run(s):
    if own:
        s["call"].run()
        if s["op"] == "chunk":
            return dict(out=s["out"], lse=s["lse"])
        o = s["call"].out
        if s["op"] == "release":
            return dict(held=o.held_pages, shares=o.shares, free_span=o.free_span,
                        free_pages=s["free_pages"])
        s["copy"].run()
        if s["op"] == "fork":
            return dict(page_table=s["page_table"], lens=o.cache_lens, held=o.held_pages,
                        shares=o.shares, free_span=o.free_span, missing=o.missing,
                        moves=o.moves, caches=s["caches"])
        return dict(page_table=o.page_table, shares=o.shares, free_span=o.free_span,
                    free_pages=s["free_pages"], moves=o.moves, caches=s["caches"])
    return _PLAIN[s["op"]](s)


def _gathered(cache, ids, scale):
    """The pages of one sequence as [heads, positions, dim] in 32 bits."""
    x = cache.view(torch.uint8)[ids].view(cache.dtype) if cache.element_size() == 1 else cache[ids]
    x = x.flatten(0, 1).float().transpose(0, 1)
    return x if scale is None else x * scale[:, None, None]


def _plain_chunk(s):
    q, (kept, new) = s["q"], s["steps"]
    H, D = q.shape[1:]
    page, Hk = s["k_cache"].shape[1:3]
    row = 0
    for b, (k0, n) in enumerate(zip(kept, new)):
        if not n:
            continue
        total = k0 + n
        ids = s["page_table"][b, :-(-total // page)].long()
        keys = _gathered(s["k_cache"], ids, s["k_scale"])[:, :total]
        values = _gathered(s["v_cache"], ids, s["v_scale"])[:, :total]
        pos = torch.arange(total, device=q.device)
        for i in range(0, n, 2048):
            m = min(2048, n - i)
            at = torch.arange(k0 + i, k0 + i + m, device=q.device)
            x = q[row + i:row + i + m].float().view(m, Hk, H // Hk, D).permute(1, 2, 0, 3)
            scores = torch.matmul(x / math.sqrt(D), keys.transpose(1, 2)[:, None])
            seen = pos <= at[:, None]
            if s["window"]:
                seen &= pos > at[:, None] - s["window"]
            scores = scores.masked_fill(~seen, float("-inf"))
            top = scores.amax(-1, keepdim=True)
            p = torch.exp(scores - top)
            sums = p.sum(-1, keepdim=True)
            o = torch.matmul(p, values[:, None]) / sums
            s["out"][row + i:row + i + m] = o.permute(2, 0, 1, 3).reshape(m, H, D).to(q.dtype)
            s["lse"][row + i:row + i + m] = (top + sums.log())[..., 0].permute(2, 0, 1).reshape(
                m, H)
        row += n
    return dict(out=s["out"], lse=s["lse"])


def _copy_rows(caches, src, dst, rows=None):
    for c in caches:
        moved = c[src]
        if rows is not None:
            keep = torch.arange(c.shape[1], device=c.device) < rows[:, None]
            moved = torch.where(keep[:, :, None, None], moved, c[dst])
        c[dst] = moved


def _plain_fork(s):
    page, table, width = s["page"], s["page_table"], s["page_table"].shape[1]
    src, held = s["src"].long(), s["held"].long()
    child = (src >= 0) & (held == 0)
    of = src.clamp_min(0)
    total = torch.minimum(s["lens"].long()[of], held[of] * page)
    full, rest = total // page, total % page
    wants = child & (rest > 0)
    rank = torch.cumsum(wants.long(), 0) - wants.long()
    have = (s["free_span"][1] - s["free_span"][0]).long()
    got = wants & (rank < have)
    fresh = s["free_pages"][(s["free_span"][0] + rank).clamp_max(s["free_pages"].numel() - 1)]
    col = torch.arange(width, device=table.device)
    theirs = table[of]
    shared = child[:, None] & (col < full[:, None])
    last = got[:, None] & (col == full[:, None])
    moved = torch.where(last, theirs, 0).sum(1)
    table.copy_(torch.where(shared, theirs, torch.where(last, fresh[:, None], table)))
    shares = s["shares"] + torch.bincount(theirs[shared].long(),
                                          minlength=s["shares"].numel()).to(torch.int32)
    lens = torch.where(child, torch.where(got | (rest == 0), total, full * page), s["lens"])
    held_out = torch.where(child, full + got, held)
    taken, i32 = got.sum(), torch.int32
    _copy_rows(s["caches"], moved[got], fresh[got].long(), rest[got])
    return dict(page_table=table, lens=lens.to(i32), held=held_out.to(i32), shares=shares,
                free_span=torch.stack([s["free_span"][0] + taken, s["free_span"][1]]).to(i32),
                missing=(wants.sum() - taken).to(i32).reshape(1), moves=taken.to(i32).reshape(1),
                caches=s["caches"])


def _plain_release(s):
    page, table = s["page"], s["page_table"]
    held = s["held"].long()
    need = (s["kept"].long() + page - 1) // page
    col = torch.arange(table.shape[1], device=table.device)
    drop = (col >= need[:, None]) & (col < held[:, None])
    shares = s["shares"] - torch.bincount(table[drop].long(),
                                          minlength=s["shares"].numel()).to(torch.int32)
    freed = torch.nonzero(shares < 0)[:, 0]
    n, first, end = freed.numel(), s["free_span"][0], s["free_span"][1]
    # in front of the list as far as there is room, the others behind it
    front = first.clamp_max(n)
    i = torch.arange(n, device=table.device)
    at = torch.where(i < front, first - front + i, end + i - front)
    s["free_pages"][at.long()] = freed.to(torch.int32)
    return dict(held=torch.minimum(held, need).to(torch.int32), shares=shares.clamp_min(0),
                free_span=torch.stack([first - front, end + n - front]).to(torch.int32),
                free_pages=s["free_pages"])


def _plain_compact(s):
    table, held, pages = s["page_table"], s["held"].long(), s["shares"].numel()
    used = torch.arange(table.shape[1], device=table.device) < held[:, None]
    live = torch.zeros(pages, dtype=torch.bool, device=table.device)
    live[table[used].long()] = True
    count = int(live.sum())
    src = torch.nonzero(live[count:])[:, 0] + count
    dst = torch.nonzero(~live[:count])[:, 0]
    to = torch.arange(pages, device=table.device)
    to[src] = dst
    shares = s["shares"].clone()
    shares[dst] = s["shares"][src]
    shares[count:] = 0
    s["free_pages"][:pages - count] = torch.arange(count, pages, device=table.device,
                                                   dtype=torch.int32)
    _copy_rows(s["caches"], src, dst)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=table.device)  # noqa: E731
    return dict(page_table=torch.where(used, to[table.long().clamp_min(0)], -1).to(torch.int32),
                shares=shares, free_span=i32([0, pages - count]), free_pages=s["free_pages"],
                moves=i32([src.numel()]), caches=s["caches"])


_PLAIN = {"chunk": _plain_chunk, "fork": _plain_fork, "release": _plain_release,
          "compact": _plain_compact}


# ------------------------------------------------------------------------ work and truth

def work(case):
    if case["op"] == "chunk":
        kept, new = _steps(case)
        seen = pairs = 0
        for k, n in zip(kept, new):
            if n:
                w = case["window"] or k + n
                seen += k + n - max(0, k + 1 - w)
                # row i sees min(k + i + 1, w) positions
                grow = min(n, max(0, w - k - 1))
                pairs += grow * k + grow * (grow + 1) // 2 + (n - grow) * w
        row = 2 * case["kv_heads"] * case["dim"] * BYTES[case["cache"]]
        io = sum(new) * case["heads"] * (2 * case["dim"] * BYTES[case["dtype"]] + 4)
        return dict(bytes=seen * row + 4 * -(-seen // case["page"]) + io,
                    flops=4 * pairs * case["heads"] * case["dim"])
    if case["op"] == "release":
        kept, held, _, _ = _cuts(case)
        drops = sum(max(0, h - -(-k // case["page"])) for k, h in zip(kept, held))
        # two counts in, one out; a dropped page's id and count, its count and place in the list
        return dict(bytes=12 * case["batch"] + drops * 16, flops=0)
    row = case["heads"] * case["dim"] * BYTES[case["cache"]] * 2 * case["layers"]
    if case["op"] == "fork":
        lens, src = _forks(case)
        wants = [lens[b] % case["page"] for b in src if b >= 0 and lens[b] % case["page"]]
        full = sum(lens[b] // case["page"] for b in src if b >= 0)
        got = len(wants) if not case["short"] else min(len(wants), max(1, len(wants) // 2))
        # a shared page's id read and written and its count changed; the last pages' rows copied
        return dict(bytes=20 * case["batch"] + 16 * full + 2 * row * sum(wants[:got]), flops=0)
    held, sharers = _live(case)
    n, pages = sum(held), case["num_pages"]
    entries = n + len(sharers) * held[0]
    # table entries and counts in and out, the free list out, and the pages that lie behind the
    # first n, in expectation, copied
    moved = n * (pages - n) // pages
    return dict(bytes=8 * entries + 8 * pages + 4 * (pages - n) + 2 * row * case["page"] * moved,
                flops=0)


def exact(case, seed):
    if case["op"] != "chunk":
        return None
    dev = torch.device("cuda")
    s = _prepare(case, torch.Generator(device=dev).manual_seed(int(seed)), dev)
    d64 = torch.float64
    H, Hk, D, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    out, lse = s["out"].to(d64), s["lse"].to(d64)
    row = 0
    for b, (k0, n) in enumerate(zip(*s["steps"])):
        at = torch.arange(k0 + n, device=dev)
        pages, within = s["page_table"][b].long()[at // page], at % page
        for h in range(Hk if n else 0):
            keys, values = s["k_cache"][pages, within, h].to(d64), s["v_cache"][pages, within,
                                                                                h].to(d64)
            if s["k_scale"] is not None:
                keys, values = keys * s["k_scale"][h].to(d64), values * s["v_scale"][h].to(d64)
            for i in range(0, n, 1024):
                rows = torch.arange(i, min(n, i + 1024), device=dev)
                far = at[None] - (k0 + rows)[:, None]   # 0: the row's own position
                hidden = far > 0
                if case["window"]:
                    hidden |= far <= -case["window"]
                last = k0 + int(rows[-1]) + 1
                for j in range(h * H // Hk, (h + 1) * H // Hk):
                    x = s["q"][row + rows, j].to(d64) @ keys[:last].T * D ** -0.5
                    x[hidden[:, :last]] = -math.inf
                    z = torch.logsumexp(x, 1)
                    lse[row + rows, j] = z
                    out[row + rows, j] = torch.exp(x - z[:, None]) @ values[:last]
        row += n
    return dict(out=out, lse=lse)
