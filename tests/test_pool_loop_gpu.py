"""The page pool and the attentions over it together, as a serving loop runs them: prompts in
chunks, samples forked off a prompt, draft rows verified and partly rejected, sequences that end,
the pool brought together; every step's attention against one over plain per-sequence histories."""

import numpy as np
import pytest
import torch

from oracle import page_pool as O
from mla_attention_speculative_gb300 import binding as B
from mla_attention_speculative_gb300 import build_lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    B.lib()
    yield
    torch.cuda.synchronize()
    B.mla_device_status()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Loop:
    """Slots over a shared pool, with two layers' caches; histories are kept beside, per slot."""

    def __init__(self, slots, page, pages, dtype, cache, seed):
        self.B, self.page, self.pages, self.dtype = slots, page, pages, dtype
        self.H, self.Hk, self.D = 8, 2, 64
        self.gen = torch.Generator(DEV).manual_seed(seed)
        z = lambda: torch.zeros(pages, page, self.Hk, self.D, device=DEV).to(cache)  # noqa: E731
        self.caches = [z() for _ in range(4)]
        self.scale = torch.full((self.Hk,), 0.02, device=DEV) if cache == E4M3 else None
        self.table = i32(np.full((slots, 40), -1))
        self.lens, self.held = i32([0] * slots), i32([0] * slots)
        self.shares = i32([0] * pages)
        self.free = torch.randperm(pages, generator=self.gen, device=DEV).to(torch.int32)
        self.span = i32([0, pages])
        self.hist = [[[] for _ in range(slots)] for _ in range(4)]   # [cache][slot] rows

    def step(self, new, kept=None):
        """`new` rows per slot behind `kept` ones: appended, then attended to."""
        kept = self.lens if kept is None else kept
        st = B.mla_page_step(kept, i32(new), self.held, self.table, self.free, self.span,
                             self.page, self.pages, sum(new) + 3)
        assert st.missing.item() == 0
        k_list = kept.tolist()
        for layer in range(2):
            kc, vc = self.caches[2 * layer:2 * layer + 2]
            q, k, v = (torch.randn(sum(new) + 3, h, self.D, generator=self.gen,
                                   device=DEV).to(self.dtype) for h in (self.H, self.Hk, self.Hk))
            B.mla_append_kv(None, k, v, None, st.positions, st.slots, kc, vc,
                            k_scale=self.scale, v_scale=self.scale)
            row = 0
            for b, n in enumerate(new):
                for c, x in ((2 * layer, k), (2 * layer + 1, v)):
                    h = self.hist[c][b]
                    del h[k_list[b]:]
                    y = x[row:row + n].float()
                    if self.scale is not None:
                        y = (y / 0.02).to(E4M3).float() * 0.02
                    h.extend(y)
                row += n
            out, lse = B.mla_chunk_attention(q, kc, vc, kept, st.cache_lens, st.row_start,
                                             self.table, k_scale=self.scale, v_scale=self.scale,
                                             return_lse=True)
            torch.cuda.synchronize()
            self.check(q, out, lse, new, k_list, layer)
        self.lens, self.held, self.span = st.cache_lens, st.held_pages, st.free_span

    def check(self, q, out, lse, new, kept, layer):
        row = 0
        for b, n in enumerate(new):
            if n:
                k, v = (torch.stack(self.hist[2 * layer + i][b]).double() for i in range(2))
                x = q[row:row + n].double().view(n, self.Hk, -1, self.D)
                s = torch.einsum("nkgd,tkd->nkgt", x, k) * self.D ** -0.5
                hidden = torch.arange(len(k), device=DEV) > (
                    kept[b] + torch.arange(n, device=DEV))[:, None]
                s = s.masked_fill(hidden[:, None, None], -float("inf"))
                p = torch.softmax(s, -1)
                want = torch.einsum("nkgt,tkd->nkgd", p, v).reshape(n, self.H, self.D)
                vabs = torch.einsum("nkgt,tkd->nkgd", p, v.abs()).reshape(n, self.H, self.D)
                # roundings: the output's and the weights' (both at most 2^-8), the e4m3
                # history above (2^-22), sums
                u = 2.0 ** -7 if self.dtype == BF16 else 2.0 ** -18
                tol = u * 2 * vabs + 1e-6
                bad = (out[row:row + n].double() - want).abs() > tol
                assert not bad.any(), (b, n, kept[b], layer)
                z = torch.logsumexp(s, -1).reshape(n, self.H)
                assert ((lse[row:row + n] - z).abs() < 1e-4 + 1e-5 * z.abs()).all()
            row += n

    def fork(self, src):
        st = B.mla_page_fork(i32(src), self.lens, self.held, self.table, self.shares, self.free,
                             self.span, self.page)
        B.mla_page_copy(self.caches, st.move_src, st.move_dst, st.moves, st.move_rows)
        assert st.missing.item() == 0
        held = self.held.tolist()
        for b, s in enumerate(src):
            if s >= 0 and held[b] == 0:
                for h in self.hist:
                    h[b] = list(h[s])
        self.lens, self.held, self.shares, self.span = (st.cache_lens, st.held_pages, st.shares,
                                                        st.free_span)

    def release(self, kept):
        kept = i32(kept)
        st = B.mla_page_release(kept, self.held, self.table, self.shares, self.free, self.span,
                                self.page)
        self.lens = torch.minimum(self.lens, kept)
        self.held, self.shares, self.span = st.held_pages, st.shares, st.free_span
        for b, k in enumerate(self.lens.tolist()):
            for h in self.hist:
                del h[b][k:]

    def compact(self):
        st = B.mla_page_compact(self.held, self.table, self.shares, self.free)
        B.mla_page_copy(self.caches, st.move_src, st.move_dst, st.moves)
        self.table, self.shares, self.span = st.page_table, st.shares, st.free_span
        return st.moves.item()

    def consistent(self):
        """Every page is on the free list once, or held by 1 + shares table rows."""
        held, table = self.held.tolist(), self.table.cpu().numpy()
        count = np.zeros(self.pages, int)
        for b in range(self.B):
            for j in range(held[b]):
                count[table[b, j]] += 1
        span = self.span.tolist()
        free = self.free.tolist()[span[0]:span[1]]
        assert len(set(free)) == len(free) and not count[free].any()
        assert len(free) + (count > 0).sum() == self.pages
        shares = self.shares.cpu().numpy()
        assert np.array_equal(shares[count > 0], count[count > 0] - 1)
        assert not shares[count == 0].any()


@pytest.mark.parametrize("dtype,cache,page", [(BF16, BF16, 16), (BF16, E4M3, 8), (FP32, FP32, 4),
                                              (BF16, BF16, 5)])
def test_serving_loop(dtype, cache, page):
    s = Loop(6, page, 400 // page * 2, dtype, cache, seed=page)
    s.step([30, 0, 17, 0, 0, 0])               # prompts in chunks
    s.step([41, 0, 3, 0, 0, 0])
    s.consistent()
    s.fork([-1, 0, -1, 0, 0, 2])               # samples of slots 0 and 2
    s.consistent()
    s.step([1, 1, 1, 1, 1, 1])                 # they part
    s.step([4, 4, 4, 4, 4, 4])                 # draft rows ...
    lens = s.lens.tolist()
    kept = [lens[0] - 3, lens[1], lens[2] - 4, lens[3] - 1, lens[4] - 2, lens[5]]
    s.release(kept)                            # ... some rejected, their pages back
    s.consistent()
    s.step([2, 3, 4, 1, 2, 0])
    s.release([0, s.lens.tolist()[1], s.lens.tolist()[2], 0, s.lens.tolist()[4], 0])   # some end
    s.consistent()
    moves = s.compact()
    assert moves > 0
    s.consistent()
    s.step([0, 2, 5, 0, 3, 0])
    s.fork([1, -1, -1, 2, -1, 4])              # and slots are used again
    s.consistent()
    s.step([9, 1, 1, 9, 1, 9])
    # a sequence cut back into a page that it shares is forked, and its old slot released
    if s.page < 16:
        cut = s.lens.tolist()[0] // s.page * s.page - 2
        s.release([s.lens.tolist()[0], 0, 0, 0, 0, 0])
        s.consistent()
        s.fork([-1, 0, -1, -1, -1, -1])
        lens = s.lens.tolist()
        s.release([lens[0], cut] + [0] * 4)
        s.fork([-1, -1, 1, -1, -1, -1])
        s.release([lens[0], 0, cut, 0, 0, 0])
        s.consistent()
        s.step([3, 0, 6, 0, 0, 0])
    s.release([0] * 6)
    s.consistent()
    span = s.span.tolist()
    assert span[1] - span[0] == s.pages
    B.mla_device_status()


def test_pool_calls_in_a_graph():
    """Fork, copy and release captured once and replayed while lengths and tables change."""
    page, P, slots = 8, 64, 6
    g = np.random.default_rng(1)
    cache = torch.randn(P, page, 2, 64, device=DEV).to(BF16)
    src, lens, held = i32([-1] * slots), i32([0] * slots), i32([0] * slots)
    table, shares, free, span = i32(np.zeros((slots, 9))), i32([0] * P), i32([-1] * P), i32([0, 0])
    kept = i32([0] * slots)
    fork = B.PreparedPageFork(src, lens, held, table, shares, free, span, page)
    copy = B.PreparedPageCopy([cache], fork.out.move_src, fork.out.move_dst, fork.out.moves,
                              fork.out.move_rows)
    back = B.PreparedPageRelease(kept, fork.out.held_pages, table, fork.out.shares, free,
                                 fork.out.free_span, page)
    graph = torch.cuda.CUDAGraph()
    for c in (fork, copy, back):
        c.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for c in (fork, copy, back):
            c.run()
    for trial in range(5):
        ids = g.permutation(P)
        n = [0 if b % 2 else int(g.integers(1, 60)) for b in range(slots)]
        used = [-(-x // page) for x in n]
        t = np.full((slots, 9), -1)
        at = 0
        for b in range(slots):
            t[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
        f = np.full(P, -1)
        f[5:5 + P - at - 5] = ids[at + 5:]
        sp = [5, 5 + P - at - 5]
        so = [int(g.integers(-1, slots)) for _ in range(slots)]
        for x, y in ((src, so), (lens, n), (held, used), (table, t), (free, f), (span, sp)):
            x.copy_(i32(y))
        before = cache.clone()
        w = O.page_fork(so, n, used, t, [0] * P, f, sp, page)
        keep = [max(0, x - int(g.integers(0, 20))) for x in w[1]]
        kept.copy_(i32(keep))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(table.cpu().numpy(), w[0]) and fork.out.cache_lens.tolist() == w[1]
        assert torch.equal(cache.cpu(), torch.as_tensor(O.page_copy(
            before.view(torch.int16).cpu().numpy(), w[6], page)).view(BF16))
        r = O.page_release(keep, w[2], w[0], w[3], f, w[4], page)
        assert back.out.held_pages.tolist() == r[0] and free.tolist() == r[2]
        assert np.array_equal(back.out.shares.cpu().numpy(), r[1])
        assert back.out.free_span.tolist() == r[3]
    B.mla_device_status()


def test_pool_calls_on_other_streams():
    page, P = 8, 64
    cases = []
    for i in range(3):
        g = np.random.default_rng(i)
        ids = g.permutation(P)
        t = np.full((4, 8), -1)
        t[0, :5], t[2, :3] = ids[:5], ids[5:8]
        f = np.concatenate([ids[8:], [-1] * 8])
        cases.append(([-1, 0, -1, 2], [37 + i, 0, 17, 0], [5, 0, 3, 0], t, [0] * P, f, [0, P - 8]))
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for c, s in zip(cases, streams):
        a = [i32(x) for x in c]
        torch.cuda.synchronize()
        outs.append((a, B.mla_page_fork(*a[:3], a[3], a[4], a[5], a[6], page,
                                        stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for c, (a, o) in zip(cases, outs):
        w = O.page_fork(*c, page)
        assert np.array_equal(a[3].cpu().numpy(), w[0]) and o.cache_lens.tolist() == w[1]
        assert np.array_equal(o.shares.cpu().numpy(), w[3])
