// The pages of a paged cache as a pool: forked to other sequences
// (mla_page_fork), given back (mla_page_release), brought together
// (mla_page_compact), and their rows copied in every cache tensor that the page
// table addresses (mla_page_copy).
//
// The first three only count and move 32-bit words, a few per sequence and
// page, so latency bounds them.  Each needs phases that see all of what the
// phase before wrote (counts changed before pages at zero are listed, say).  For
// tables of up to kWide entries they are one launch of one cluster of eight CTAs,
// whose hardware barrier takes a fraction of a launch's time; beyond, the phases
// that walk over table entries are launches of their own over the whole machine.
// Whatever is placed in order (pages of the free list, moves) is placed by
// exclusive sums over consecutive runs, so results never depend on the order in
// which threads arrive.
//
// Each lets the next launch of the stream take its place early, which waits for all
// of it before it reads: a launch's time less (us in a graph: 32 forks 11.7 -> 11.4,
// 32 sequences cut back 8.5 -> 8.2, 256 pages compacted 15.7 -> 15.1).  The copies
// do not, they fill the machine.

#include <cuda_runtime.h>

#include <climits>

#include "mla_internal.h"
#include "sm103_ptx.cuh"

namespace mla {

static __device__ int g_pool_status;

int pool_device_status(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_pool_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_pool_status, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

namespace {

constexpr int kThreads = 1024;
constexpr int kCtas = 8;  // the largest cluster that every GPU context may launch
constexpr int kAll = kThreads * kCtas;
constexpr int kRun = 4;  // entries of a table row a thread has on their way at once

__device__ __forceinline__ void bad_page() { atomicCAS(&g_pool_status, 0, kBadPageSite); }

// A run of `n` consecutive items for each thread of the cluster, or for each warp.
struct Run {
  int lo, hi;
  __device__ __forceinline__ Run(int n, int at, int of) {
    const int per = (int)(((long long)n + of - 1) / of);
    const long long a = (long long)at * per;
    lo = (int)min((long long)n, a);
    hi = (int)min((long long)n, a + per);
  }
};
__device__ __forceinline__ Run thread_run(int n, int rank) {
  return Run(n, rank * kThreads + (int)threadIdx.x, kAll);
}
// (whole lines: a warp's run is read 32 neighbours at a time)
__device__ __forceinline__ Run warp_run(int n, int rank) {
  Run r((n + 31) / 32, rank * (kThreads / 32) + (int)(threadIdx.x >> 5), kAll / 32);
  r.lo = min(n, r.lo * 32);
  r.hi = min(n, r.hi * 32);
  return r;
}

struct Scan {
  int warp[kThreads / 32];
  int total;  // of this CTA, read by the others
};

// Exclusive sum of x over the cluster's threads in order, and the sum of all.
// Holds one cluster barrier, so what any thread wrote to global memory before
// is seen by all behind it.  A Scan is used once in a kernel.
__device__ __forceinline__ int cluster_scan(Scan& s, int x, int rank, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) s.warp[warp] = sum;
  __syncthreads();
  int before = 0, mine = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int y = s.warp[w];
    if (w < warp) before += y;
    mine += y;
  }
  if (threadIdx.x == 0) s.total = mine;
  sm103::cluster_sync();
  all = 0;
  const uint32_t at = sm103::smem_u32(&s.total);
#pragma unroll
  for (int r = 0; r < kCtas; ++r) {
    int y;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(y) : "r"(sm103::mapa(at, r)) : "memory");
    if (r < rank) before += y;
    all += y;
  }
  return before + sum - x;
}

// Copies n words where the output is another array than the input, by all threads of
// the launch.
__device__ __forceinline__ void copy_words(const int32_t* from, int32_t* to, int n) {
  if (from == to) return;
  const int g = blockIdx.x * kThreads + threadIdx.x, quads = n / 4, all = gridDim.x * kThreads;
  for (int i = g; i < quads; i += all)
    reinterpret_cast<int4*>(to)[i] = reinterpret_cast<const int4*>(from)[i];
  for (int i = quads * 4 + g; i < n; i += all) to[i] = from[i];
}

struct FreeSpan {
  int first, end;
  __device__ __forceinline__ FreeSpan(const int32_t* span, int capacity) {
    first = min(max(span[0], 0), capacity);
    end = min(max(span[1], first), capacity);
  }
};

// Calls f for the table entries lo <= j < hi of every sequence, with range(b, lo, hi,
// aux) saying which: f gets kRun sequences b[], entries j[] (-1: none) and the
// sequences' aux[] to a thread at a time.  A warp takes the entries of a few
// sequences (as many as spread the batch over all warps, 32 at most) one after the
// other as if they were one row, so that single entries of many sequences fill its
// lanes, and several warps share a sequence where there are few.
template <typename Where, typename F>
__device__ __forceinline__ void for_entries(int batch, Where where, F f) {
  const int warps = gridDim.x * (kThreads / 32);
  const int lane = threadIdx.x & 31, warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int size = min(32, (batch + warps - 1) / warps), groups = (batch + size - 1) / size;
  const int share = max(1, warps / groups);  // warps that share a group
  for (int g = warp / share; g < groups; g += warps / share) {
    const int mine = g * size + lane;
    int lo = 0, hi = 0, x = 0;
    if (lane < size && mine < batch) where(mine, lo, hi, x);
    const int count = max(0, hi - lo);
    // (32 rows of a table of less than 2^31 entries in all)
    uint32_t upto = (uint32_t)count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t total = __shfl_sync(~0u, upto, 31);
    const int start = lo - (int)(upto - (uint32_t)count);  // entry = place + start
    for (uint32_t e0 = (uint32_t)(warp % share) * 32 * kRun; e0 < total;
         e0 += (uint32_t)share * 32 * kRun) {
      int b[kRun], j[kRun], aux[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const uint32_t e = e0 + i * 32 + lane;
        int owner = 0;  // the first lane whose sums pass e
#pragma unroll
        for (int step = 16; step > 0; step >>= 1)
          if (__shfl_sync(~0u, upto, owner + step - 1) <= e) owner += step;
        owner = min(owner, 31);
        const int first = __shfl_sync(~0u, start, owner);
        aux[i] = __shfl_sync(~0u, x, owner);
        b[i] = g * size + owner;
        j[i] = e < total ? (int)(e + (uint32_t)first) : -1;
      }
      f(b, j, aux);
    }
  }
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------

struct ForkParams {
  const int32_t *src, *lens, *held;
  int32_t* table;
  const int32_t *shares, *free_pages, *free_span;
  int32_t *lens_out, *held_out, *shares_out, *span_out, *missing, *move_src, *move_dst, *move_rows,
      *moves;
  int batch, width, page, num_pages, free_capacity;
  PageDiv div;
  // The source of an idle slot that takes another sequence's pages, or -1.
  __device__ __forceinline__ int source(int b) const {
    const int s = src[b];
    return s >= 0 && s < batch && held[b] <= 0 ? s : -1;
  }
  // Rows that a sequence has pages for, and its whole pages among them.
  __device__ __forceinline__ int rows(int s, int& full) const {
    const int h = min(max(held[s], 0), width);
    const int t = (int)min((long long)max(lens[s], 0), (long long)h * page);
    full = div(t);
    return t;
  }
};

// The whole pages of the forked slots.
__device__ __forceinline__ void fork_entries(const ForkParams& p) {
  for_entries(
      p.batch,
      [&](int b, int&, int& hi, int& s) {
        s = p.source(b);
        if (s >= 0) p.rows(s, hi);
      },
      [&](const int (&b)[kRun], const int (&j)[kRun], const int (&s)[kRun]) {
        int id[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (j[i] >= 0) id[i] = p.table[(long long)s[i] * p.width + j[i]];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          if (j[i] < 0) continue;
          p.table[(long long)b[i] * p.width + j[i]] = id[i];
          if (id[i] >= 0 && id[i] < p.num_pages) atomicAdd(p.shares_out + id[i], 1);
          else bad_page();
        }
      });
}

// One cluster.  `entries`: the whole pages as well, not in a launch behind this one.
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kThreads)
    page_fork_kernel(const ForkParams p, const bool entries) {
  __shared__ Scan s_scan;
  const int rank = (int)sm103::cluster_ctarank();
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  copy_words(p.shares, p.shares_out, p.num_pages);
  const Run run = thread_run(p.batch, rank);
  int wants = 0;
  for (int b = run.lo; b < run.hi; ++b) {
    const int s = p.source(b);
    if (s < 0) continue;
    int full;
    const int t = p.rows(s, full);
    if (t > full * p.page) ++wants;
  }
  const FreeSpan free(p.free_span, p.free_capacity);
  const int have = free.end - free.first;
  int all;
  int at = cluster_scan(s_scan, wants, rank, all);
  const int taken = min(all, have);
  for (int b = run.lo; b < run.hi; ++b) {
    const int s = p.source(b);
    if (s < 0) {
      p.lens_out[b] = p.lens[b];
      p.held_out[b] = p.held[b];
      continue;
    }
    int full;
    const int t = p.rows(s, full), rest = t - full * p.page;
    bool own = false;
    if (rest > 0) {
      own = at < have;
      if (own) {
        const int id = p.free_pages[free.first + at];
        const int from = p.table[(long long)s * p.width + full];
        // (listed all the same: the copy passes over such a move)
        if (id < 0 || id >= p.num_pages || from < 0 || from >= p.num_pages) bad_page();
        p.move_src[at] = from;
        p.move_dst[at] = id;
        p.move_rows[at] = rest;
        p.table[(long long)b * p.width + full] = id;
      }
      ++at;
    }
    p.lens_out[b] = rest > 0 && !own ? full * p.page : t;
    p.held_out[b] = full + (own ? 1 : 0);
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.span_out[0] = free.first + taken;
    p.span_out[1] = free.end;
    p.missing[0] = all - taken;
    p.moves[0] = taken;
  }
  if (entries) fork_entries(p);
  sm103::cluster_sync();  // no CTA ends while another reads its sum
}

__global__ void __launch_bounds__(kThreads) page_fork_entries_kernel(const ForkParams p) {
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  fork_entries(p);
}

// ---------------------------------------------------------------------------
// Release
// ---------------------------------------------------------------------------

struct ReleaseParams {
  const int32_t *kept, *held, *table, *shares;
  int32_t* free_pages;
  const int32_t* free_span;
  int32_t *held_out, *shares_out, *span_out, *released;
  int batch, width, page, num_pages, free_capacity;
  PageDiv div;
  __device__ __forceinline__ void range(int b, int& need, int& h) const {
    h = min(max(held[b], 0), width);
    const int k = kept[b];
    need = min(h, k > 0 ? div(k - 1) + 1 : 0);
  }
};

// A count holds the holders of a page beyond the first, so every drop takes one
// off and the pages that end below zero are the ones nobody holds any more.
__device__ __forceinline__ void release_entries(const ReleaseParams& p) {
  for_entries(
      p.batch, [&](int b, int& lo, int& hi, int&) { p.range(b, lo, hi); },
      [&](const int (&b)[kRun], const int (&j)[kRun], const int (&)[kRun]) {
        int id[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (j[i] >= 0) id[i] = p.table[(long long)b[i] * p.width + j[i]];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          if (j[i] < 0) continue;
          if (id[i] >= 0 && id[i] < p.num_pages) atomicSub(p.shares_out + id[i], 1);
          else bad_page();
        }
      });
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < p.batch; b += gridDim.x * kThreads) {
    int need, h;
    p.range(b, need, h);
    p.held_out[b] = need;
  }
}

// One cluster.  `entries`: the drops as well, not in launches ahead of this one.
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kThreads)
    page_release_kernel(const ReleaseParams p, const bool entries) {
  __shared__ Scan s_scan;
  const int rank = (int)sm103::cluster_ctarank(), lane = threadIdx.x & 31;
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  const FreeSpan free(p.free_span, p.free_capacity);
  if (entries) {
    if (p.shares != p.shares_out) {
      copy_words(p.shares, p.shares_out, p.num_pages);
      sm103::cluster_sync();
    }
    release_entries(p);
    sm103::cluster_sync();
  }
  const Run run = warp_run(p.num_pages, rank);
  auto freed = [&](int i) { return i + lane < run.hi && __ldcg(p.shares_out + i + lane) < 0; };
  int mine = 0;  // of this warp
#pragma unroll 8
  for (int i = run.lo; i < run.hi; i += 32) mine += __popc(__ballot_sync(~0u, freed(i)));
  int all;
  int at = cluster_scan(s_scan, lane == 0 ? mine : 0, rank, all);
  at = __shfl_sync(~0u, at, 0);
  // in front of the list as far as there is room, the others behind it
  const int front = min(all, free.first);
  constexpr int kAhead = 4;  // words of a lane on their way together
  for (int i0 = run.lo; i0 < run.hi && mine > 0; i0 += 32 * kAhead) {
    bool is[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) is[k] = freed(i0 + 32 * k);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + 32 * k + lane;
      const unsigned those = __ballot_sync(~0u, is[k]);
      if (is[k]) {
        const int n = at + __popc(those & ((1u << lane) - 1));
        const long long to = n < front ? free.first - front + n : (long long)free.end + n - front;
        if (to < p.free_capacity) p.free_pages[to] = i;
        p.shares_out[i] = 0;
      }
      at += __popc(those);
      mine -= __popc(those);
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.span_out[0] = free.first - front;
    p.span_out[1] = (int)min((long long)free.end + all - front, (long long)p.free_capacity);
    p.released[0] = all;
  }
  sm103::cluster_sync();
}

__global__ void __launch_bounds__(kThreads)
    copy_words_kernel(const int32_t* from, int32_t* to, const int n) {
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  copy_words(from, to, n);
}

__global__ void __launch_bounds__(kThreads) page_release_entries_kernel(const ReleaseParams p) {
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  release_entries(p);
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------

struct CompactParams {
  const int32_t *held, *table, *shares;
  int32_t *table_out, *shares_out, *free_pages, *span_out, *move_src, *move_dst, *moves;
  int32_t* mark;  // workspace [num_pages]: 1 for a live page; 1 + its place among the moves
  int batch, width, num_pages;
};

__device__ __forceinline__ int compact_held(const CompactParams& p, int b) {
  return min(max(p.held[b], 0), p.width);
}

__device__ __forceinline__ void compact_clear(const CompactParams& p) {
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.num_pages; i += gridDim.x * kThreads)
    p.mark[i] = 0;
}

__device__ __forceinline__ void compact_mark(const CompactParams& p) {
  for_entries(
      p.batch, [&](int b, int&, int& hi, int&) { hi = compact_held(p, b); },
      [&](const int (&b)[kRun], const int (&j)[kRun], const int (&)[kRun]) {
        int id[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (j[i] >= 0) id[i] = p.table[(long long)b[i] * p.width + j[i]];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          if (j[i] < 0) continue;
          if (id[i] >= 0 && id[i] < p.num_pages) p.mark[id[i]] = 1;
          else bad_page();
        }
      });
}

// With L = `total` live pages.
__device__ __forceinline__ void compact_table(const CompactParams& p, int total) {
  for_entries(
      p.batch,
      [&](int b, int&, int& hi, int& h) {
        hi = p.width;
        h = compact_held(p, b);
      },
      [&](const int (&b)[kRun], const int (&j)[kRun], const int (&h)[kRun]) {
        int id[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          id[i] = j[i] >= 0 && j[i] < h[i] ? p.table[(long long)b[i] * p.width + j[i]] : -1;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (id[i] >= total && id[i] < p.num_pages)
            id[i] = __ldcg(p.move_dst + __ldcg(p.mark + id[i]) - 1);
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (j[i] >= 0) p.table_out[(long long)b[i] * p.width + j[i]] = id[i];
      });
}

// One cluster.  The n-th live page at or beyond L goes to the n-th hole below L;
// sources and destinations have no page in common.  `entries`: the marks and the
// table as well, not in launches ahead of this one and behind it.
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kThreads)
    page_compact_kernel(const CompactParams p, const bool entries) {
  __shared__ Scan s_live, s_high;
  const int rank = (int)sm103::cluster_ctarank(), g = rank * kThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1;
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  if (entries) {
    compact_clear(p);
    sm103::cluster_sync();
    compact_mark(p);
    sm103::cluster_sync();
  }
  const Run run = warp_run(p.num_pages, rank);
  auto live = [&](int i) { return i + lane < run.hi && __ldcg(p.mark + i + lane) != 0; };
  int mine = 0;  // live pages of this warp
#pragma unroll 4
  for (int i = run.lo; i < run.hi; i += 32) mine += __popc(__ballot_sync(~0u, live(i)));
  int total;
  int before = cluster_scan(s_live, lane == 0 ? mine : 0, rank, total);
  before = __shfl_sync(~0u, before, 0);
  int high = 0;  // those at or beyond L
#pragma unroll 4
  for (int i = run.lo; i < run.hi; i += 32)
    high += __popc(__ballot_sync(~0u, live(i) && i + lane >= total));
  int moves;
  int from = cluster_scan(s_high, lane == 0 ? high : 0, rank, moves);
  from = __shfl_sync(~0u, from, 0);
  for (int i = run.lo; i < run.hi; i += 32) {
    const bool is = live(i);
    const unsigned those = __ballot_sync(~0u, is);
    const unsigned up = __ballot_sync(~0u, is && i + lane >= total);
    if (!is && i + lane < min(total, run.hi)) {
      p.move_dst[i + lane - before - __popc(those & below)] = i + lane;
    } else if (is && i + lane >= total) {
      const int n = from + __popc(up & below);
      p.move_src[n] = i + lane;
      p.mark[i + lane] = n + 1;
    }
    before += __popc(those);
    from += __popc(up);
  }
  sm103::cluster_sync();
  for (int i = g; i < moves; i += kAll) {
    const int a = __ldcg(p.move_src + i), z = __ldcg(p.move_dst + i);
    p.shares_out[z] = p.shares[a];
    p.shares_out[a] = 0;
  }
  // (the marks below L are still 0 and 1; a hole's count is written above)
  for (int i = g; i < p.num_pages; i += kAll) {
    const bool is_live = __ldcg(p.mark + i) != 0;
    if (i < total) {
      if (is_live) p.shares_out[i] = p.shares[i];
    } else {
      if (!is_live) p.shares_out[i] = 0;
      p.free_pages[i - total] = i;
    }
  }
  if (g == 0) {
    p.span_out[0] = 0;
    p.span_out[1] = p.num_pages - total;
    p.moves[0] = moves;
  }
  if (entries) compact_table(p, total);
  sm103::cluster_sync();
}

__global__ void __launch_bounds__(kThreads) page_compact_clear_kernel(const CompactParams p) {
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  compact_clear(p);
}
__global__ void __launch_bounds__(kThreads) page_compact_mark_kernel(const CompactParams p) {
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  compact_mark(p);
}
__global__ void __launch_bounds__(kThreads) page_compact_table_kernel(const CompactParams p) {
  sm103::pdl_wait();
  sm103::pdl_launch_dependents();
  compact_table(p, p.num_pages - p.span_out[1]);
}

// ---------------------------------------------------------------------------
// Copy
// ---------------------------------------------------------------------------
//
// Bound by memory: every byte is read and written once.  A CTA takes 32 KB of
// one page of one tensor at a time, eight 16-byte vectors a thread on their way
// together, and CTAs walk over (page, tensor, piece) with a grid that fills the
// machine, so that few large pages and many small ones both spread evenly.

constexpr int kCopyThreads = 256, kCopyVecs = 8;
constexpr int kPiece = kCopyThreads * kCopyVecs;
constexpr int kViews = 128;

struct CopyView {
  char* base;
  int64_t page_stride, row_stride, head_stride;
  int heads, vecs;  // runs of a row, 16-byte vectors of a run
};

struct CopyParams {
  CopyView view[kViews];
  int piece[kViews + 1];  // pieces of a whole page before each view
  const int32_t *src, *dst, *rows, *moves;
  int views, capacity, page, num_pages;
};

__global__ void __launch_bounds__(kCopyThreads)
    page_copy_kernel(const __grid_constant__ CopyParams p) {
  sm103::pdl_wait();
  int n = p.capacity;
  if (p.moves) n = min(max(p.moves[0], 0), n);
  const int pieces = p.piece[p.views];
  const long long units = (long long)n * pieces;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int m = (int)(u / pieces), q = (int)(u - (long long)m * pieces);
    int a = 0, z = p.views;
    while (z - a > 1) {
      const int mid = (a + z) >> 1;
      if (p.piece[mid] <= q) a = mid; else z = mid;
    }
    const CopyView& v = p.view[a];
    const int from = p.src[m], to = p.dst[m];
    const int rows = p.rows ? min(max(p.rows[m], 0), p.page) : p.page;
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages) {
      if (q == 0 && threadIdx.x == 0) bad_page();
      continue;
    }
    // vector x of the page's copied part: run, row, vector of the row
    const int per_head = rows * v.vecs, most = v.heads * per_head;
    const int x0 = (q - p.piece[a]) * kPiece + threadIdx.x;
    const bool dense = v.row_stride == (int64_t)v.vecs * 16;
    auto offset = [&](int x) -> int64_t {
      const int h = v.heads == 1 ? 0 : x / per_head, y = x - h * per_head;
      if (dense) return h * v.head_stride + (int64_t)y * 16;
      const int r = y / v.vecs;
      return h * v.head_stride + r * v.row_stride + (int64_t)(y - r * v.vecs) * 16;
    };
    const char* s = v.base + from * v.page_stride;
    char* d = v.base + to * v.page_stride;
    uint4 w[kCopyVecs];
    int64_t off[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
      const int x = x0 + i * kCopyThreads;
      if (x < most) {
        off[i] = offset(x);
        w[i] = *reinterpret_cast<const uint4*>(s + off[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (x0 + i * kCopyThreads < most) *reinterpret_cast<uint4*>(d + off[i]) = w[i];
  }
}

// ---------------------------------------------------------------------------
// Checks
// ---------------------------------------------------------------------------

struct Named {
  const void* p;
  const char* name;
};

mla_status_t pointers_ok(const char* what, const Named* list, int n) {
  for (int i = 0; i < n; ++i) {
    if (list[i].p == nullptr || ((uintptr_t)list[i].p & 15u)) {
      set_error("%s: %s is NULL or not 16-byte aligned", what, list[i].name);
      return MLA_ERR_INVALID_ARG;
    }
  }
  return MLA_OK;
}

struct Range {
  uintptr_t lo, hi;
  Range(const void* p, int64_t words) : lo((uintptr_t)p), hi(lo + (uintptr_t)words * 4) {}
  bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

// Outputs apart from the inputs and from one another; pair (out_same, in_same)
// may be one array.
mla_status_t apart(const char* what, const Range* in, int ni, const Range* out, int no,
                   const int (*same)[2], int ns) {
  for (int i = 0; i < no; ++i) {
    bool bad = false;
    for (int j = 0; j < ni; ++j) {
      bool pair = false;
      for (int k = 0; k < ns; ++k)
        pair = pair || (same[k][0] == i && same[k][1] == j && out[i].lo == in[j].lo);
      bad = bad || (!pair && out[i].meets(in[j]));
    }
    for (int j = 0; j < i; ++j) bad = bad || out[i].meets(out[j]);
    if (bad) {
      set_error("%s: an output overlaps another buffer of the call", what);
      return MLA_ERR_INVALID_ARG;
    }
  }
  return MLA_OK;
}

mla_status_t sizes_ok(const char* what, int batch, int width, int page, int num_pages) {
  if (batch < 1 || batch > 65535 || width < 1 || page < 1 || num_pages < 1 ||
      num_pages > (1 << 30) || (int64_t)batch * width > INT_MAX) {
    set_error("%s: need 1 <= batch <= 65535, max_pages_per_seq and page_size >= 1, num_pages in "
              "[1, 2^30], batch * max_pages_per_seq < 2^31 (batch=%d max_pages=%d page_size=%d "
              "num_pages=%d)",
              what, batch, width, page, num_pages);
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

// Table entries beyond which a walk over them is a launch over the whole machine: eight
// CTAs take about 4000 entries a microsecond, a launch costs two.
constexpr int64_t kWide = 32768;

bool wide(int batch, int width) { return (int64_t)batch * width > kWide; }

dim3 whole_machine() { return dim3((unsigned)device_sm_count() * 2); }

mla_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  set_error("CUDA error %d (%s)", (int)e, cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_page_fork(
    const int32_t* src_of, const int32_t* cache_lens, const int32_t* held_pages, int32_t batch,
    int32_t* page_table, int32_t max_pages_per_seq, int32_t page_size, int32_t num_pages,
    const int32_t* shares, const int32_t* free_pages, int32_t free_capacity,
    const int32_t* free_span, int32_t* cache_lens_out, int32_t* held_pages_out,
    int32_t* shares_out, int32_t* free_span_out, int32_t* missing_out, int32_t* move_src_out,
    int32_t* move_dst_out, int32_t* move_rows_out, int32_t* moves_out, void* stream) {
  const char* what = "page fork";
  mla_status_t st = sizes_ok(what, batch, max_pages_per_seq, page_size, num_pages);
  if (st != MLA_OK) return st;
  if (free_capacity < 1) {
    set_error("%s: free_capacity %d is below 1", what, free_capacity);
    return MLA_ERR_INVALID_ARG;
  }
  const Named ptrs[] = {{src_of, "src_of"}, {cache_lens, "cache_lens"},
                        {held_pages, "held_pages"}, {page_table, "page_table"},
                        {shares, "shares"}, {free_pages, "free_pages"},
                        {free_span, "free_span"}, {cache_lens_out, "cache_lens_out"},
                        {held_pages_out, "held_pages_out"}, {shares_out, "shares_out"},
                        {free_span_out, "free_span_out"}, {missing_out, "missing_out"},
                        {move_src_out, "move_src_out"}, {move_dst_out, "move_dst_out"},
                        {move_rows_out, "move_rows_out"}, {moves_out, "moves_out"}};
  st = pointers_ok(what, ptrs, 16);
  if (st != MLA_OK) return st;
  const int B = batch;
  const Range in[] = {{src_of, B}, {cache_lens, B}, {held_pages, B}, {shares, num_pages},
                      {free_pages, free_capacity}, {free_span, 2}};
  const Range out[] = {{page_table, (int64_t)B * max_pages_per_seq}, {cache_lens_out, B},
                       {held_pages_out, B}, {shares_out, num_pages}, {free_span_out, 2},
                       {missing_out, 1}, {move_src_out, B}, {move_dst_out, B},
                       {move_rows_out, B}, {moves_out, 1}};
  const int same[][2] = {{3, 3}};
  st = apart(what, in, 6, out, 10, same, 1);
  if (st != MLA_OK) return st;
  ForkParams p;
  p.src = src_of;
  p.lens = cache_lens;
  p.held = held_pages;
  p.table = page_table;
  p.shares = shares;
  p.free_pages = free_pages;
  p.free_span = free_span;
  p.lens_out = cache_lens_out;
  p.held_out = held_pages_out;
  p.shares_out = shares_out;
  p.span_out = free_span_out;
  p.missing = missing_out;
  p.move_src = move_src_out;
  p.move_dst = move_dst_out;
  p.move_rows = move_rows_out;
  p.moves = moves_out;
  p.batch = batch;
  p.width = max_pages_per_seq;
  p.page = page_size;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  p.div = PageDiv(page_size);
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("page_fork", s);
  const bool split = wide(batch, max_pages_per_seq);
  cudaError_t e =
      launch_dependent(page_fork_kernel, dim3(kCtas), dim3(kThreads), 0, s, p, !split);
  if (e == cudaSuccess && split)
    e = launch_dependent(page_fork_entries_kernel, whole_machine(), dim3(kThreads), 0, s, p);
  return launched(e);
}

extern "C" mla_status_t mla_page_release(
    const int32_t* kept_lens, const int32_t* held_pages, int32_t batch, const int32_t* page_table,
    int32_t max_pages_per_seq, int32_t page_size, int32_t num_pages, const int32_t* shares,
    int32_t* free_pages, int32_t free_capacity, const int32_t* free_span, int32_t* held_pages_out,
    int32_t* shares_out, int32_t* free_span_out, int32_t* released_out, void* stream) {
  const char* what = "page release";
  mla_status_t st = sizes_ok(what, batch, max_pages_per_seq, page_size, num_pages);
  if (st != MLA_OK) return st;
  if (free_capacity < num_pages) {
    set_error("%s: a free list of %d entries may be too short for %d pages", what, free_capacity,
              num_pages);
    return MLA_ERR_INVALID_ARG;
  }
  const Named ptrs[] = {{kept_lens, "kept_lens"}, {held_pages, "held_pages"},
                        {page_table, "page_table"}, {shares, "shares"},
                        {free_pages, "free_pages"}, {free_span, "free_span"},
                        {held_pages_out, "held_pages_out"}, {shares_out, "shares_out"},
                        {free_span_out, "free_span_out"}, {released_out, "released_out"}};
  st = pointers_ok(what, ptrs, 10);
  if (st != MLA_OK) return st;
  const int B = batch;
  const Range in[] = {{kept_lens, B}, {held_pages, B},
                      {page_table, (int64_t)B * max_pages_per_seq}, {shares, num_pages},
                      {free_span, 2}};
  const Range out[] = {{free_pages, free_capacity}, {held_pages_out, B}, {shares_out, num_pages},
                       {free_span_out, 2}, {released_out, 1}};
  const int same[][2] = {{2, 3}};
  st = apart(what, in, 5, out, 5, same, 1);
  if (st != MLA_OK) return st;
  ReleaseParams p;
  p.kept = kept_lens;
  p.held = held_pages;
  p.table = page_table;
  p.shares = shares;
  p.free_pages = free_pages;
  p.free_span = free_span;
  p.held_out = held_pages_out;
  p.shares_out = shares_out;
  p.span_out = free_span_out;
  p.released = released_out;
  p.batch = batch;
  p.width = max_pages_per_seq;
  p.page = page_size;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  p.div = PageDiv(page_size);
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("page_release", s);
  const bool split = wide(batch, max_pages_per_seq);
  cudaError_t e = cudaSuccess;
  if (split && shares != shares_out)
    e = launch_dependent(copy_words_kernel, whole_machine(), dim3(kThreads), 0, s, shares,
                         shares_out, num_pages);
  if (e == cudaSuccess && split)
    e = launch_dependent(page_release_entries_kernel, whole_machine(), dim3(kThreads), 0, s, p);
  if (e == cudaSuccess)
    e = launch_dependent(page_release_kernel, dim3(kCtas), dim3(kThreads), 0, s, p, !split);
  return launched(e);
}

extern "C" mla_status_t mla_page_compact_workspace_bytes(int32_t num_pages, size_t* bytes) {
  if (bytes == nullptr || num_pages < 1) {
    set_error("page compact: need num_pages >= 1 and a place for the bytes (num_pages=%d)",
              num_pages);
    return MLA_ERR_INVALID_ARG;
  }
  *bytes = ((size_t)num_pages * 4 + 255) & ~(size_t)255;
  return MLA_OK;
}

extern "C" mla_status_t mla_page_compact(
    const int32_t* held_pages, int32_t batch, const int32_t* page_table, int32_t max_pages_per_seq,
    int32_t num_pages, const int32_t* shares, int32_t* page_table_out, int32_t* shares_out,
    int32_t* free_pages, int32_t free_capacity, int32_t* free_span_out, int32_t* move_src_out,
    int32_t* move_dst_out, int32_t* moves_out, void* workspace, size_t workspace_bytes,
    void* stream) {
  const char* what = "page compact";
  mla_status_t st = sizes_ok(what, batch, max_pages_per_seq, 1, num_pages);
  if (st != MLA_OK) return st;
  if (free_capacity < num_pages) {
    set_error("%s: a free list of %d entries may be too short for %d pages", what, free_capacity,
              num_pages);
    return MLA_ERR_INVALID_ARG;
  }
  const Named ptrs[] = {{held_pages, "held_pages"}, {page_table, "page_table"},
                        {shares, "shares"}, {page_table_out, "page_table_out"},
                        {shares_out, "shares_out"}, {free_pages, "free_pages"},
                        {free_span_out, "free_span_out"}, {move_src_out, "move_src_out"},
                        {move_dst_out, "move_dst_out"}, {moves_out, "moves_out"}};
  st = pointers_ok(what, ptrs, 10);
  if (st != MLA_OK) return st;
  size_t need = 0;
  st = mla_page_compact_workspace_bytes(num_pages, &need);
  if (st != MLA_OK) return st;
  if (workspace == nullptr || workspace_bytes < need) {
    set_error("workspace of %zu bytes is smaller than the %zu this call needs", workspace_bytes,
              need);
    return MLA_ERR_WORKSPACE;
  }
  if ((uintptr_t)workspace & 255u) {
    set_error("workspace is not 256-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  const int B = batch;
  const int64_t entries = (int64_t)B * max_pages_per_seq, most = num_pages / 2;
  const Range in[] = {{held_pages, B}, {page_table, entries}, {shares, num_pages}};
  const Range out[] = {{page_table_out, entries}, {shares_out, num_pages},
                       {free_pages, free_capacity}, {free_span_out, 2}, {move_src_out, most},
                       {move_dst_out, most}, {moves_out, 1}, {workspace, (int64_t)need / 4}};
  const int same[][2] = {{0, 1}, {1, 2}};
  st = apart(what, in, 3, out, 8, same, 2);
  if (st != MLA_OK) return st;
  CompactParams p;
  p.held = held_pages;
  p.table = page_table;
  p.shares = shares;
  p.table_out = page_table_out;
  p.shares_out = shares_out;
  p.free_pages = free_pages;
  p.span_out = free_span_out;
  p.move_src = move_src_out;
  p.move_dst = move_dst_out;
  p.moves = moves_out;
  p.mark = (int32_t*)workspace;
  p.batch = batch;
  p.width = max_pages_per_seq;
  p.num_pages = num_pages;
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("page_compact", s);
  const bool split = wide(batch, max_pages_per_seq);
  const dim3 all = whole_machine();
  cudaError_t e = cudaSuccess;
  if (split) e = launch_dependent(page_compact_clear_kernel, all, dim3(kThreads), 0, s, p);
  if (e == cudaSuccess && split)
    e = launch_dependent(page_compact_mark_kernel, all, dim3(kThreads), 0, s, p);
  if (e == cudaSuccess)
    e = launch_dependent(page_compact_kernel, dim3(kCtas), dim3(kThreads), 0, s, p, !split);
  if (e == cudaSuccess && split)
    e = launch_dependent(page_compact_table_kernel, all, dim3(kThreads), 0, s, p);
  return launched(e);
}

extern "C" mla_status_t mla_page_copy(const mla_page_view_t* views, int32_t num_views,
                                      int32_t page_size, int32_t num_pages,
                                      const int32_t* move_src, const int32_t* move_dst,
                                      const int32_t* move_rows, const int32_t* moves,
                                      int32_t capacity, void* stream) {
  const char* what = "page copy";
  if (views == nullptr || num_views < 1 || num_views > kViews || page_size < 1 || num_pages < 1 ||
      capacity < 0) {
    set_error("%s: need 1 to %d views, page_size and num_pages >= 1, capacity >= 0 (views=%d "
              "page_size=%d num_pages=%d capacity=%d)", what, kViews, num_views, page_size,
              num_pages, capacity);
    return MLA_ERR_INVALID_ARG;
  }
  CopyParams p;
  int64_t pieces = 0;
  for (int i = 0; i < num_views; ++i) {
    const mla_page_view_t& v = views[i];
    if (v.base == nullptr || ((uintptr_t)v.base & 15u)) {
      set_error("%s: the base of view %d is NULL or not 16-byte aligned", what, i);
      return MLA_ERR_INVALID_ARG;
    }
    const int64_t strides[3] = {v.page_stride, v.row_stride, v.head_stride};
    const int64_t extent[3] = {num_pages, page_size, v.heads};
    bool bad = v.heads < 1 || v.width < 16 || v.width % 16 != 0;
    for (int k = 0; k < 3 && !bad; ++k)
      bad = strides[k] < 0 || strides[k] % 16 != 0 || (extent[k] > 1 && strides[k] < v.width);
    if (bad) {
      set_error("%s: view %d needs heads >= 1, a width and strides of whole 16 bytes, the "
                "strides at least the width (heads=%d width=%d page %lld row %lld head %lld)",
                what, i, v.heads, v.width, (long long)v.page_stride, (long long)v.row_stride,
                (long long)v.head_stride);
      return MLA_ERR_INVALID_ARG;
    }
    // heads side by side are one run of bytes, and so are whole pages of them
    CopyView& c = p.view[i];
    const bool dense = v.heads == 1 || v.head_stride == v.width;
    const int64_t run = dense ? (int64_t)v.heads * v.width : v.width;
    const int64_t vecs = (int64_t)page_size * v.heads * (v.width / 16);
    if (vecs > INT_MAX - kPiece || run / 16 > INT_MAX) {
      set_error("%s: a page of view %d is larger than 32 GB", what, i);
      return MLA_ERR_UNSUPPORTED;
    }
    c.base = (char*)v.base;
    c.page_stride = v.page_stride;
    c.row_stride = page_size > 1 ? v.row_stride : run;
    c.head_stride = v.head_stride;
    c.heads = dense ? 1 : v.heads;
    c.vecs = (int)(run / 16);
    p.piece[i] = (int)pieces;
    pieces += (vecs + kPiece - 1) / kPiece;
    if (pieces > INT_MAX) {
      set_error("%s: the views' pages are too large for one call", what);
      return MLA_ERR_UNSUPPORTED;
    }
  }
  p.piece[num_views] = (int)pieces;
  if (capacity == 0) return MLA_OK;
  const Named ptrs[] = {{move_src, "move_src"}, {move_dst, "move_dst"}};
  mla_status_t st = pointers_ok(what, ptrs, 2);
  if (st != MLA_OK) return st;
  if (((uintptr_t)move_rows | (uintptr_t)moves) & 15u) {
    set_error("%s: move_rows or moves is not 16-byte aligned", what);
    return MLA_ERR_INVALID_ARG;
  }
  p.src = move_src;
  p.dst = move_dst;
  p.rows = move_rows;
  p.moves = moves;
  p.views = num_views;
  p.capacity = capacity;
  p.page = page_size;
  p.num_pages = num_pages;
  const int64_t units = (int64_t)capacity * pieces;
  const int64_t most = (int64_t)device_sm_count() * 6;
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("page_copy", s);
  return launched(launch_dependent(page_copy_kernel, dim3((unsigned)(units < most ? units : most)),
                                   dim3(kCopyThreads), 0, s, p));
}
