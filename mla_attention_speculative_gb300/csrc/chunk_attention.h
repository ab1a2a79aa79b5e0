// Interface between the chunk attention's entry point, its planner and its
// kernels.
//
// The queries of one sequence and key/value head are taken as rows: row r is
// token r / group, head r % group of its group, so that few tokens and many
// heads fill a tile as well as many tokens and few heads.  A unit is a tile of
// `bm` such rows; it costs `unit_cost` plus one per tile of `bn` cached positions
// that any of its rows sees.  All units, in order of sequence, key/value head
// and tile, laid end to end are cut into equal shares, one per CTA, so a unit
// may fall into several shares: each leaves a part, and the join adds them up.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "mla_internal.h"

namespace mla {
namespace chunk {

constexpr int kMaxCtas = 512;
// What a unit costs besides its tiles, in tiles: its queries, its first and last
// waits, its edge tiles and its outputs (us at 3 / 6 / 8 / 11 / 14 on tensor cores:
// a prompt of 8192 rows 415 / 395 / 400 / 409 / 421, prompts and steps over an e4m3
// cache 817 / 756 / 745 / 742 / 754, 16 steps of 1 to 8 rows 39.1 / 35.3 / 35.4 / 36.8 /
// 39.1; a window of fp32 on CUDA cores 64.1 at 1, 64.2 at 2, 64.2 at 3, 75.2 at 4).
// Those are 128 wide in pages of 64.  One number serves all widths and feeds, and at 3 / 5 /
// 8 / 12 / 18 it is near the best one for prompts of any width (4096 rows, 16 heads on 4:
// 64 wide 67 / 68 / 69 / 71 / 77, 192 wide 144 / 136 / 135 / 143 / 154, 256 wide 159 / 144 /
// 146 / 154 / 165; e4m3 87 / 82 / 80 / 83 / 89, 263 / 227 / 219 / 233 / 252 and 247 / 228 /
// 222 / 234 / 264), too high for steps of wide heads and slow feeds (16 steps, 256 wide 66 /
// 66 / 70 / 74 / 78, e4m3 69 / 74 / 80 / 88 / 96; bf16 in pages of 20 98 / 108 / 119 / 136 /
// 150, e4m3 in pages of 17 187 / 189 / 221 / 243 / 279).
constexpr int kCoresCost = 2, kTensorCost = 8;
// A share does not begin in the first or last `snap` tiles of a unit: on tensor cores
// a tile takes less than the join of a part (16 steps of 1 to 8 rows, us at 0 / 1 / 2 / 3:
// 35.4 / 35.4 / 37.1 / 38.8; the others the same, with fewer parts to join the larger
// it is), on CUDA cores several times as long (the window of fp32, at 0 / 1 / 2: 64 /
// 71 / 87).
constexpr int kCoresSnap = 0, kTensorSnap = 1;
// The least a share holds.
constexpr int kMinShare = 4;

// Where a share begins: a unit and a tile within it (b == batch: behind the last).
struct Start {
  int b, kvh, q, tile;
};
// A unit that is cut and begins in this share (its last segment): the shares that
// hold a part of it, this one and the next ones (0: nothing to join), and its rows.
struct Record {
  int parts, kvh;
  int row0;    // its sequence's first row of the step
  int r0, r1;  // its rows of the sequence and head
  int unused[3];
};

struct Params {
  const void* q;
  int64_t q_stride;
  const void *k, *v;
  int64_t page_stride, row_stride, head_stride;
  const float *k_scale, *v_scale;
  const int32_t *kept, *lens, *row_start, *table;
  void* out;
  float* lse;
  // workspace
  Start* starts;     // [ctas + 1]; NULL: each CTA finds its own
  Record* rec;       // [ctas]
  long long* base;   // [batch + 1] cost before each sequence
  float2* part_ml;   // [2 * ctas][bm] running maximum (base 2) and sum
  float* part_o;     // [2 * ctas][bm][dp] unnormalised; both NULL where no unit may be cut
  int heads, kv_heads, group, dim, dp, batch, rows, page, width, num_pages, window;
  int capacity;      // rows of a table's pages
  int bm, bn, ctas, unit_cost, snap;
  PageDiv page_div, group_div;
  float scale_log2;  // softmax scale * log2(e)
};

// One sequence of a step.
struct Sequence {
  int row0, tokens;  // its rows of the step
  int kept, length;  // position of the first one; cached rows
  int tiles;         // units per key/value head

  __device__ __forceinline__ void load(const Params& p, int b) {
    const int a = p.row_start[b], z = p.row_start[b + 1];
    row0 = min(max(a, 0), p.rows);
    tokens = min(max(z, row0), p.rows) - row0;
    kept = max(p.kept[b], 0);
    length = min(max(p.lens[b], 0), p.capacity);
    // (rows * heads < 2^31)
    tiles = (tokens * p.group + p.bm - 1) / p.bm;
  }
};

// What one unit covers.
struct Unit {
  int r0, r1;        // rows of its sequence and head: r0 .. r1 - 1
  int lo, hi;        // positions that any of its rows sees: lo .. hi - 1
  int tile0, tiles;  // tiles of bn positions

  __device__ __forceinline__ void set(const Params& p, const Sequence& s, int q) {
    r0 = q * p.bm;
    r1 = min(r0 + p.bm, s.tokens * p.group);
    const int first = p.group_div(r0), last = p.group_div(r1 - 1);
    hi = (int)min((long long)s.kept + last + 1, (long long)s.length);
    lo = p.window ? (int)min(max((long long)s.kept + first + 1 - p.window, 0ll), (long long)hi) : 0;
    tile0 = lo / p.bn;
    tiles = hi > lo ? (hi - 1) / p.bn + 1 - tile0 : 0;
  }
};

// Last position token i sees, and the first one.
__device__ __forceinline__ int last_seen(const Sequence& s, int i) {
  return (int)min((long long)s.kept + i, (long long)s.length - 1);
}
__device__ __forceinline__ int first_seen(const Params& p, const Sequence& s, int i) {
  return p.window ? (int)min(max((long long)s.kept + i + 1 - p.window, 0ll), 2147483647ll) : 0;
}

// What a share holds of one unit.
struct Segment {
  Unit unit;
  int t0, t1;        // tiles of the unit: t0 .. t1 - 1
  bool first, last;  // the unit's first tile, its last one are among them
};

// The segments of one share in order.  Every thread of a warp calls it with the
// same state.
struct Walk {
  Start at, end;
  Sequence seq;
  bool loaded;

  // `first`: the sequence that `from` names
  __device__ __forceinline__ void begin(const Start& from, const Start& to,
                                        const Sequence& first) {
    at = from;
    end = to;
    seq = first;
    loaded = true;
  }
  __device__ __forceinline__ bool in_last() const {
    return at.b == end.b && at.kvh == end.kvh && at.q == end.q;
  }
  // The segment at `at`, whose sequence is loaded.
  __device__ __forceinline__ Segment segment(const Params& p) const {
    Segment g;
    g.unit.set(p, seq, at.q);
    g.t0 = at.tile;
    g.t1 = g.unit.tiles;
    if (in_last()) g.t1 = min(g.t1, end.tile);
    g.first = g.t0 == 0;
    g.last = g.t1 == g.unit.tiles;
    return g;
  }
  // The next segment; false behind the last.
  __device__ __forceinline__ bool next(const Params& p, Segment& g) {
    if (in_last() && at.tile >= end.tile) return false;
    // (a workspace that another call is writing at the same time gives wrong
    // results, but no address outside this call's buffers)
    if (at.b < 0 || at.b >= p.batch || at.kvh < 0 || at.kvh >= p.kv_heads || at.tile < 0)
      return false;
    if (!loaded) {
      seq.load(p, at.b);
      loaded = true;
    }
    if (at.q < 0 || at.q >= seq.tiles) return false;
    g = segment(p);
    return at.tile <= g.unit.tiles;
  }
  // Past the segment.
  __device__ __forceinline__ void advance(const Params& p, const Segment& g) {
    if (!g.last) {
      at = end;
      return;
    }
    at.tile = 0;
    if (++at.q < seq.tiles) return;
    at.q = 0;
    if (++at.kvh < p.kv_heads) return;
    at.kvh = 0;
    at.b = next_sequence(p, at.b + 1);
    loaded = false;
  }
  // The first sequence at or behind b that has rows, 32 at a time; `batch` if none.
  __device__ __forceinline__ int next_sequence(const Params& p, int b) const {
    const int lane = threadIdx.x & 31;
    for (; b < p.batch; b += 32) {
      const int x = b + lane;
      bool some = false;
      if (x < p.batch && x <= end.b) {
        const int a = min(max(p.row_start[x], 0), p.rows), z = min(p.row_start[x + 1], p.rows);
        some = z > a;
      }
      const unsigned any = __ballot_sync(~0u, some);
      if (any) return b + __ffs(any) - 1;
      if (b + 32 > end.b) break;
    }
    return p.batch;
  }
};

// ---------------------------------------------------------------------------
// Where the shares begin
// ---------------------------------------------------------------------------

__device__ __forceinline__ int unit_cost(const Params& p, const Sequence& s, int q) {
  Unit u;
  u.set(p, s, q);
  return p.unit_cost + u.tiles;
}

// The cost of one sequence and key/value head, b < batch or none; a warp together
// where a lane's sequence has many units.
__device__ __forceinline__ long long sequence_cost(const Params& p, int b, Sequence& s) {
  constexpr int kAlone = 4;  // units a thread adds up by itself
  const int lane = threadIdx.x & 31;
  s = {0, 0, 0, 0, 0};
  if (b < p.batch) s.load(p, b);
  long long cost = 0;
  if (s.tiles <= kAlone)
    for (int q = 0; q < s.tiles; ++q) cost += unit_cost(p, s, q);
  unsigned many = __ballot_sync(~0u, s.tiles > kAlone);
  while (many) {
    const int from = __ffs(many) - 1;
    many &= many - 1;
    Sequence x;
    x.row0 = 0;
    x.tokens = __shfl_sync(~0u, s.tokens, from);
    x.kept = __shfl_sync(~0u, s.kept, from);
    x.length = __shfl_sync(~0u, s.length, from);
    x.tiles = __shfl_sync(~0u, s.tiles, from);
    long long sum = 0;
    for (int q = lane; q < x.tiles; q += 32) sum += unit_cost(p, x, q);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == from) cost = sum;
  }
  return cost;
}

// What a share holds at least, in all of `total` cost.
__device__ __forceinline__ long long share_size(const Params& p, long long total) {
  const long long even = (total + p.ctas - 1) / p.ctas;
  return even < kMinShare ? kMinShare : even;
}

// A share's beginning, and the unit that its place x lies in.
struct Place {
  Start st;
  Sequence seq;
  int q, tiles;      // that unit and its tiles
  long long x0;      // where it begins
  __device__ __forceinline__ bool inside() const { return st.tile > 0; }
};

// The place of share c, by a warp; base(b): the cost before sequence b, sequence(b).
template <typename Base, typename Seq>
__device__ __forceinline__ Place find_place(const Params& p, int c, long long total, Base base,
                                            Seq sequence) {
  const int lane = threadIdx.x & 31;
  const long long x = (long long)c * share_size(p, total);
  Place r;
  r.st = {p.batch, 0, 0, 0};
  r.seq = {0, 0, 0, 0, 0};
  r.q = r.tiles = 0;
  r.x0 = 0;
  if (x >= total || c >= p.ctas) return r;
  int lo = 0, hi = p.batch - 1;  // the first sequence whose cost ends behind x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (base(mid + 1) > x) hi = mid; else lo = mid + 1;
  }
  r.seq = sequence(lo);
  const long long from = base(lo), all = base(lo + 1) - from;
  // (32-bit divisions where the numbers allow, and they mostly do)
  long long one, rest = x - from;
  int kvh;
  if (all <= 0x7FFFFFFF) {
    one = (int)all / p.kv_heads;
    kvh = (int)rest / (int)one;
  } else {
    one = all / p.kv_heads;
    kvh = (int)(rest / one);
  }
  rest -= kvh * one;
  r.st.b = lo;
  r.st.kvh = kvh;
  for (int q0 = 0; q0 < r.seq.tiles; q0 += 32) {
    const int q = q0 + lane;
    const int mine = q < r.seq.tiles ? unit_cost(p, r.seq, q) : 0;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    const unsigned behind = __ballot_sync(~0u, upto > rest);
    if (behind) {
      const int at = __ffs(behind) - 1;
      r.q = q0 + at;
      r.tiles = __shfl_sync(~0u, mine, at) - p.unit_cost;
      rest -= __shfl_sync(~0u, upto - mine, at);
      break;
    }
    rest -= __shfl_sync(~0u, upto, 31);
  }
  r.x0 = x - rest;
  r.st.q = r.q;
  r.st.tile = (int)rest - p.unit_cost;
  if (r.st.tile <= p.snap) {
    r.st.tile = 0;
  } else if (r.st.tile >= r.tiles - p.snap) {
    // the next unit's beginning
    r.st.tile = 0;
    if (++r.st.q == r.seq.tiles) {
      r.st.q = 0;
      if (++r.st.kvh == p.kv_heads) {
        r.st.kvh = 0;
        // the next sequence with rows: idle ones' sums are equal
        const long long z = base(lo + 1);
        int a = lo + 1, e = p.batch;
        while (a < e) {
          const int mid = (a + e) >> 1;
          if (base(mid + 1) > z) e = mid; else a = mid + 1;
        }
        r.st.b = a;
      }
    }
  }
  return r;
}

// What share c leaves to join, given where it and the next one begin.
__device__ __forceinline__ Record make_record(const Params& p, int c, long long total,
                                              const Start& a, const Place& e) {
  Record r = {0, 0, 0, 0, 0, {0, 0, 0}};
  const bool same = a.b == e.st.b && a.kvh == e.st.kvh && a.q == e.st.q;
  // share c ends within a unit that it begins
  if (e.st.b >= p.batch || !e.inside() || (same && a.tile > 0)) return r;
  // the places behind e, a share apart, that lie within the unit as well
  const long long size = share_size(p, total);
  const long long x = (long long)(c + 1) * size;
  const long long last = e.x0 + p.unit_cost + e.tiles - p.snap - 1;
  Unit u;
  u.set(p, e.seq, e.q);
  r.parts = 2 + (int)((last - x) / size);
  r.kvh = e.st.kvh;
  r.row0 = e.seq.row0;
  r.r0 = u.r0;
  r.r1 = u.r1;
  return r;
}

// The beginnings of this CTA's share and the next one's, and its record, with a
// sequence to a thread: batch <= kInside.  `scratch`: shared memory, used until the
// call returns.
constexpr int kInside = 256;
struct PlanScratch {
  Sequence seq[kInside];
  long long cost[kInside], base[kInside + 1];
  long long warp[kInside / 32];
  Start start[2];
};
__device__ __forceinline__ void find_share(const Params& p, int cta, PlanScratch& t, Start& from,
                                           Start& to, Sequence& first) {
  constexpr int kWarps = kInside / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // neighbouring sequences in different warps, so that long ones are added up side by side
  if (warp < kWarps) {
    const int b = lane * kWarps + warp;
    Sequence s;
    t.cost[b] = sequence_cost(p, b, s) * p.kv_heads;
    t.seq[b] = s;
  }
  __syncthreads();
  long long upto = 0;
  if (warp < kWarps) {
    upto = t.cost[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) t.warp[warp] = upto;
  }
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long y = t.warp[w];
    if (w < warp) before += y;
    total += y;
  }
  if (warp < kWarps) t.base[tid + 1] = before + upto;
  if (tid == 0) t.base[0] = 0;
  __syncthreads();
  auto base = [&](int b) { return t.base[b]; };
  Place e;
  if (warp < 2) {
    e = find_place(p, cta + warp, total, base, [&](int b) { return t.seq[b]; });
    if (lane == 0) t.start[warp] = e.st;
  }
  __syncthreads();
  from = t.start[0];
  to = t.start[1];
  if (from.b < p.batch) first = t.seq[from.b];
  if (warp == 1 && lane == 0) p.rec[cta] = make_record(p, cta, total, from, e);
  __syncthreads();
}

// The same from the workspace, where a launch ahead has put them.  (All threads get what
// one of them read, and units that no share may cut are not: a workspace that another
// call is writing at the same time gives wrong results, but no threads that disagree on
// the barriers to come, and no parts where there is no room for them.)
__device__ __forceinline__ void read_share(const Params& p, int cta, PlanScratch& t, Start& from,
                                           Start& to, Sequence& first) {
  if (threadIdx.x < 2) {
    Start s = p.starts[cta + threadIdx.x];
    if (p.part_o == nullptr) s.tile = 0;
    t.start[threadIdx.x] = s;
  }
  __syncthreads();
  from = t.start[0];
  to = t.start[1];
  if (from.b >= 0 && from.b < p.batch) first.load(p, from.b);
  __syncthreads();
}

// Element types of a call: q/out and cache bf16; q/out bf16 beside an e4m3
// cache; all fp32.
enum Kind { kBf16 = 0, kE4m3 = 1, kFp32 = 2 };

// Weights beside an e4m3 cache are scaled by 2^kShift.
constexpr float kShift = 7.f;

struct Kernel {
  int bm, bn, dp, occupancy, unit_cost, snap;
  cudaError_t (*launch)(const Params& p, int ctas, cudaStream_t stream);
};
// CUDA cores (fp32); tensor cores with a bf16 cache in pages of whole runs of 8
// rows, in any other pages, and with an e4m3 cache.
Kernel kernel_cores(int dim);
Kernel kernel_tma(int dim);
Kernel kernel_rows(int dim);
Kernel kernel_convert(int dim);

int cores_status(bool clear);
int tma_status(bool clear);
int rows_status(bool clear);
int convert_status(bool clear);

}  // namespace chunk
}  // namespace mla
