// Attention of a step's new rows over a paged key/value cache
// (mla_chunk_attention): argument checks, the planner that cuts the work into
// equal shares, and the kernel that joins the parts of units cut between CTAs.

#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "chunk_attention.h"
#include "sm103_ptx.cuh"

namespace mla {

int chunk_device_status(bool clear) {
  const int words[4] = {chunk::tma_status(clear), chunk::rows_status(clear),
                        chunk::convert_status(clear), chunk::cores_status(clear)};
  int v = 0;
  for (int w : words) {
    if (w < 0) return -1;
    if (v == 0) v = w;
  }
  return v;
}

namespace chunk {
namespace {

// ---------------------------------------------------------------------------
// Planner
// ---------------------------------------------------------------------------
//
// Lengths are on the GPU only, so the shares are made there: one CTA sums the
// costs of all sequences (a sequence a thread, a warp together where one has
// many units) and a warp finds each share's beginning.

constexpr int kPlanThreads = 1024;
constexpr int kKeep = 2048;  // sequences whose sums stay in shared memory
constexpr int kAlone = 4;    // units a thread adds up by itself

__device__ __forceinline__ int unit_cost(const Params& p, const Sequence& s, int q) {
  Unit u;
  u.set(p, s, q);
  return kUnitCost + u.tiles;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const Params p) {
  __shared__ long long s_warp[32];
  __shared__ long long s_base[kKeep + 1];
  __shared__ Start s_start[kMaxCtas + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm103::pdl_wait();
  long long carry = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    Sequence s = {0, 0, 0, 0, 0};
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
    cost *= p.kv_heads;
    long long upto = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    long long before = carry;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const long long y = s_warp[w];
      if (w < warp) before += y;
      carry += y;
    }
    if (b < p.batch) {
      p.base[b + 1] = before + upto;
      if (b < kKeep) s_base[b + 1] = before + upto;
    }
    __syncthreads();
  }
  if (tid == 0) p.base[0] = s_base[0] = 0;
  __syncthreads();
  const long long total = carry;
  auto base = [&](int b) { return p.batch <= kKeep ? s_base[b] : p.base[b]; };
  const long long even = (total + p.ctas - 1) / p.ctas;
  const long long share = even < kMinShare ? kMinShare : even;
  for (int c = warp; c <= p.ctas; c += kPlanThreads / 32) {
    const long long x = (long long)c * share;
    Start st = {p.batch, 0, 0, 0};
    if (x < total && c < p.ctas) {
      int lo = 0, hi = p.batch - 1;  // the first sequence whose cost ends behind x
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (base(mid + 1) > x) hi = mid; else lo = mid + 1;
      }
      Sequence s;
      s.load(p, lo);
      const long long one = (base(lo + 1) - base(lo)) / p.kv_heads;
      long long rest = x - base(lo);
      st.b = lo;
      st.kvh = (int)(rest / one);
      rest -= st.kvh * one;
      int tiles = 0;
      for (int q0 = 0;; q0 += 32) {
        const int q = q0 + lane;
        const int mine = q < s.tiles ? unit_cost(p, s, q) : 0;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(~0u, upto, o);
          if (lane >= o) upto += y;
        }
        const unsigned behind = __ballot_sync(~0u, upto > rest);
        if (behind) {
          const int at = __ffs(behind) - 1;
          st.q = q0 + at;
          tiles = __shfl_sync(~0u, mine, at) - kUnitCost;
          rest -= __shfl_sync(~0u, upto - mine, at);
          break;
        }
        rest -= __shfl_sync(~0u, upto, 31);
        if (q0 + 32 >= s.tiles) {  // (cannot be: x lies before this sequence's end)
          st = {p.batch, 0, 0, 0};
          break;
        }
      }
      // rest: of the unit's cost, what lies before the share
      st.tile = (int)rest - kUnitCost;
      if (st.b < p.batch) {
        if (st.tile <= kSnap) {
          st.tile = 0;
        } else if (st.tile >= tiles - kSnap) {
          // the next unit's beginning
          st.tile = 0;
          if (++st.q == s.tiles) {
            st.q = 0;
            if (++st.kvh == p.kv_heads) {
              st.kvh = 0;
              // the next sequence with rows
              const long long z = base(st.b + 1);
              int a = st.b + 1, e = p.batch;
              while (a < e) {
                const int mid = (a + e) >> 1;
                if (base(mid + 1) > z) e = mid; else a = mid + 1;
              }
              st.b = a;
            }
          }
        }
      }
    }
    if (lane == 0) {
      s_start[c] = st;
      p.starts[c] = st;
    }
  }
  __syncthreads();
  for (int c = tid; c < p.ctas; c += kPlanThreads) {
    Record r = {0, 0, 0, 0};
    const Start e = s_start[c + 1], a = s_start[c];
    auto same = [](const Start& x, const Start& y) {
      return x.b == y.b && x.kvh == y.kvh && x.q == y.q;
    };
    // share c ends within a unit that it begins
    if (e.b < p.batch && e.tile > 0 && !(same(a, e) && a.tile > 0)) {
      int k = c + 1;
      while (k + 1 <= p.ctas && same(s_start[k + 1], e)) ++k;
      r = {k - c + 1, e.b, e.kvh, e.q};
    }
    p.rec[c] = r;
  }
}

// ---------------------------------------------------------------------------
// Join
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256, kJoinRow = 64, kJoinRows = kJoinThreads / kJoinRow;
constexpr int kJoinLoads = 8, kJoinY = 8;

// The parts of a cut unit's rows are weighted by 2^(m - max m) and added up in
// order, so repeated calls give the same bits.  64 threads take a row: a vector of
// four columns each, and what threads are left walk over the parts side by side.
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const Params p, const int kind) {
  __shared__ float s_w[kJoinRows][kMaxCtas], s_l[kJoinRows][kMaxCtas];
  __shared__ float s_red[kJoinRows][2];
  __shared__ float4 s_acc[kJoinThreads];
  sm103::pdl_wait();
  const int tid = threadIdx.x, r = tid / kJoinRow, i0 = tid % kJoinRow, cta = blockIdx.x;
  const Record rec = p.rec[cta];
  // (a workspace that another call is writing at the same time gives wrong
  // results, but no address outside this call's buffers)
  if (rec.parts <= 1 || rec.parts > p.ctas - cta || rec.b < 0 || rec.b >= p.batch || rec.kvh < 0 ||
      rec.kvh >= p.kv_heads)
    return;
  Sequence s;
  s.load(p, rec.b);
  if (rec.q < 0 || rec.q >= s.tiles) return;
  Unit u;
  u.set(p, s, rec.q);
  const int rows = u.r1 - u.r0;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? 2 * cta + 1 : 2 * (cta + k)); };
  const int cols = p.dp / 4, groups = kJoinRow / cols;
  const int grp = i0 / cols, c = i0 - grp * cols;
  const float vs = p.v_scale ? p.v_scale[rec.kvh] : 1.f;
  for (int row0 = blockIdx.y * kJoinRows; row0 < rows; row0 += kJoinY * kJoinRows) {
    const int row = row0 + r;
    const bool live = row < rows;
    const int parts = live ? rec.parts : 0;
    float M = -INFINITY;
    for (int k = i0; k < parts; k += kJoinRow) {
      const float2 ml = p.part_ml[slot(k) * p.bm + row];
      s_w[r][k] = ml.x;
      s_l[r][k] = ml.y;
      M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    if ((tid & 31) == 0) s_red[r][i0 >> 5] = M;
    __syncthreads();
    M = fmaxf(s_red[r][0], s_red[r][1]);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int k = i0; k < parts; k += kJoinRow) {
      const float w = sm103::ex2(s_w[r][k] - base);
      s_w[r][k] = w;
      L += w * s_l[r][k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(~0u, L, o);
    __syncthreads();
    if ((tid & 31) == 0) s_red[r][i0 >> 5] = L;
    __syncthreads();
    L = s_red[r][0] + s_red[r][1];
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp < groups) {
      const float* part = p.part_o + (int64_t)row * p.dp + c * 4;
      const int64_t step = (int64_t)p.bm * p.dp;
      for (int k0 = grp; k0 < parts; k0 += groups * kJoinLoads) {
        float4 x[kJoinLoads];
#pragma unroll
        for (int i = 0; i < kJoinLoads; ++i) {
          const int k = k0 + i * groups;
          if (k < parts) x[i] = *reinterpret_cast<const float4*>(part + slot(k) * step);
        }
#pragma unroll
        for (int i = 0; i < kJoinLoads; ++i) {
          const int k = k0 + i * groups;
          if (k < parts) {
            const float w = s_w[r][k];
            // (a part whose rows all weigh nothing holds zeros, or NaN where the row is NaN)
            a.x = fmaf(w, x[i].x, a.x);
            a.y = fmaf(w, x[i].y, a.y);
            a.z = fmaf(w, x[i].z, a.z);
            a.w = fmaf(w, x[i].w, a.w);
          }
        }
      }
    }
    s_acc[tid] = a;
    __syncthreads();
    if (live) {
      const int i = p.group_div(u.r0 + row), j = u.r0 + row - i * p.group;
      const int64_t head = (int64_t)(s.row0 + i) * p.heads + rec.kvh * p.group + j;
      if (i0 < cols && c * 4 < p.dim) {
        for (int g = 1; g < groups; ++g) {
          const float4 y = s_acc[r * kJoinRow + g * cols + c];
          a.x += y.x;
          a.y += y.y;
          a.z += y.z;
          a.w += y.w;
        }
        const float inv = L == 0.f ? 0.f : vs / L;
        if (kind == kFp32)
          *reinterpret_cast<float4*>((float*)p.out + head * p.dim + c * 4) =
              make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        else
          *reinterpret_cast<uint2*>((__nv_bfloat16*)p.out + head * p.dim + c * 4) = make_uint2(
              sm103::pack_bf16(a.x * inv, a.y * inv), sm103::pack_bf16(a.z * inv, a.w * inv));
      }
      if (i0 == 0 && p.lse)
        p.lse[head] =
            L == 0.f ? -INFINITY
                     : (M + (log2f(L) - (kind == kE4m3 ? kShift : 0.f))) * 0.6931471805599453f;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

int kind_of(const mla_kv_geometry_t* g) {
  return g->dtype == MLA_DTYPE_FP32 ? kFp32 : g->cache_dtype == MLA_DTYPE_E4M3 ? kE4m3 : kBf16;
}

Kernel kernel_of(const mla_kv_geometry_t* g, int page_size) {
  const int kind = kind_of(g), dim = g->head_dim;
  return kind == kFp32        ? kernel_cores(dim)
         : kind == kE4m3      ? kernel_convert(dim)
         : page_size % 8 == 0 ? kernel_tma(dim)
                              : kernel_rows(dim);
}

struct Plan {
  Kernel k;
  int ctas;
  bool cut;  // a unit may fall into several shares
  size_t off_rec, off_base, off_ml, off_o, bytes;
};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

Plan make_plan(const mla_kv_geometry_t* g, int batch, int rows, int page_size, int max_pages) {
  Plan d;
  d.k = kernel_of(g, page_size);
  const int group = g->num_heads / g->num_kv_heads;
  const int64_t tiles = ((int64_t)page_size * max_pages + d.k.bn - 1) / d.k.bn;
  // no sequence has more than `rows` rows, and each may end in a unit of its own
  const int64_t live = batch < rows ? batch : rows;
  const int64_t units = (((int64_t)rows * group + d.k.bm - 1) / d.k.bm + live) * g->num_kv_heads;
  int64_t ctas = (int64_t)device_sm_count() * d.k.occupancy;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  // (units * tiles may be beyond 64 bits only where either is far beyond the CTAs)
  const int64_t most = units > ctas || tiles > ctas ? ctas : units * tiles;
  if (ctas > most) ctas = most;
  if (ctas < 1) ctas = 1;
  d.ctas = (int)ctas;
  d.cut = tiles > 2 * kSnap + 1;
  size_t off = align256(sizeof(Start) * (ctas + 1));
  d.off_rec = off;
  off = align256(off + sizeof(Record) * ctas);
  d.off_base = off;
  off = align256(off + sizeof(long long) * ((size_t)batch + 1));
  d.off_ml = off;
  if (d.cut) {
    const size_t parts = (size_t)2 * ctas * d.k.bm;
    off = align256(off + sizeof(float2) * parts);
    d.off_o = off;
    off = align256(off + sizeof(float) * parts * d.k.dp);
  } else {
    d.off_o = off;
  }
  d.bytes = off;
  return d;
}

cudaError_t run(const Plan& d, const Params& p, int kind, cudaStream_t stream) {
  cudaError_t e;
  {
    KernelTimer kt("chunk_plan", stream);
    e = launch_dependent(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
  }
  if (e != cudaSuccess) return e;
  e = d.k.launch(p, d.ctas, stream);
  if (e != cudaSuccess || !d.cut) return e;
  KernelTimer kt("chunk_join", stream);
  return launch_dependent(chunk_join_kernel, dim3((unsigned)d.ctas, kJoinY), dim3(kJoinThreads), 0,
                          stream, p, kind);
}

mla_status_t sizes_ok(const mla_kv_geometry_t* g, int batch, int rows, int page_size,
                      int max_pages) {
  const mla_status_t st = kv_geometry_ok(g);
  if (st != MLA_OK) return st;
  if (batch < 1 || batch > 65535 || rows < 0 || page_size < 1 || max_pages < 1 ||
      (int64_t)page_size * max_pages > INT_MAX - 1023) {
    set_error("chunk: need 1 <= batch <= 65535, rows >= 0, page_size and max_pages_per_seq >= 1 "
              "with at most 2^31 - 1024 rows between them (batch=%d rows=%d page_size=%d "
              "max_pages=%d)", batch, rows, page_size, max_pages);
    return MLA_ERR_INVALID_ARG;
  }
  if ((int64_t)rows * g->num_heads > INT_MAX - 1023) {
    set_error("chunk: %d rows of %d heads are too many for one call", rows, g->num_heads);
    return MLA_ERR_UNSUPPORTED;
  }
  return MLA_OK;
}

}  // namespace
}  // namespace chunk
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_chunk_workspace_bytes(const mla_kv_geometry_t* g, int32_t batch,
                                                  int32_t rows, int32_t page_size,
                                                  int32_t max_pages_per_seq, size_t* bytes) {
  if (bytes == nullptr) {
    set_error("bytes output is NULL");
    return MLA_ERR_INVALID_ARG;
  }
  const mla_status_t st = chunk::sizes_ok(g, batch, rows, page_size, max_pages_per_seq);
  if (st != MLA_OK) return st;
  *bytes = rows == 0 ? 0 : chunk::make_plan(g, batch, rows, page_size, max_pages_per_seq).bytes;
  return MLA_OK;
}

extern "C" mla_status_t mla_chunk_attention(
    const mla_kv_geometry_t* g, const void* q, int64_t q_row_stride, int32_t rows,
    const mla_kv_cache_t* cache, const int32_t* kept_lens, const int32_t* cache_lens,
    const int32_t* row_start, int32_t batch, const int32_t* page_table, int32_t max_pages_per_seq,
    int32_t window, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  mla_status_t st = kv_geometry_ok(g);
  if (st != MLA_OK) return st;
  st = kv_cache_ok(g, cache);
  if (st != MLA_OK) return st;
  st = chunk::sizes_ok(g, batch, rows, cache->page_size, max_pages_per_seq);
  if (st != MLA_OK) return st;
  if (window < 0) {
    set_error("chunk: window %d is negative", window);
    return MLA_ERR_INVALID_ARG;
  }
  if (rows == 0) return MLA_OK;
  const void* ptrs[] = {q, kept_lens, cache_lens, row_start, page_table, out};
  const char* names[] = {"q", "kept_lens", "cache_lens", "row_start", "page_table", "out"};
  for (int i = 0; i < 6; ++i) {
    if (ptrs[i] == nullptr || ((uintptr_t)ptrs[i] & 15u)) {
      set_error("chunk: %s is NULL or not 16-byte aligned", names[i]);
      return MLA_ERR_INVALID_ARG;
    }
  }
  if ((uintptr_t)lse & 3u) {
    set_error("chunk: lse is not 4-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  const int eb = g->dtype == MLA_DTYPE_BF16 ? 2 : 4;
  const int64_t row = (int64_t)g->num_heads * g->head_dim;
  if (q_row_stride < row || q_row_stride * eb % 16 != 0) {
    set_error("chunk: q_row_stride %lld must be at least %lld and a multiple of 16 bytes",
              (long long)q_row_stride, (long long)row);
    return MLA_ERR_INVALID_ARG;
  }
  const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)out;
  const uintptr_t q1 = q0 + (uintptr_t)(((rows - 1) * q_row_stride + row) * eb);
  const uintptr_t o1 = o0 + (uintptr_t)(rows * row * eb);
  if (q0 < o1 && o0 < q1) {
    set_error("chunk: out overlaps q");
    return MLA_ERR_INVALID_ARG;
  }
  const chunk::Plan d =
      chunk::make_plan(g, batch, rows, cache->page_size, max_pages_per_seq);
  if (workspace == nullptr || workspace_bytes < d.bytes) {
    set_error("workspace of %zu bytes is smaller than the %zu this call needs", workspace_bytes,
              d.bytes);
    return MLA_ERR_WORKSPACE;
  }
  if ((uintptr_t)workspace & 255u) {
    set_error("workspace is not 256-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  chunk::Params p;
  p.q = q;
  p.q_stride = q_row_stride;
  p.k = cache->k;
  p.v = cache->v;
  p.page_stride = cache->page_stride;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.kept = kept_lens;
  p.lens = cache_lens;
  p.row_start = row_start;
  p.table = page_table;
  p.out = out;
  p.lse = lse;
  char* ws = (char*)workspace;
  p.starts = (chunk::Start*)ws;
  p.rec = (chunk::Record*)(ws + d.off_rec);
  p.base = (long long*)(ws + d.off_base);
  p.part_ml = (float2*)(ws + d.off_ml);
  p.part_o = (float*)(ws + d.off_o);
  p.heads = g->num_heads;
  p.kv_heads = g->num_kv_heads;
  p.group = g->num_heads / g->num_kv_heads;
  p.dim = g->head_dim;
  p.dp = d.k.dp;
  p.batch = batch;
  p.rows = rows;
  p.page = cache->page_size;
  p.width = max_pages_per_seq;
  p.num_pages = cache->num_pages;
  p.window = window;
  p.capacity = (int)((int64_t)max_pages_per_seq * cache->page_size);
  p.bm = d.k.bm;
  p.bn = d.k.bn;
  p.ctas = d.ctas;
  p.page_div = PageDiv(cache->page_size);
  p.group_div = PageDiv(p.group);
  const double scale = g->softmax_scale > 0.f ? (double)g->softmax_scale
                                              : 1.0 / std::sqrt((double)g->head_dim);
  p.scale_log2 = (float)(scale * 1.4426950408889634);
  const cudaError_t e = chunk::run(d, p, chunk::kind_of(g), (cudaStream_t)stream);
  if (e != cudaSuccess) {
    set_error("CUDA error %d (%s)", (int)e, cudaGetErrorString(e));
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}
