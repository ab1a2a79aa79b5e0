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
// Lengths are on the GPU only, so the shares are made there.  Up to kInside
// sequences each CTA of the attention finds its own share, which takes it 2 to 3
// us; a launch ahead of it would take more (16 sequences 8.5 us by itself).
// Beyond, one CTA sums the costs of all sequences and a warp finds each share's
// beginning.

constexpr int kPlanThreads = 1024;
constexpr int kKeep = 2048;  // sequences whose sums stay in shared memory

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const Params p) {
  __shared__ long long s_warp[32];
  __shared__ long long s_base[kKeep + 1];
  __shared__ Start s_start[kMaxCtas + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm103::pdl_wait();
  long long total = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int b = b0 + tid;
    Sequence own;
    long long upto = sequence_cost(p, b, own) * p.kv_heads;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    long long before = total;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const long long y = s_warp[w];
      if (w < warp) before += y;
      total += y;
    }
    if (b < p.batch) {
      p.base[b + 1] = before + upto;
      if (b < kKeep) s_base[b + 1] = before + upto;
    }
    __syncthreads();
  }
  if (tid == 0) p.base[0] = s_base[0] = 0;
  __syncthreads();
  auto base = [&](int b) { return p.batch <= kKeep ? s_base[b] : p.base[b]; };
  auto sequence = [&](int b) {
    Sequence s;
    s.load(p, b);
    return s;
  };
  for (int c = warp; c <= p.ctas; c += kPlanThreads / 32) {
    const Place e = find_place(p, c, total, base, sequence);
    if (lane == 0) {
      s_start[c] = e.st;
      p.starts[c] = e.st;
    }
  }
  __syncthreads();
  for (int c = warp; c < p.ctas; c += kPlanThreads / 32) {
    const Place e = find_place(p, c + 1, total, base, sequence);
    if (lane == 0) p.rec[c] = make_record(p, c, total, s_start[c], e);
  }
}

// ---------------------------------------------------------------------------
// Join
// ---------------------------------------------------------------------------

// Rows of a unit are spread over kJoinY CTAs, most of which have none in short steps
// (us at 32 / 16 / 12: 16 steps 35.4 / 33.8 / 33.4, a prompt of 8192 rows 396 / 392 /
// 391, one context of 131072 with 38 parts a row 64.8 / 64.7 / 74).  Eight loads of a
// row's parts at once fit 64 registers, so four CTAs an SM (16 loads and two CTAs: 61 for
// the long context, 36 and 401 for the others).
constexpr int kJoinThreads = 256, kJoinY = 16, kJoinLoads = 8;

// The parts of a cut unit's rows are weighted by 2^(m - max m) and added up in
// order, so repeated calls give the same bits.  A warp takes a row, a lane four
// columns of it at a time; few parts, as in a prompt, are all asked for beside their
// maxima and sums (152 cut units of 256 rows: one trip to memory a row, not three).
__global__ void __launch_bounds__(kJoinThreads, 4) chunk_join_kernel(const Params p, const int kind) {
  sm103::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x;
  const Record rec = p.rec[cta];
  const int rows = rec.r1 - rec.r0;
  // (a workspace that another call is writing at the same time gives wrong
  // results, but no address outside this call's buffers)
  if (rec.parts <= 1 || rec.parts > p.ctas - cta || rec.kvh < 0 || rec.kvh >= p.kv_heads ||
      rec.row0 < 0 || rec.r0 < 0 || rows > p.bm ||
      rec.r1 > (int64_t)(p.rows - rec.row0) * p.group)
    return;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? 2 * cta + 1 : 2 * (cta + k)); };
  const float vs = p.v_scale ? p.v_scale[rec.kvh] : 1.f;
  const int64_t step = (int64_t)p.bm * p.dp;
  auto write = [&](int row, int c, float4 a, float M, float L) {
    const int i = p.group_div(rec.r0 + row), j = rec.r0 + row - i * p.group;
    const int64_t head = (int64_t)(rec.row0 + i) * p.heads + rec.kvh * p.group + j;
    if (c == 0 && p.lse)
      p.lse[head] =
          L == 0.f ? -INFINITY
                   : (M + (log2f(L) - (kind == kE4m3 ? kShift : 0.f))) * 0.6931471805599453f;
    if (c >= p.dim) return;
    if (L == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);  // (it may be no numbers)
    const float inv = L == 0.f ? 0.f : vs / L;
    if (kind == kFp32)
      *reinterpret_cast<float4*>((float*)p.out + head * p.dim + c) =
          make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    else
      *reinterpret_cast<uint2*>((__nv_bfloat16*)p.out + head * p.dim + c) = make_uint2(
          sm103::pack_bf16(a.x * inv, a.y * inv), sm103::pack_bf16(a.z * inv, a.w * inv));
  };
  // (a part whose rows all weigh nothing holds zeros, or NaN where the row is NaN)
  auto add = [](float4& a, float w, const float4& x) {
    a.x = fmaf(w, x.x, a.x);
    a.y = fmaf(w, x.y, a.y);
    a.z = fmaf(w, x.z, a.z);
    a.w = fmaf(w, x.w, a.w);
  };
  constexpr int kWarps = kJoinThreads / 32, kFew = 4;
  if (rec.parts <= kFew) {
    for (int row = blockIdx.y * kWarps + warp; row < rows; row += kJoinY * kWarps) {
      for (int c = 4 * lane; c - 4 * lane < p.dim; c += 128) {
        float2 ml[kFew];
        float4 x[kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
          ml[k] = make_float2(-INFINITY, 0.f);
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k >= rec.parts) continue;
          ml[k] = p.part_ml[slot(k) * p.bm + row];
          if (c < p.dim)
            x[k] = *reinterpret_cast<const float4*>(p.part_o + slot(k) * step +
                                                    (int64_t)row * p.dp + c);
        }
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < kFew; ++k) M = fmaxf(M, ml[k].x);
        const float base = M == -INFINITY ? 0.f : M;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
          if (k >= rec.parts) continue;
          const float w = sm103::ex2(ml[k].x - base);
          L = fmaf(w, ml[k].y, L);
          add(a, w, x[k]);
        }
        write(row, c, a, M, L);
      }
    }
    return;
  }
  for (int row = blockIdx.y * kWarps + warp; row < rows; row += kJoinY * kWarps) {
    float M = -INFINITY;
    for (int k = lane; k < rec.parts; k += 32) M = fmaxf(M, p.part_ml[slot(k) * p.bm + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    for (int c = 4 * lane; c - 4 * lane < p.dim; c += 128) {
      const float* part = p.part_o + (int64_t)row * p.dp + c;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
      for (int k0 = 0; k0 < rec.parts; k0 += 32) {
        const int n = min(32, rec.parts - k0);
        float w = 0.f, l = 0.f;
        if (lane < n) {
          const float2 ml = p.part_ml[slot(k0 + lane) * p.bm + row];
          w = sm103::ex2(ml.x - base);
          l = w * ml.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
        L += l;
        for (int k1 = 0; k1 < n; k1 += kJoinLoads) {
          float4 x[kJoinLoads];
#pragma unroll
          for (int e = 0; e < kJoinLoads; ++e)
            if (c < p.dim && k1 + e < n)
              x[e] = *reinterpret_cast<const float4*>(part + slot(k0 + k1 + e) * step);
#pragma unroll
          for (int e = 0; e < kJoinLoads; ++e) {
            const float we = __shfl_sync(~0u, w, (k1 + e) & 31);
            if (c < p.dim && k1 + e < n) add(a, we, x[e]);
          }
        }
      }
      write(row, c, a, M, L);
    }
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
  d.cut = tiles > 2 * d.k.snap + 1;
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
  cudaError_t e = cudaSuccess;
  if (p.starts != nullptr) {
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
  // (the caches are not looked at: their strides may leave room for other buffers)
  struct Span {
    const char* name;
    const void* at;
    int64_t bytes;
  };
  const int64_t lse_bytes = (int64_t)rows * g->num_heads * 4, scales = (int64_t)g->num_kv_heads * 4;
  const Span spans[] = {
      {"out", out, rows * row * eb},
      {"lse", lse, lse_bytes},
      {"the workspace", workspace, (int64_t)d.bytes},
      {"q", q, ((rows - 1) * q_row_stride + row) * eb},
      {"kept_lens", kept_lens, (int64_t)batch * 4},
      {"cache_lens", cache_lens, (int64_t)batch * 4},
      {"row_start", row_start, ((int64_t)batch + 1) * 4},
      {"page_table", page_table, (int64_t)batch * max_pages_per_seq * 4},
      {"k_scale", cache->k_scale, scales},
      {"v_scale", cache->v_scale, scales},
  };
  constexpr int kWritten = 3, kSpans = sizeof(spans) / sizeof(spans[0]);
  for (int i = 0; i < kWritten; ++i) {
    for (int j = i + 1; j < kSpans; ++j) {
      const uintptr_t a = (uintptr_t)spans[i].at, b = (uintptr_t)spans[j].at;
      if (a != 0 && b != 0 && a < b + (uintptr_t)spans[j].bytes &&
          b < a + (uintptr_t)spans[i].bytes) {
        set_error("chunk: %s overlaps %s", spans[i].name, spans[j].name);
        return MLA_ERR_INVALID_ARG;
      }
    }
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
  p.starts = batch > chunk::kInside ? (chunk::Start*)ws : nullptr;
  p.rec = (chunk::Record*)(ws + d.off_rec);
  p.base = (long long*)(ws + d.off_base);
  p.part_ml = d.cut ? (float2*)(ws + d.off_ml) : nullptr;
  p.part_o = d.cut ? (float*)(ws + d.off_o) : nullptr;
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
  p.unit_cost = d.k.unit_cost;
  p.snap = d.k.snap;
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
