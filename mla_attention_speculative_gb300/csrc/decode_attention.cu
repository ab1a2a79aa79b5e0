// Attention of one new token per sequence over a paged key/value cache
// (mla_decode_attention): argument checks, the choice of kernel, and the
// kernel that joins the parts of sequences cut between CTAs.  The attention
// itself is in decode_kernel.cuh.

#include <cuda_bf16.h>

#include <climits>
#include <cmath>
#include <mutex>

#include "decode_attention.h"
#include "sm103_ptx.cuh"

namespace mla {

int decode_device_status(bool clear) {
  const int words[3] = {decode::bf16_status(clear), decode::e4m3_status(clear),
                        decode::fp32_status(clear)};
  int v = 0;
  for (int w : words) {
    if (w < 0) return -1;
    if (v == 0) v = w;
  }
  return v;
}

mla_status_t kv_geometry_ok(const mla_kv_geometry_t* g) {
  if (g == nullptr) {
    set_error("geometry is NULL");
    return MLA_ERR_INVALID_ARG;
  }
  if (g->num_heads < 1 || g->num_kv_heads < 1 || g->head_dim < 1 ||
      g->num_heads % g->num_kv_heads != 0) {
    set_error("geometry needs num_heads a positive multiple of num_kv_heads and head_dim >= 1 "
              "(heads=%d kv_heads=%d dim=%d)", g->num_heads, g->num_kv_heads, g->head_dim);
    return MLA_ERR_INVALID_ARG;
  }
  if (g->dtype != MLA_DTYPE_BF16 && g->dtype != MLA_DTYPE_FP32) {
    set_error("unknown dtype %d", g->dtype);
    return MLA_ERR_INVALID_ARG;
  }
  if (g->cache_dtype != g->dtype &&
      !(g->cache_dtype == MLA_DTYPE_E4M3 && g->dtype == MLA_DTYPE_BF16)) {
    set_error("a cache of dtype %d does not go with dtype %d (the same, or e4m3 with bf16)",
              g->cache_dtype, g->dtype);
    return MLA_ERR_UNSUPPORTED;
  }
  const int vec = g->dtype == MLA_DTYPE_FP32 ? 4 : g->cache_dtype == MLA_DTYPE_E4M3 ? 16 : 8;
  if (g->head_dim % vec != 0 || g->head_dim > 256) {
    set_error("head_dim %d must be a multiple of %d up to 256", g->head_dim, vec);
    return MLA_ERR_INVALID_ARG;
  }
  if (g->num_heads > 65535) {
    set_error("%d heads are more than 65535", g->num_heads);
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

mla_status_t kv_cache_ok(const mla_kv_geometry_t* g, const mla_kv_cache_t* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) {
    set_error("the cache or one of its bases is NULL");
    return MLA_ERR_INVALID_ARG;
  }
  if (((uintptr_t)c->k | (uintptr_t)c->v) & 15u) {
    set_error("a cache base is not 16-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  if (c->page_size < 1 || c->num_pages < 1) {
    set_error("cache needs page_size and num_pages >= 1 (%d, %d)", c->page_size, c->num_pages);
    return MLA_ERR_INVALID_ARG;
  }
  const int64_t eb = g->cache_dtype == MLA_DTYPE_FP32 ? 4 : g->cache_dtype == MLA_DTYPE_E4M3 ? 1 : 2;
  const int64_t strides[3] = {c->page_stride, c->row_stride, c->head_stride};
  const int64_t extent[3] = {c->num_pages, c->page_size, g->num_kv_heads};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || strides[i] * eb % 16 != 0 ||
        (extent[i] > 1 && strides[i] < g->head_dim)) {
      set_error("cache strides (page %lld, row %lld, head %lld) must be 16-byte multiples and "
                "cover head_dim", (long long)c->page_stride, (long long)c->row_stride,
                (long long)c->head_stride);
      return MLA_ERR_INVALID_ARG;
    }
  }
  if ((c->k_scale || c->v_scale) && g->cache_dtype != MLA_DTYPE_E4M3) {
    set_error("k_scale and v_scale go with an e4m3 cache only");
    return MLA_ERR_INVALID_ARG;
  }
  if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3u) {
    set_error("a cache scale is not 4-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

namespace decode {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinLoads = 8;  // parts a thread asks for at once

// The parts of a row, in the share its segment begins in and the next ones,
// are weighted by exp(m - max m) and summed in order.  They are few and small
// (16 rows of 1 KB a share at most), so this is bound by the latency of its
// loads: TPR threads take a row, groups of them walk over the parts side by
// side with kJoinLoads parts on their way at once, the first of them while the
// weights are made.  Few segments have many parts each: then a whole CTA
// takes a row (T = 131072: 50.1 us a call against 51.5 with 64 threads);
// many segments have few: 64 threads a row leave fewer CTAs with nothing to do.
template <int TPR>
__global__ void __launch_bounds__(kJoinThreads)
    decode_join_kernel(const Params p, const int ctas, const int rows_max, const int rows_live,
                       const int dp, const int kind) {
  constexpr int RPC = kJoinThreads / TPR, WPR = TPR / 32;
  __shared__ float s_w[RPC][kMaxCtas], s_l[RPC][kMaxCtas];
  __shared__ float s_red[RPC][WPR];
  __shared__ float4 s_acc[kJoinThreads];
  // (No later kernel is let in early from here.  The attention's equal shares
  // need its CTAs spread evenly; started while this kernel still held parts of
  // the SMs, a next call's ended up three on one SM and none on another, and 32
  // sequences of up to 32768 positions took 452 us instead of 327.)
  sm103::pdl_wait();
  const int tid = threadIdx.x, r = tid / TPR, i0 = tid % TPR, unit = blockIdx.y * RPC + r;
  // this row of the segment's: head `sub` of its group, row `head_row` of the row tile
  const int sub = unit / rows_live, head_row = unit - sub * rows_live;
  const int row = sub * rows_max + head_row, stride = p.hg * rows_max;
  const Record rec = p.rec[blockIdx.x];
  // (a workspace that another call is writing at the same time gives wrong
  // results, but no address outside this call's buffers)
  if (rec.parts <= 0 || rec.cta < 0 || rec.cta >= ctas || rec.parts > ctas - rec.cta ||
      rec.b < 0 || rec.b >= p.batch || rec.hr < 0 || rec.hr >= p.kv_groups * p.row_tiles)
    return;
  const int kvg = rec.hr / p.row_tiles, rt = rec.hr - kvg * p.row_tiles;
  const int kvh = kvg * p.hg + sub;
  const bool live = sub < p.hg && head_row < min(rows_max, p.group - rt * rows_max);
  const int parts = live ? rec.parts : 0;
  // part k: the last segment of the first share, then the first one of those behind it
  auto slot = [&](int k) { return (int64_t)(k == 0 ? 2 * rec.cta + 1 : 2 * (rec.cta + k)); };
  float M = -INFINITY;
  for (int k = i0; k < parts; k += TPR) {
    const float2 ml = p.part_ml[slot(k) * stride + row];
    s_w[r][k] = ml.x;
    s_l[r][k] = ml.y;
    M = fmaxf(M, ml.x);
  }
  const int cols = dp / 4, groups = TPR / cols;
  const int grp = i0 / cols, c = i0 - grp * cols;
  const float* part = p.part_o + (int64_t)row * dp + c * 4;
  const int64_t step = (int64_t)stride * dp;
  float4 x[kJoinLoads];
  auto ask = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      const int k = k0 + i * groups;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < parts) x[i] = *reinterpret_cast<const float4*>(part + slot(k) * step);
    }
  };
  if (grp < groups) ask(grp);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
  if ((tid & 31) == 0) s_red[r][i0 >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WPR; ++w) M = fmaxf(M, s_red[r][w]);
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int k = i0; k < parts; k += TPR) {
    const float w = sm103::ex2(s_w[r][k] - base);
    s_w[r][k] = w;
    L += w * s_l[r][k];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(~0u, L, o);
  __syncthreads();
  if ((tid & 31) == 0) s_red[r][i0 >> 5] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) L += s_red[r][w];

  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (grp < groups) {
    for (int k0 = grp; k0 < parts; k0 += groups * kJoinLoads) {
      if (k0 > grp) ask(k0);
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i) {
        const int k = k0 + i * groups;
        if (k < parts) {
          const float w = s_w[r][k];
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
  if (!live) return;
  const int64_t head = (int64_t)rec.b * p.heads + kvh * p.group + rt * rows_max + head_row;
  if (i0 < cols && c * 4 < p.dim) {
    for (int g = 1; g < groups; ++g) {
      const float4 y = s_acc[r * TPR + g * cols + c];
      a.x += y.x;
      a.y += y.y;
      a.z += y.z;
      a.w += y.w;
    }
    const float vs = p.v_scale ? p.v_scale[kvh] : 1.f;
    const float inv = L == 0.f ? 0.f : vs / L;
    if (kind == kFp32)
      *reinterpret_cast<float4*>((float*)p.out + head * p.dim + c * 4) =
          make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    else
      *reinterpret_cast<uint2*>((__nv_bfloat16*)p.out + head * p.dim + c * 4) = make_uint2(
          sm103::pack_bf16(a.x * inv, a.y * inv), sm103::pack_bf16(a.z * inv, a.w * inv));
  }
  if (i0 == 0 && p.lse)
    p.lse[head] = L == 0.f ? -INFINITY
                           : (M + log2f(L) - (kind == kE4m3 ? kShift : 0.f)) * 0.6931471805599453f;
}

// The kernel of a geometry, how its work is cut, and the workspace.
struct Plan {
  Kernel k;
  int kind, row_tiles, ctas;
  int hg, pw, tile, kv_groups;
  bool cut;         // a segment may fall into several shares
  bool by_segment;  // records by segment: fewer than CTAs
  int records;
  size_t off_ml, off_o, bytes;
};

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

Kernel kernel_of(const mla_kv_geometry_t* g, int kind) {
  // one row multiple when the group fits it: half the products and registers
  const int nt = g->num_heads / g->num_kv_heads <= (kind == kFp32 ? 4 : 8) ? 1 : 2;
  return kind == kFp32   ? kernel_fp32(g->head_dim, nt)
         : kind == kE4m3 ? kernel_e4m3(g->head_dim, nt)
                         : kernel_bf16(g->head_dim, nt);
}

int kind_of(const mla_kv_geometry_t* g) {
  return g->dtype == MLA_DTYPE_FP32 ? kFp32 : g->cache_dtype == MLA_DTYPE_E4M3 ? kE4m3 : kBf16;
}

// The plan with `hg` key/value heads to a tile.
mla_status_t plan_for(const mla_kv_geometry_t* g, int32_t batch, int32_t page_size,
                      int32_t max_pages, int hg, Plan* out) {
  Plan& d = *out;
  d.kind = kind_of(g);
  const int group = g->num_heads / g->num_kv_heads;
  d.k = kernel_of(g, d.kind);
  d.row_tiles = (group + d.k.rows - 1) / d.k.rows;
  d.hg = hg;
  d.pw = d.k.warps / hg;
  d.tile = d.pw * d.k.wp;
  d.kv_groups = g->num_kv_heads / hg;
  const int64_t hrs = (int64_t)d.kv_groups * d.row_tiles;
  const int64_t tiles = ((int64_t)page_size * max_pages + d.tile - 1) / d.tile;
  const int64_t most = (int64_t)batch * hrs * tiles;
  if (most > ((int64_t)1 << 48)) {
    set_error("decode: batch %d x %lld rows of a table is beyond what is planned for", batch,
              (long long)page_size * max_pages);
    return MLA_ERR_UNSUPPORTED;
  }
  int64_t ctas = (int64_t)device_sm_count() * d.k.occupancy;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  if (ctas > most) ctas = most;
  d.ctas = (int)ctas;
  d.cut = tiles > 1;
  d.by_segment = batch * hrs <= ctas;
  d.records = d.by_segment ? (int)(batch * hrs) : (int)ctas;
  const size_t rows = (size_t)2 * ctas * hg * d.k.rows;
  size_t off = align256(sizeof(Record) * d.records);
  d.off_ml = off;
  off = align256(off + sizeof(float2) * rows);
  d.off_o = off;
  off = align256(off + sizeof(float) * rows * d.k.dp);
  d.bytes = d.cut ? off : 0;
  return MLA_OK;
}

// Whether a tile may hold `hg` heads: they share its warps evenly, and the
// kernel keeps a head's queries per warp (fp32 keeps them per CTA).
bool heads_fit(const mla_kv_geometry_t* g, int hg) {
  const int kind = kind_of(g);
  const Kernel k = kernel_of(g, kind);
  return hg == 1 || (k.fn_heads != nullptr && g->num_kv_heads % hg == 0 && k.warps % hg == 0);
}

// Heads that lie side by side in a cache row and are no whole 128-byte lines
// share lines with their neighbours, whose CTAs come by at another time: the
// lines are fetched again (heads of 80 in bf16: 637 MB for 437).  And single
// lines a row apart come from DRAM slower than two at a time.  So a tile takes
// as many neighbouring heads as make whole lines, two at least, a warp or two
// each (32 sequences of 1024 to 32768: 80 wide 327 -> 223 us, 96 wide 329 ->
// 259, 64 wide 187 -> 172; e4m3, 64 sequences: 64 wide 146 -> 102, 128 wide in
// groups of 4 165 -> 160), if the cache is beyond what L2 keeps between two
// heads: the merge and the join have more to do, and below that the lines are
// found in L2 (16 sequences of up to 4099, 80 wide, found there: 22.5 us with one
// head to a tile, 24.7 with four).  The lengths are known on the GPU only: short
// sequences in a large pool with wide tables take the larger merges as well (32
// of 100 positions, 80 wide: 13.8 us against 11.9).
mla_status_t make_plan(const mla_kv_geometry_t* g, const mla_kv_cache_t* cache, int32_t batch,
                       int32_t max_pages, Plan* out) {
  const mla_status_t st = plan_for(g, batch, cache->page_size, max_pages, 1, out);
  constexpr int64_t kLine = 128, kRun = 256;
  constexpr double kLarge = 256.0 * 1024 * 1024;
  const int64_t piece = (int64_t)g->head_dim * (g->cache_dtype == MLA_DTYPE_E4M3   ? 1
                                                : g->cache_dtype == MLA_DTYPE_FP32 ? 4
                                                                                   : 2);
  // what the call can read: the tables' pages, and no more than the pool has
  int64_t pages = (int64_t)batch * max_pages;
  if (pages > cache->num_pages) pages = cache->num_pages;
  const double bytes = 2.0 * piece * g->num_kv_heads * cache->page_size * pages;
  auto whole = [&](int64_t run) { return run % kLine == 0 && run >= kRun; };
  if (st != MLA_OK || !out->cut || whole(piece) || bytes < kLarge ||
      cache->head_stride >= cache->row_stride)
    return st;
  int hg = 1;
  while (hg < 4 && !whole(hg * piece) && heads_fit(g, 2 * hg)) hg *= 2;
  return hg == 1 ? st : plan_for(g, batch, cache->page_size, max_pages, hg, out);
}

// Allow a kernel its shared memory, once per kernel and device.
cudaError_t allow_smem(const Kernel& k, void (*fn)(Params)) {
  struct Done {
    int device;
    void (*fn)(Params);
  };
  constexpr int kMost = 512;
  static std::mutex mu;
  static Done done[kMost];
  static int count = 0;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < count; ++i)
    if (done[i].device == dev && done[i].fn == fn) return cudaSuccess;
  e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
  if (e == cudaSuccess && count < kMost) done[count++] = {dev, fn};
  return e;
}

cudaError_t launch(const Plan& d, const Params& p, cudaStream_t stream) {
  void (*fn)(Params) = d.hg > 1 ? d.k.fn_heads : d.k.fn;
  cudaError_t e = allow_smem(d.k, fn);
  if (e != cudaSuccess) return e;
  {
    KernelTimer kt("decode_attn", stream);
    e = launch_dependent(fn, dim3((unsigned)d.ctas), dim3(d.k.warps * 32), d.k.smem, stream, p);
  }
  if (e != cudaSuccess || !d.cut) return e;
  const int live = p.group < d.k.rows ? p.group : d.k.rows, rows = live * d.hg;
  KernelTimer kt("decode_join", stream);
  if (d.by_segment)
    return launch_dependent(decode_join_kernel<kJoinThreads>,
                            dim3((unsigned)d.records, (unsigned)rows), dim3(kJoinThreads), 0,
                            stream, p, d.ctas, d.k.rows, live, d.k.dp, d.kind);
  return launch_dependent(
      decode_join_kernel<64>,
      dim3((unsigned)d.records, (unsigned)((rows * 64 + kJoinThreads - 1) / kJoinThreads)),
      dim3(kJoinThreads), 0, stream, p, d.ctas, d.k.rows, live, d.k.dp, d.kind);
}

}  // namespace
}  // namespace decode

static mla_status_t decode_sizes_ok(const mla_kv_geometry_t* g, int32_t batch, int32_t page_size,
                                    int32_t max_pages) {
  const mla_status_t st = kv_geometry_ok(g);
  if (st != MLA_OK) return st;
  if (batch < 1 || batch > 65535 || page_size < 1 || max_pages < 1 ||
      (int64_t)page_size * max_pages > INT_MAX - 1023) {
    set_error("decode: need 1 <= batch <= 65535, page_size and max_pages_per_seq >= 1 with at "
              "most 2^31 - 1024 rows between them (batch=%d page_size=%d max_pages=%d)",
              batch, page_size, max_pages);
    return MLA_ERR_INVALID_ARG;
  }
  return MLA_OK;
}

}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_decode_workspace_bytes(const mla_kv_geometry_t* g, int32_t batch,
                                                   int32_t page_size, int32_t max_pages_per_seq,
                                                   size_t* bytes) {
  if (bytes == nullptr) {
    set_error("bytes output is NULL");
    return MLA_ERR_INVALID_ARG;
  }
  const mla_status_t st = decode_sizes_ok(g, batch, page_size, max_pages_per_seq);
  if (st != MLA_OK) return st;
  // the cache's layout decides how many heads a tile holds: room for each
  *bytes = 0;
  for (int hg = 1; hg <= 4; hg *= 2) {
    if (!decode::heads_fit(g, hg)) continue;
    decode::Plan d;
    const mla_status_t pst = decode::plan_for(g, batch, page_size, max_pages_per_seq, hg, &d);
    if (pst != MLA_OK) return pst;
    if (d.bytes > *bytes) *bytes = d.bytes;
  }
  return MLA_OK;
}

extern "C" mla_status_t mla_decode_attention(
    const mla_kv_geometry_t* g, const void* q, int64_t q_row_stride, const mla_kv_cache_t* cache,
    const int32_t* cache_lens, int32_t batch, const int32_t* page_table,
    int32_t max_pages_per_seq, int32_t window, void* out, float* lse, void* workspace,
    size_t workspace_bytes, void* stream) {
  mla_status_t st = kv_geometry_ok(g);
  if (st != MLA_OK) return st;
  st = kv_cache_ok(g, cache);
  if (st != MLA_OK) return st;
  st = decode_sizes_ok(g, batch, cache->page_size, max_pages_per_seq);
  if (st != MLA_OK) return st;
  if (window < 0) {
    set_error("decode: window %d is negative", window);
    return MLA_ERR_INVALID_ARG;
  }
  const void* ptrs[] = {q, cache_lens, page_table, out};
  const char* names[] = {"q", "cache_lens", "page_table", "out"};
  for (int i = 0; i < 4; ++i) {
    if (ptrs[i] == nullptr || ((uintptr_t)ptrs[i] & 15u)) {
      set_error("decode: %s is NULL or not 16-byte aligned", names[i]);
      return MLA_ERR_INVALID_ARG;
    }
  }
  if ((uintptr_t)lse & 3u) {
    set_error("decode: lse is not 4-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  const int eb = g->dtype == MLA_DTYPE_BF16 ? 2 : 4;
  if (q_row_stride < (int64_t)g->num_heads * g->head_dim || q_row_stride * eb % 16 != 0) {
    set_error("decode: q_row_stride %lld must be at least %lld and a multiple of 16 bytes",
              (long long)q_row_stride, (long long)g->num_heads * g->head_dim);
    return MLA_ERR_INVALID_ARG;
  }
  // in place only row for row: a head's queries are used by the CTA that writes its
  // output, or by those whose parts the join, behind all of them, puts there
  const int64_t row = (int64_t)g->num_heads * g->head_dim;
  const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)out;
  const uintptr_t q1 = q0 + (uintptr_t)(((batch - 1) * q_row_stride + row) * eb);
  const uintptr_t o1 = o0 + (uintptr_t)(batch * row * eb);
  if (q0 < o1 && o0 < q1 && !(q == out && q_row_stride == row)) {
    set_error("decode: out overlaps q without being q");
    return MLA_ERR_INVALID_ARG;
  }
  decode::Plan d;
  st = decode::make_plan(g, cache, batch, max_pages_per_seq, &d);
  if (st != MLA_OK) return st;
  size_t need = 0;
  st = mla_decode_workspace_bytes(g, batch, cache->page_size, max_pages_per_seq, &need);
  if (st != MLA_OK) return st;
  if (workspace_bytes < need || (need > 0 && workspace == nullptr)) {
    set_error("workspace of %zu bytes is smaller than the %zu this call needs", workspace_bytes,
              need);
    return MLA_ERR_WORKSPACE;
  }
  if ((uintptr_t)workspace & 255u) {
    set_error("workspace is not 256-byte aligned");
    return MLA_ERR_INVALID_ARG;
  }
  decode::Params p;
  p.q = q;
  p.q_stride = q_row_stride;
  p.k = cache->k;
  p.v = cache->v;
  p.page_stride = cache->page_stride;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.lens = cache_lens;
  p.table = page_table;
  p.out = out;
  p.lse = lse;
  p.rec = d.cut ? (decode::Record*)workspace : nullptr;
  p.by_segment = d.by_segment ? 1 : 0;
  p.part_ml = d.cut ? (float2*)((char*)workspace + d.off_ml) : nullptr;
  p.part_o = d.cut ? (float*)((char*)workspace + d.off_o) : nullptr;
  p.heads = g->num_heads;
  p.kv_groups = d.kv_groups;
  p.hg = d.hg;
  p.pw = d.pw;
  p.tile = d.tile;
  p.tile_div = PageDiv(d.tile);
  p.group = g->num_heads / g->num_kv_heads;
  p.row_tiles = d.row_tiles;
  p.dim = g->head_dim;
  p.batch = batch;
  p.page = cache->page_size;
  p.div = PageDiv(cache->page_size);
  p.width = max_pages_per_seq;
  p.num_pages = cache->num_pages;
  p.window = window;
  const double scale = g->softmax_scale > 0.f ? (double)g->softmax_scale
                                              : 1.0 / std::sqrt((double)g->head_dim);
  p.scale_log2 = (float)(scale * 1.4426950408889634);
  const cudaError_t e = decode::launch(d, p, (cudaStream_t)stream);
  if (e != cudaSuccess) {
    set_error("CUDA error %d (%s)", (int)e, cudaGetErrorString(e));
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}
