// Attention of one new token per sequence over a paged key/value cache
// (mla_decode_attention): the drafter's decode step.
//
//   s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// One pass over the cache with the running maximum m and sum: a CTA takes one
// query head of one sequence, a warp every fourth position, the lanes the
// head's elements.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <climits>
#include <cmath>

#include "mla_internal.h"

namespace mla {

static __device__ int g_decode_status;

int decode_device_status(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_decode_status, &z, sizeof(int)) != cudaSuccess) return -1;
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

namespace {

struct DecodeParams {
  const void* q;
  int64_t q_stride;
  const void *k, *v;
  int64_t page_stride, row_stride, head_stride;
  const float *k_scale, *v_scale;
  const int32_t* lens;
  const int32_t* table;
  void* out;
  float* lse;
  int heads, kv_heads, dim, batch, page, width, num_pages, window;
  float scale;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__nv_fp8_e4m3 x) { return (float)x; }
__device__ __forceinline__ void from_float(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

constexpr int kPerLane = 8;  // head_dim <= 256

template <typename T, typename CT>
__global__ void __launch_bounds__(128) decode_rows_kernel(DecodeParams p) {
  __shared__ float s_m[4], s_l[4], s_o[4][256];
  const int h = blockIdx.x, b = blockIdx.y, hk = h / (p.heads / p.kv_heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T_b = (int)min((long long)max(p.lens[b], 0), (long long)p.width * p.page);
  const int lo = p.window > 0 ? max(0, T_b - p.window) : 0;
  float q[kPerLane], o[kPerLane];
  const float ks = p.k_scale ? p.k_scale[hk] : 1.f, vs = p.v_scale ? p.v_scale[hk] : 1.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.dim ? to_float(((const T*)p.q)[b * p.q_stride + (int64_t)h * p.dim + d]) : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = lo + warp; t < T_b; t += 4) {
    const int id = p.table[(int64_t)b * p.width + t / p.page];
    const bool good = id >= 0 && id < p.num_pages;
    if (!good && lane == 0) atomicCAS(&g_decode_status, 0, kBadPageSite);
    const int64_t at = good ? id * p.page_stride + (int64_t)(t % p.page) * p.row_stride +
                                  hk * p.head_stride
                            : 0;
    float s = 0.f, v[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int d = lane + 32 * i;
      const bool live = good && d < p.dim;
      s = fmaf(q[i], live ? to_float(((const CT*)p.k)[at + d]) : 0.f, s);
      v[i] = live ? to_float(((const CT*)p.v)[at + d]) : 0.f;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= p.scale * ks;
    const float m2 = fmaxf(m, s);
    const float base = m2 == -INFINITY ? 0.f : m2;
    const float f = __expf(m - base), w = __expf(s - base);
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) o[i] = o[i] * f + w * v[i];
    m = m2;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f, f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = __expf(s_m[w] - base);
    L += f[w] * s_l[w];
  }
  for (int d = threadIdx.x; d < p.dim; d += 128) {
    float acc = 0.f;
    for (int w = 0; w < 4; ++w) acc += f[w] * s_o[w][d];
    from_float(L == 0.f ? 0.f : acc / L * vs,
               (T*)p.out + ((int64_t)b * p.heads + h) * p.dim + d);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(int64_t)b * p.heads + h] = L == 0.f ? -INFINITY : base + logf(L);
}

}  // namespace

static mla_status_t decode_sizes_ok(const mla_kv_geometry_t* g, int32_t batch, int32_t page_size,
                                    int32_t max_pages) {
  const mla_status_t st = kv_geometry_ok(g);
  if (st != MLA_OK) return st;
  if (batch < 1 || batch > 65535 || page_size < 1 || max_pages < 1 ||
      (int64_t)page_size * max_pages > INT_MAX) {
    set_error("decode: need 1 <= batch <= 65535, page_size and max_pages_per_seq >= 1 with at "
              "most 2^31 - 1 rows between them (batch=%d page_size=%d max_pages=%d)",
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
  *bytes = 0;
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
  DecodeParams p;
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
  p.heads = g->num_heads;
  p.kv_heads = g->num_kv_heads;
  p.dim = g->head_dim;
  p.batch = batch;
  p.page = cache->page_size;
  p.width = max_pages_per_seq;
  p.num_pages = cache->num_pages;
  p.window = window;
  p.scale = g->softmax_scale > 0.f ? g->softmax_scale
                                   : (float)(1.0 / std::sqrt((double)g->head_dim));
  const cudaStream_t s = (cudaStream_t)stream;
  const dim3 grid((unsigned)p.heads, (unsigned)batch);
  {
    KernelTimer kt("decode_rows", s);
    if (eb == 4)
      decode_rows_kernel<float, float><<<grid, 128, 0, s>>>(p);
    else if (g->cache_dtype == MLA_DTYPE_E4M3)
      decode_rows_kernel<__nv_bfloat16, __nv_fp8_e4m3><<<grid, 128, 0, s>>>(p);
    else
      decode_rows_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 128, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("CUDA error %d (%s)", (int)e, cudaGetErrorString(e));
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}
