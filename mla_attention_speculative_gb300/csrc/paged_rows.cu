// The paged-cache side of a serving step: page tables and slots built on the
// GPU (mla_page_step), and the step's rows written into the latent cache
// (mla_append_latent) or a key/value cache (mla_append_kv).
//
// None of these triggers the next kernel early, so a verify or decode call
// that follows (and may read the cache before its own wait) starts after the
// rows are in place.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <climits>
#include <type_traits>

#include "mla_internal.h"
#include "sm103_ptx.cuh"

namespace mla {

static __device__ int g_paged_status;

int paged_device_status(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_paged_status, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

namespace {

// ---------------------------------------------------------------------------
// Page step
// ---------------------------------------------------------------------------
//
// Two exclusive sums over the sequences (rows, pages asked for) place every
// row and every new page; the rest is one lookup each.  A CTA computes the
// sums itself, a run of sequences per thread, so no CTA waits for another: the
// counts (12 bytes a sequence) stay in L2, and a step has far more rows than
// sequences or is bound by latency anyway.  The sums of up to 4096 sequences
// (beyond: of groups of sequences) stay in shared memory, where each row, each
// new page and each sequence, dealt out evenly over all threads, finds its
// place by a binary search.  New pages are read from the free list by
// position, never from the table that this launch writes.

constexpr int kEntries = 4096;  // sums kept in shared memory

struct PageStepParams {
  const int32_t* kept;
  const int32_t* fresh;
  const int32_t* held;
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* free_span;
  int32_t* lens_out;
  int32_t* held_out;
  int32_t* row_start;
  int32_t* positions;
  int64_t* slots;
  int32_t* span_out;
  int32_t* missing;
  int batch, width, page, num_pages, free_capacity, max_rows;
  int capacity;  // rows of a table's pages, INT_MAX at most
  int rows_per_cta;
  PageDiv div;
};

struct Sums {
  long long rows;
  int pages;  // (batch * width < 2^31)
};

__device__ __forceinline__ int sat32(long long x) { return x > INT_MAX ? INT_MAX : (int)x; }

// One sequence: its clamped counts, the pages it asks for, and (once the sums
// before it are known) what it gets.
struct Sequence {
  int kept, fresh, held, total, grow;
  __device__ __forceinline__ void load(const PageStepParams& p, int b) {
    set(p, p.kept[b], p.fresh[b], p.held[b]);
  }
  __device__ __forceinline__ void set(const PageStepParams& p, int k, int f, int h) {
    kept = max(k, 0);
    fresh = max(f, 0);
    held = min(max(h, 0), p.width);
    total = (int)min((uint32_t)kept + (uint32_t)fresh, (uint32_t)p.capacity);
    grow = total > 0 ? max(0, p.div(total - 1) + 1 - held) : 0;
  }
  __device__ __forceinline__ int got(int have, int pages) const {
    return min(grow, max(0, have - pages));
  }
};

__device__ __forceinline__ void load4(const int32_t* p, int (&x)[4]) {
  const int4 v = *reinterpret_cast<const int4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// The last of n ascending sums that is at or before x.
__device__ __forceinline__ int find_entry(const int* sums, int n, int x) {
  int a = 0, z = n;
  while (z - a > 1) {
    const int m = (a + z) >> 1;
    if (sums[m] <= x) a = m; else z = m;
  }
  return a;
}

// ROWS: consecutive rows a thread places at a time.
template <int THREADS, int ROWS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    page_step_kernel(const PageStepParams p) {
  // before each entry's sequences (rows saturate: no row that is wanted lies there)
  __shared__ int s_row[kEntries], s_page[kEntries];
  __shared__ Sums s_warp[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm103::pdl_wait();
  const int span0 = p.free_span[0], span1 = p.free_span[1];

  // ---- the sums; `per` consecutive sequences a thread, `size` an entry
  const int size = (p.batch + kEntries - 1) / kEntries;
  const int per = ((p.batch + THREADS - 1) / THREADS + size - 1) / size * size;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  Sums mine = {0, 0};
  Sequence q;
  int b = b0;
  if (per % 4 == 0) {
    for (; b + 4 <= b1; b += 4) {
      int k[4], f[4], h[4];
      load4(p.kept + b, k);
      load4(p.fresh + b, f);
      load4(p.held + b, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q.set(p, k[i], f[i], h[i]);
        mine.rows += q.fresh;
        mine.pages += q.grow;
      }
    }
  }
  for (; b < b1; ++b) {
    q.load(p, b);
    mine.rows += q.fresh;
    mine.pages += q.grow;
  }
  Sums sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long r = __shfl_up_sync(~0u, sum.rows, o);
    const int g = __shfl_up_sync(~0u, sum.pages, o);
    if (lane >= o) {
      sum.rows += r;
      sum.pages += g;
    }
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  Sums all = {0, 0};
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const Sums x = s_warp[w];
    if (w < warp) {
      sum.rows += x.rows;
      sum.pages += x.pages;
    }
    all.rows += x.rows;
    all.pages += x.pages;
  }
  {
    Sums base = {sum.rows - mine.rows, sum.pages - mine.pages};
    int e = b0 / size, b = b0;
    if (size == 1 && per % 4 == 0) {
      for (; b + 4 <= b1; b += 4) {
        int k[4], f[4], h[4];
        load4(p.kept + b, k);
        load4(p.fresh + b, f);
        load4(p.held + b, h);
#pragma unroll
        for (int i = 0; i < 4; ++i, ++e) {
          s_row[e] = sat32(base.rows);
          s_page[e] = base.pages;
          q.set(p, k[i], f[i], h[i]);
          base.rows += q.fresh;
          base.pages += q.grow;
        }
      }
    }
    for (; b < b1; b += size, ++e) {
      s_row[e] = sat32(base.rows);
      s_page[e] = base.pages;
      if (per == 1) break;
      for (int i = 0; i < size && b + i < b1; ++i) {
        q.load(p, b + i);
        base.rows += q.fresh;
        base.pages += q.grow;
      }
    }
  }
  __syncthreads();
  const int entries = (p.batch + size - 1) / size;
  const int first = min(max(span0, 0), p.free_capacity);
  const int end = min(max(span1, first), p.free_capacity);
  const int have = end - first;

  // ---- this CTA's rows
  const long long r0 = (long long)blockIdx.x * p.rows_per_cta;
  const long long r1 = min(r0 + p.rows_per_cta, (long long)p.max_rows);
  for (long long g = r0 + tid * ROWS; g < r1; g += THREADS * ROWS) {
    int pos_of[ROWS], id_of[ROWS], off_of[ROWS];
    const int live = (int)max(0ll, min((long long)ROWS, all.rows - g));
    int b = -1;
    long long rows = 0;  // the sums before sequence b
    int pages = 0;
    auto next = [&]() {
      rows += q.fresh;
      pages += q.grow;
      q.load(p, ++b);
    };
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      pos_of[i] = -1;
      id_of[i] = -1;
      off_of[i] = -1;  // no page
      if (i >= live) continue;
      // the row before's sequence or the next one; else a search, so that a run of idle
      // slots costs no more than its entry's (one by one, 1022 of them between two
      // sequences of three rows took 60 us)
      bool found = i > 0;
      if (found && g + i >= rows + q.fresh) {
        next();
        found = g + i < rows + q.fresh;
      }
      if (!found) {
        const int e = find_entry(s_row, entries, (int)g + i);
        if (e * size > b) {
          b = e * size;
          rows = s_row[e];
          pages = s_page[e];
          q.load(p, b);
        }
        while (g + i >= rows + q.fresh) next();
      }
      const int owned = q.held + q.got(have, pages);
      const long long pos = q.kept + (g + i - rows);
      pos_of[i] = sat32(pos);
      if (pos >= q.total) continue;
      const int page = p.div((int)pos);
      if (page < owned) {
        off_of[i] = (int)pos - page * p.page;
        id_of[i] = page < q.held ? p.table[(long long)b * p.width + page]
                               : p.free_pages[first + pages + (page - q.held)];
      }
    }
    long long slot_of[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      slot_of[i] = -1;
      if (off_of[i] < 0) continue;
      if (id_of[i] >= 0 && id_of[i] < p.num_pages) slot_of[i] = (long long)id_of[i] * p.page + off_of[i];
      else atomicCAS(&g_paged_status, 0, kBadPageSite);
    }
    if constexpr (ROWS == 4) {
      if (g + ROWS <= r1) {
        *reinterpret_cast<int4*>(p.positions + g) = make_int4(pos_of[0], pos_of[1], pos_of[2], pos_of[3]);
        longlong2* d = reinterpret_cast<longlong2*>(p.slots + g);
        d[0] = make_longlong2(slot_of[0], slot_of[1]);
        d[1] = make_longlong2(slot_of[2], slot_of[3]);
        continue;
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (g + i >= r1) continue;
      p.positions[g + i] = pos_of[i];
      p.slots[g + i] = slot_of[i];
    }
  }

  // ---- new table entries
  const int taken = min(all.pages, have);
  // (unsigned: a grid's stride beyond `taken`, which may be close to 2^31)
  for (uint32_t at_free = blockIdx.x * THREADS + tid; at_free < (uint32_t)taken;
       at_free += gridDim.x * THREADS) {
    const int i = (int)at_free, e = find_entry(s_page, entries, i);
    int b = e * size;
    int at = s_page[e];
    q.load(p, b);
    while (i >= at + q.grow) {
      at += q.grow;
      q.load(p, ++b);
    }
    p.table[(long long)b * p.width + q.held + (i - at)] = p.free_pages[first + i];
  }

  // ---- per sequence
  for (int b = blockIdx.x * THREADS + tid; b < p.batch; b += gridDim.x * THREADS) {
    const int e = b / size;
    long long rows = s_row[e];
    int pages = s_page[e];
    for (int x = e * size; x < b; ++x) {
      q.load(p, x);
      rows += q.fresh;
      pages += q.grow;
    }
    q.load(p, b);
    const int owned = q.held + q.got(have, pages);
    p.held_out[b] = owned;
    p.lens_out[b] = (int)min((long long)q.total, (long long)owned * p.page);
    p.row_start[b] = sat32(rows);
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.row_start[p.batch] = sat32(all.rows);
    p.span_out[0] = first + taken;
    p.span_out[1] = end;
    p.missing[0] = all.pages - taken;
  }
}

// ---------------------------------------------------------------------------
// Rows into the caches
// ---------------------------------------------------------------------------
//
// Both appends only move data (a row's heads in, the same bytes out, a few
// multiplications between), so they are bound by memory: 16383 rows of 48
// heads of 128 61 us, 6.75 TB/s; 8191 latent rows of 32 heads 48 us, 6.0 TB/s
// (256 of 128 heads 4.8 us, 5.4 TB/s).  A thread moves two
// 16-byte vectors at a time: the two that a rotation mixes (vector i and i +
// half of the rotated part, or two neighbours when pairs are interleaved), so
// the rotation needs no exchange between threads and reads the same run of
// cosines and sines in both forms.  A thread keeps its place within the head
// and walks over heads, so the row's cosines and sines are loaded once.

template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  float v[N];
};

__device__ __forceinline__ void store_vec(float* p, const Vec<float>& x) {
  *reinterpret_cast<float4*>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const Vec<__nv_bfloat16>& x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.v[2 * i], x.v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// Eight values as e4m3, saturating (NaN stays NaN).
__device__ __forceinline__ void store_vec(__nv_fp8_e4m3* p, const Vec<__nv_bfloat16>& x) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.v[4 * i], x.v[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.v[4 * i + 2], x.v[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint4 load_raw(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void unpack(const uint4& r, Vec<float>& x) {
  x.v[0] = __uint_as_float(r.x);
  x.v[1] = __uint_as_float(r.y);
  x.v[2] = __uint_as_float(r.z);
  x.v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, Vec<__nv_bfloat16>& x) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.v[2 * i] = __uint_as_float(w[i] << 16);
    x.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The cosines and sines of one item: Vec::N angles.
template <typename T>
struct Angles {
  static constexpr int N = Vec<T>::N;
  float c[N], s[N];
  __device__ __forceinline__ void load(const float* table, long long row, int rope, int item) {
    const float* p = table + row * rope + item * N;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + i);
      const float4 b = *reinterpret_cast<const float4*>(p + rope / 2 + i);
      c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
      s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
    }
  }
  __device__ __forceinline__ void turn(Vec<T>& x, Vec<T>& y, bool interleaved) const {
    if (interleaved) {  // pairs within the two neighbouring vectors
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Vec<T>& z = i < N / 2 ? x : y;
        const int k = 2 * (i % (N / 2));
        const float a = z.v[k], b = z.v[k + 1];
        z.v[k] = fmaf(a, c[i], -(b * s[i]));
        z.v[k + 1] = fmaf(b, c[i], a * s[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float a = x.v[i], b = y.v[i];
        x.v[i] = fmaf(a, c[i], -(b * s[i]));
        y.v[i] = fmaf(b, c[i], a * s[i]);
      }
    }
  }
};

// The two vectors of item i of a head: `turned` rotated items first (the
// rotated part starts at vector `rot0`), then pairs of the `rest` others from
// vector `rest0`.  v1 < 0: the item has one vector only.
__device__ __forceinline__ void item_vectors(int i, int turned, int rot0, int rest0, int rest,
                                             bool interleaved, int& v0, int& v1) {
  if (i < turned) {
    v0 = rot0 + (interleaved ? 2 * i : i);
    v1 = interleaved ? v0 + 1 : v0 + turned;
  } else {
    const int j = 2 * (i - turned);
    v0 = rest0 + j;
    v1 = j + 1 < rest ? v0 + 1 : -1;
  }
}

struct AppendKVParams {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  void* q_out;
  void *k_cache, *v_cache;
  int64_t page_stride, row_stride, head_stride, cache_rows;
  const float *k_scale, *v_scale;
  int page, table_rows, rope, interleaved;
  int q_heads, kv_heads, dim;  // q_heads 0: the cache only
  int items, turned;
  PageDiv div;
};

template <typename T, typename CT, int K>
__global__ void __launch_bounds__(256) append_kv_kernel(const AppendKVParams p) {
  constexpr int N = Vec<T>::N;
  sm103::pdl_wait();
  const long long row = blockIdx.x;
  const int pos = p.positions[row];
  const int64_t slot = p.slots[row];
  const int item = threadIdx.x;
  int v0, v1;
  item_vectors(item, p.turned, 0, 2 * p.turned, p.dim / N - 2 * p.turned, p.interleaved != 0, v0,
               v1);
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int h0 = blockIdx.y * (K * blockDim.y) + threadIdx.y;
  uint4 xr[K], yr[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int h = h0 + i * blockDim.y;
    xr[i] = yr[i] = make_uint4(0u, 0u, 0u, 0u);
    if (h >= heads) continue;
    const int hk = h - p.q_heads;
    const T* src = hk < 0             ? (const T*)p.q + row * p.q_stride + (int64_t)h * p.dim
                   : hk < p.kv_heads ? (const T*)p.k + row * p.k_stride + (int64_t)hk * p.dim
                                     : (const T*)p.v + row * p.v_stride +
                                           (int64_t)(hk - p.kv_heads) * p.dim;
    xr[i] = load_raw(src + v0 * N);
    if (v1 >= 0) yr[i] = load_raw(src + v1 * N);
  }
  if (pos < 0 || (p.rope > 0 && pos >= p.table_rows)) return;
  const bool cached = slot >= 0 && slot < p.cache_rows;
  int64_t at = 0;
  if (cached) {
    const int64_t pg = (slot >> 31) == 0 ? (int64_t)p.div((int)slot) : slot / p.page;
    at = pg * p.page_stride + (slot - pg * p.page) * p.row_stride;
  }
  Angles<T> ang;
  if (item < p.turned) ang.load(p.cos_sin, pos, p.rope, item);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int h = h0 + i * blockDim.y;
    if (h >= heads) continue;
    const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
    if (!is_q && !cached) continue;
    Vec<T> x, y;
    unpack(xr[i], x);
    unpack(yr[i], y);
    if (item < p.turned && !is_v) ang.turn(x, y, p.interleaved != 0);
    if (is_q) {
      T* dst = (T*)p.q_out + (row * p.q_heads + h) * p.dim;
      store_vec(dst + v0 * N, x);
      if (v1 >= 0) store_vec(dst + v1 * N, y);
    } else {
      const int hk = h - p.q_heads - (is_v ? p.kv_heads : 0);
      CT* dst = (CT*)(is_v ? p.v_cache : p.k_cache) + at + hk * p.head_stride;
      if constexpr (sizeof(CT) == 1) {
        const float* sc = is_v ? p.v_scale : p.k_scale;
        if (sc) {
          const float s = sc[hk];
#pragma unroll
          for (int e = 0; e < N; ++e) {
            x.v[e] = __fdiv_rn(x.v[e], s);
            y.v[e] = __fdiv_rn(y.v[e], s);
          }
        }
      }
      store_vec(dst + v0 * N, x);
      if (v1 >= 0) store_vec(dst + v1 * N, y);
    }
  }
}

struct AppendLatentParams {
  const void *q, *kv, *weight;
  int64_t q_stride, kv_stride;
  float eps;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  void *q_nope, *q_rope, *c_kv, *k_rope;
  int64_t ckv_stride, kr_stride, cache_rows;
  int table_rows, interleaved;
  int heads, rank, nope, rope;
  int items, turned;
  int rows, kv_ctas, head_ctas;  // head_ctas of one row
};

// The first CTAs take the rows' latents and keys, a warp a row, so that the
// sum of squares needs no barrier (with a CTA a row these, mostly waiting,
// held half of the machine's places: 8191 rows took 62 us, now 48); the others
// a run of one row's query heads each.
template <typename T, int K>
__global__ void __launch_bounds__(256) append_latent_kernel(const AppendLatentParams p) {
  constexpr int N = Vec<T>::N;
  sm103::pdl_wait();
  if ((int)blockIdx.x >= p.kv_ctas) {
    const int cta = blockIdx.x - p.kv_ctas, run = cta % p.head_ctas;
    const long long row = cta / p.head_ctas;
    const int pos = p.positions[row];
    const int item = threadIdx.x;
    int v0, v1;
    item_vectors(item, p.turned, p.nope / N, 0, p.nope / N, p.interleaved != 0, v0, v1);
    const int h0 = run * (K * blockDim.y) + threadIdx.y;
    uint4 xr[K], yr[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int h = h0 + i * blockDim.y;
      xr[i] = yr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h >= p.heads) continue;
      const T* src = (const T*)p.q + row * p.q_stride + (int64_t)h * (p.nope + p.rope);
      xr[i] = load_raw(src + v0 * N);
      if (v1 >= 0) yr[i] = load_raw(src + v1 * N);
    }
    if (pos < 0 || pos >= p.table_rows) return;
    Angles<T> ang;
    if (item < p.turned) ang.load(p.cos_sin, pos, p.rope, item);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int h = h0 + i * blockDim.y;
      if (h >= p.heads) continue;
      const int64_t head = row * p.heads + h;
      if (item < p.turned) {
        Vec<T> x, y;
        unpack(xr[i], x);
        unpack(yr[i], y);
        ang.turn(x, y, p.interleaved != 0);
        T* dst = (T*)p.q_rope + head * p.rope - p.nope;
        store_vec(dst + v0 * N, x);
        store_vec(dst + v1 * N, y);
      } else {
        T* dst = (T*)p.q_nope + head * p.nope;
        *reinterpret_cast<uint4*>(dst + v0 * N) = xr[i];
        if (v1 >= 0) *reinterpret_cast<uint4*>(dst + v1 * N) = yr[i];
      }
    }
    return;
  }

  const int tid = threadIdx.y * blockDim.x + threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int warps = (blockDim.x * blockDim.y) >> 5;  // (whole ones)
  const long long row = (long long)blockIdx.x * warps + warp;
  if (warp >= warps || row >= p.rows) return;
  const int pos = p.positions[row];
  const int64_t slot = p.slots[row];
  const T* src = (const T*)p.kv + row * p.kv_stride;
  const int nv = p.rank / N;
  // rank <= 1024 is at most 256 vectors, rope <= 128 at most 16 rotated items
  constexpr int kMost = 256 / 32 * (int)sizeof(T) / 4;
  uint4 x[kMost], w[kMost], ra, rb;
  int v0 = 0, v1 = 0;
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    const int i = lane + m * 32;
    x[m] = w[m] = make_uint4(0u, 0u, 0u, 0u);
    if (i >= nv) continue;
    x[m] = load_raw(src + i * N);
    if (p.weight) w[m] = load_raw((const T*)p.weight + i * N);
  }
  if (lane < p.turned) {
    item_vectors(lane, p.turned, nv, 0, 0, p.interleaved != 0, v0, v1);
    ra = load_raw(src + v0 * N);
    rb = load_raw(src + v1 * N);
  }
  if (pos < 0 || pos >= p.table_rows || slot < 0 || slot >= p.cache_rows) return;
  T* c = (T*)p.c_kv + slot * p.ckv_stride;
  if (lane < p.turned) {
    T* kr = (T*)p.k_rope + slot * p.kr_stride;
    Angles<T> ang;
    ang.load(p.cos_sin, pos, p.rope, lane);
    Vec<T> a, b;
    unpack(ra, a);
    unpack(rb, b);
    ang.turn(a, b, p.interleaved != 0);
    store_vec(kr + (v0 - nv) * N, a);
    store_vec(kr + (v1 - nv) * N, b);
  }
  __syncwarp();
  if (p.weight == nullptr) {
#pragma unroll
    for (int m = 0; m < kMost; ++m)
      if (lane + m * 32 < nv) *reinterpret_cast<uint4*>(c + (lane + m * 32) * N) = x[m];
    return;
  }
  float sum = 0.f;
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    Vec<T> a;
    unpack(x[m], a);
#pragma unroll
    for (int e = 0; e < N; ++e) sum = fmaf(a.v[e], a.v[e], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const float scale = __frsqrt_rn(sum / p.rank + p.eps);
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    if (lane + m * 32 >= nv) continue;
    Vec<T> a, b;
    unpack(x[m], a);
    unpack(w[m], b);
#pragma unroll
    for (int e = 0; e < N; ++e) a.v[e] = a.v[e] * scale * b.v[e];
    store_vec(c + (lane + m * 32) * N, a);
  }
}

bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

struct Named {
  const void* p;
  const char* name;
  bool optional;
};

mla_status_t check_pointers(const char* what, const Named* list, int n) {
  for (int i = 0; i < n; ++i) {
    if (list[i].p == nullptr) {
      if (list[i].optional) continue;
      set_error("%s: %s is NULL", what, list[i].name);
      return MLA_ERR_INVALID_ARG;
    }
    if (misaligned(list[i].p)) {
      set_error("%s: %s is not 16-byte aligned", what, list[i].name);
      return MLA_ERR_INVALID_ARG;
    }
  }
  return MLA_OK;
}

mla_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  set_error("CUDA error %d (%s)", (int)e, cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

struct Range {
  uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) {
  return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)(p ? bytes : 0)};
}
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// Threads of an append: blockDim.x items of a head, blockDim.y heads.
dim3 item_block(int items) { return dim3((unsigned)items, (unsigned)(128 / items < 1 ? 1 : 128 / items)); }

// Heads a thread takes: one when the rows are few (the more CTAs the better),
// up to four, which share one load of the cosines and are on their way
// together, when there are enough rows to fill the machine anyway.
int heads_per_thread(int heads, int by, int rows) {
  const int64_t fill = (int64_t)device_sm_count() * 8;
  int k = 1;
  while (k < 4 && (int64_t)rows * ((heads + 2 * k * by - 1) / (2 * k * by)) >= fill) k *= 2;
  return k;
}

template <typename T>
cudaError_t launch_latent(int k, dim3 grid, dim3 block, cudaStream_t s,
                          const AppendLatentParams& p) {
  auto* fn = k == 4   ? append_latent_kernel<T, 4>
             : k == 2 ? append_latent_kernel<T, 2>
                      : append_latent_kernel<T, 1>;
  return launch_dependent(fn, grid, block, 0, s, p);
}

template <typename T, typename CT>
cudaError_t launch_kv(int k, dim3 grid, dim3 block, cudaStream_t s, const AppendKVParams& p) {
  auto* fn = k == 4   ? append_kv_kernel<T, CT, 4>
             : k == 2 ? append_kv_kernel<T, CT, 2>
                      : append_kv_kernel<T, CT, 1>;
  return launch_dependent(fn, grid, block, 0, s, p);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_page_step(
    const int32_t* kept_lens, const int32_t* new_tokens, const int32_t* held_pages, int32_t batch,
    int32_t* page_table, int32_t max_pages_per_seq, int32_t page_size, int32_t num_pages,
    const int32_t* free_pages, int32_t free_capacity, const int32_t* free_span,
    int32_t* cache_lens_out, int32_t* held_pages_out, int32_t* row_start_out,
    int32_t* positions_out, int64_t* slots_out, int32_t max_rows, int32_t* free_span_out,
    int32_t* missing_out, void* stream) {
  if (batch < 1 || batch > 65535 || max_pages_per_seq < 1 || page_size < 1 || num_pages < 1 ||
      free_capacity < 0 || max_rows < 0 || (int64_t)batch * max_pages_per_seq > INT_MAX) {
    set_error("page step: need 1 <= batch <= 65535, max_pages_per_seq, page_size and num_pages "
              ">= 1, batch * max_pages_per_seq < 2^31, free_capacity and max_rows >= 0 "
              "(batch=%d max_pages=%d page_size=%d num_pages=%d free=%d rows=%d)",
              batch, max_pages_per_seq, page_size, num_pages, free_capacity, max_rows);
    return MLA_ERR_INVALID_ARG;
  }
  const Named ptrs[] = {{kept_lens, "kept_lens", false},
                        {new_tokens, "new_tokens", false},
                        {held_pages, "held_pages", false},
                        {page_table, "page_table", false},
                        {free_pages, "free_pages", free_capacity == 0},
                        {free_span, "free_span", false},
                        {cache_lens_out, "cache_lens_out", false},
                        {held_pages_out, "held_pages_out", false},
                        {row_start_out, "row_start_out", false},
                        {positions_out, "positions_out", max_rows == 0},
                        {slots_out, "slots_out", max_rows == 0},
                        {free_span_out, "free_span_out", false},
                        {missing_out, "missing_out", false}};
  mla_status_t st = check_pointers("page step", ptrs, 13);
  if (st != MLA_OK) return st;
  const int64_t seqs = (int64_t)batch * 4;
  const Range in[] = {range(kept_lens, seqs), range(new_tokens, seqs), range(held_pages, seqs),
                      range(free_pages, (int64_t)free_capacity * 4), range(free_span, 8)};
  const Range out[] = {range(page_table, (int64_t)batch * max_pages_per_seq * 4),
                       range(cache_lens_out, seqs), range(held_pages_out, seqs),
                       range(row_start_out, seqs + 4), range(positions_out, (int64_t)max_rows * 4),
                       range(slots_out, (int64_t)max_rows * 8), range(free_span_out, 8),
                       range(missing_out, 4)};
  for (int i = 0; i < 8; ++i) {
    bool bad = false;
    for (const Range& r : in) bad = bad || overlap(out[i], r);
    for (int j = 0; j < i; ++j) bad = bad || overlap(out[i], out[j]);
    if (bad) {
      set_error("page step: an output overlaps another buffer of the call");
      return MLA_ERR_INVALID_ARG;
    }
  }
  PageStepParams p;
  p.kept = kept_lens;
  p.fresh = new_tokens;
  p.held = held_pages;
  p.table = page_table;
  p.free_pages = free_pages;
  p.free_span = free_span;
  p.lens_out = cache_lens_out;
  p.held_out = held_pages_out;
  p.row_start = row_start_out;
  p.positions = positions_out;
  p.slots = slots_out;
  p.span_out = free_span_out;
  p.missing = missing_out;
  p.batch = batch;
  p.width = max_pages_per_seq;
  p.page = page_size;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  p.max_rows = max_rows;
  p.div = PageDiv(page_size);
  p.capacity = (int)((int64_t)max_pages_per_seq * page_size > INT_MAX
                         ? INT_MAX
                         : (int64_t)max_pages_per_seq * page_size);
  // 256 threads, whose barriers are cheap, and a row a thread: up to 1024 sequences
  // whatever their rows, up to 4096 with four rows each.  (us in a graph, against 1024
  // threads and four rows a thread: 257 sequences of 1 and of 261 rows 3.9 and 4.1
  // against 6.9 and 8.2, 1024 3.9 and 6.7 against 7.7 and 8.9, 4096 of 4 rows 7.6
  // against 10.6.)  Beyond, 1024 threads, so that fewer CTAs make the sums of all
  // sequences, and four rows (4096 of 32 rows 10.2 against 17.7, of 261 rows 12.3
  // against 26.5; 2048 of 261 rows 9.7 against 11.4, but of 32 rows 9.8 against 5.6).
  const bool small = batch <= 1024 || (batch <= kEntries && max_rows <= 4 * (int64_t)batch);
  const int threads = small ? 256 : 1024;
  const int64_t per_pass = (int64_t)threads * (small ? 1 : 4);
  int64_t ctas = ((int64_t)max_rows + per_pass - 1) / per_pass;
  if (ctas < batch / threads) ctas = batch / threads;
  const int64_t most = (int64_t)device_sm_count() * (1024 / threads);
  if (ctas > most) ctas = most;
  if (ctas < 1) ctas = 1;
  const int64_t share = ((int64_t)max_rows + ctas - 1) / ctas;
  p.rows_per_cta = (int)((share + 3) / 4 * 4);
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("page_step", s);
  return launched(launch_dependent(small ? page_step_kernel<256, 1> : page_step_kernel<1024, 4>,
                                   dim3((unsigned)ctas), dim3(threads), 0, s, p));
}

extern "C" mla_status_t mla_append_latent(
    const mla_geometry_t* g, const void* q, int64_t q_row_stride, const void* kv,
    int64_t kv_row_stride, const void* norm_weight, float eps, const float* cos_sin,
    int32_t table_rows, int32_t interleaved, const int32_t* positions, const int64_t* slots,
    int32_t rows, void* q_nope, void* q_rope, void* c_kv, void* k_rope, int64_t c_kv_row_stride,
    int64_t k_rope_row_stride, int64_t cache_rows, void* stream) {
  if (!geometry_ok(g)) return MLA_ERR_INVALID_ARG;
  const int eb = g->dtype == MLA_DTYPE_BF16 ? 2 : 4;
  const int H = g->num_heads, r = g->kv_lora_rank, n = g->qk_nope_dim, d = g->rope_dim;
  if (d < 16 || d % 16 != 0) {
    set_error("append latent: rope_dim %d is not a positive multiple of 16", d);
    return MLA_ERR_INVALID_ARG;
  }
  if (rows < 0 || table_rows < 1 || cache_rows < 1 || !(eps >= 0.f)) {
    set_error("append latent: need rows >= 0, table_rows and cache_rows >= 1, eps >= 0 (rows=%d "
              "table_rows=%d cache_rows=%lld)", rows, table_rows, (long long)cache_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (rows == 0) return MLA_OK;
  const bool no_q = q == nullptr;
  const Named ptrs[] = {{q, "q", true},
                        {kv, "kv", false},
                        {norm_weight, "norm_weight", true},
                        {cos_sin, "cos_sin", false},
                        {positions, "positions", false},
                        {slots, "slots", false},
                        {q_nope, "q_nope", no_q},
                        {q_rope, "q_rope", no_q},
                        {c_kv, "c_kv", false},
                        {k_rope, "k_rope", false}};
  mla_status_t st = check_pointers("append latent", ptrs, 10);
  if (st != MLA_OK) return st;
  const int64_t strides[] = {q_row_stride, kv_row_stride, c_kv_row_stride, k_rope_row_stride};
  const int64_t least[] = {(int64_t)H * (n + d), r + d, r, d};
  const char* names[] = {"q_row_stride", "kv_row_stride", "c_kv_row_stride", "k_rope_row_stride"};
  for (int i = no_q ? 1 : 0; i < 4; ++i) {
    if (strides[i] < least[i] || strides[i] * eb % 16 != 0) {
      set_error("append latent: %s %lld must be at least %lld and a multiple of 16 bytes",
                names[i], (long long)strides[i], (long long)least[i]);
      return MLA_ERR_INVALID_ARG;
    }
  }
  AppendLatentParams p;
  p.q = q;
  p.kv = kv;
  p.weight = norm_weight;
  p.q_stride = q_row_stride;
  p.kv_stride = kv_row_stride;
  p.eps = eps;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.slots = slots;
  p.q_nope = q_nope;
  p.q_rope = q_rope;
  p.c_kv = c_kv;
  p.k_rope = k_rope;
  p.ckv_stride = c_kv_row_stride;
  p.kr_stride = k_rope_row_stride;
  p.cache_rows = cache_rows;
  p.table_rows = table_rows;
  p.interleaved = interleaved;
  p.heads = H;
  p.rank = r;
  p.nope = n;
  p.rope = d;
  const int N = 16 / eb;
  p.turned = d / 2 / N;
  p.items = p.turned + (n / N + 1) / 2;
  const dim3 block = item_block(p.items);
  const int k = heads_per_thread(H, (int)block.y, rows), hpc = k * (int)block.y;
  const int warps = (int)(block.x * block.y) / 32;
  p.rows = rows;
  p.kv_ctas = (int)(((int64_t)rows + warps - 1) / warps);
  p.head_ctas = (H + hpc - 1) / hpc;
  const int64_t ctas = p.kv_ctas + (no_q ? 0 : (int64_t)rows * p.head_ctas);
  if (ctas > INT_MAX) {
    set_error("append latent: %d rows of %d heads are too many for one call", rows, H);
    return MLA_ERR_UNSUPPORTED;
  }
  const dim3 grid((unsigned)ctas);
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("append_latent", s);
  return launched(eb == 2 ? launch_latent<__nv_bfloat16>(k, grid, block, s, p)
                          : launch_latent<float>(k, grid, block, s, p));
}

extern "C" mla_status_t mla_append_kv(
    const mla_kv_geometry_t* g, const void* q, int64_t q_row_stride, const void* k,
    int64_t k_row_stride, const void* v, int64_t v_row_stride, const float* cos_sin,
    int32_t table_rows, int32_t rope_dim, int32_t interleaved, const int32_t* positions,
    const int64_t* slots, int32_t rows, void* q_out, const mla_kv_cache_t* cache, void* stream) {
  mla_status_t st = kv_geometry_ok(g);
  if (st != MLA_OK) return st;
  st = kv_cache_ok(g, cache);
  if (st != MLA_OK) return st;
  const int eb = g->dtype == MLA_DTYPE_BF16 ? 2 : 4;
  const int H = g->num_heads, Hk = g->num_kv_heads, D = g->head_dim;
  if (rows < 0 || rope_dim < 0 || rope_dim > D || rope_dim % 16 != 0 ||
      (rope_dim > 0 && table_rows < 1)) {
    set_error("append kv: need rows >= 0, rope_dim a multiple of 16 up to head_dim, table_rows "
              ">= 1 with a rotation (rows=%d rope_dim=%d table_rows=%d)", rows, rope_dim,
              table_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (rows == 0) return MLA_OK;
  const bool no_q = q == nullptr;
  const Named ptrs[] = {{q, "q", true},
                        {k, "k", false},
                        {v, "v", false},
                        {cos_sin, "cos_sin", rope_dim == 0},
                        {positions, "positions", false},
                        {slots, "slots", false},
                        {q_out, "q_out", no_q}};
  st = check_pointers("append kv", ptrs, 7);
  if (st != MLA_OK) return st;
  const int64_t strides[] = {q_row_stride, k_row_stride, v_row_stride};
  const int64_t least[] = {(int64_t)H * D, (int64_t)Hk * D, (int64_t)Hk * D};
  const char* names[] = {"q_row_stride", "k_row_stride", "v_row_stride"};
  for (int i = no_q ? 1 : 0; i < 3; ++i) {
    if (strides[i] < least[i] || strides[i] * eb % 16 != 0) {
      set_error("append kv: %s %lld must be at least %lld and a multiple of 16 bytes", names[i],
                (long long)strides[i], (long long)least[i]);
      return MLA_ERR_INVALID_ARG;
    }
  }
  if (!no_q) {
    // in place only row for row
    const bool same = q == q_out && q_row_stride == least[0];
    const Range a = range(q, ((int64_t)(rows - 1) * q_row_stride + least[0]) * eb);
    const Range b = range(q_out, (int64_t)rows * least[0] * eb);
    if (!same && overlap(a, b)) {
      set_error("append kv: q_out overlaps q without being q");
      return MLA_ERR_INVALID_ARG;
    }
  }
  AppendKVParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_row_stride;
  p.k_stride = k_row_stride;
  p.v_stride = v_row_stride;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.slots = slots;
  p.q_out = q_out;
  p.k_cache = cache->k;
  p.v_cache = cache->v;
  p.page_stride = cache->page_stride;
  p.row_stride = cache->row_stride;
  p.head_stride = cache->head_stride;
  p.cache_rows = (int64_t)cache->num_pages * cache->page_size;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.page = cache->page_size;
  p.table_rows = table_rows;
  p.rope = rope_dim;
  p.interleaved = interleaved;
  p.q_heads = no_q ? 0 : H;
  p.kv_heads = Hk;
  p.dim = D;
  const int N = 16 / eb;
  p.turned = rope_dim / 2 / N;
  p.items = p.turned + ((D / N - 2 * p.turned) + 1) / 2;
  const int heads = p.q_heads + 2 * Hk;
  const dim3 block = item_block(p.items);
  p.div = PageDiv(cache->page_size);
  const int kk = heads_per_thread(heads, (int)block.y, rows), hpc = kk * (int)block.y;
  const dim3 grid((unsigned)rows, (unsigned)((heads + hpc - 1) / hpc));
  if (grid.y > 65535u) {
    set_error("append kv: %d heads are too many", heads);
    return MLA_ERR_UNSUPPORTED;
  }
  const cudaStream_t s = (cudaStream_t)stream;
  KernelTimer kt("append_kv", s);
  if (eb == 4) return launched(launch_kv<float, float>(kk, grid, block, s, p));
  if (g->cache_dtype == MLA_DTYPE_E4M3)
    return launched(launch_kv<__nv_bfloat16, __nv_fp8_e4m3>(kk, grid, block, s, p));
  return launched(launch_kv<__nv_bfloat16, __nv_bfloat16>(kk, grid, block, s, p));
}
