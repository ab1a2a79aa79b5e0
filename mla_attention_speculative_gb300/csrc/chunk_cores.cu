// Attention of a step's new rows over a paged key/value cache on CUDA cores, for
// fp32.
//
// A CTA of 256 threads takes 64 query rows (tokens times the heads of one group)
// against tiles of 64 cached positions: S = Q K^T with a 4 x 4 block of S to a
// thread, a running maximum and sum per row in registers, P through shared
// memory, and O += P V with 4 rows of DP / 16 columns to a thread.  Everything
// is held and summed in fp32.
//
// 8 sequences of 1 to 129 rows, a window of 1000 over up to 4129 positions, 20 heads on 4
// of 80: 61 us in a graph, 2 of them the join's.  A tile of heads of 80 (held as 96) is
// 64 * 64 * 176 multiply-adds, 5632 cycles of an SM.  The cut gives no CTA more than 4 of
// the 1012 tiles (kMinShare), so the fullest SM multiplies for 45000 of the 107000 cycles
// that it is active: the multiply-add pipe is 40 % busy, issue slots 56 %, and a third of
// the instructions are no multiply-adds.  The rest is waiting: a tile's page ids, then the
// rows they lead to, then the barrier, with nothing of the next tile under way.  (Tried:
// asynchronous copies of the next tile, behind its page ids all the same, 68 us for 64
// then, multiply-adds of pairs 72, both 75.)

#include <mutex>
#include <type_traits>

#include "chunk_attention.h"
#include "sm103_ptx.cuh"

namespace mla {

static __device__ int g_chunk_cores_status;

namespace chunk {

int cores_status(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_chunk_cores_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_chunk_cores_status, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

namespace {

constexpr int kBM = 64, kBN = 64, kThreads = 256;

template <int DP>
struct Layout {
  static constexpr int LD = DP + 4;   // floats of a row: 16-byte reads of eight rows meet no bank twice
  static constexpr int LP = kBN + 4;
  static constexpr int SMEM = (3 * 64 * LD + kBM * LP) * 4;
  static constexpr int OCC = 2 * (SMEM + 1024) <= 227 * 1024 ? 2 : 1;
};

__device__ __forceinline__ void put16(float* dst, const float* src) {
  *reinterpret_cast<float4*>(dst) = *reinterpret_cast<const float4*>(src);
}
template <int DP>
__global__ void __launch_bounds__(kThreads, Layout<DP>::OCC) chunk_cores_kernel(const Params p) {
  using L = Layout<DP>;
  constexpr int LD = L::LD, LP = L::LP, NO = DP / 32;
  extern __shared__ float4 s_raw[];
  float* sQ = reinterpret_cast<float*>(s_raw);
  float* sK = sQ + 64 * LD;
  float* sV = sK + 64 * LD;
  float* sP = sV + 64 * LD;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int cta = blockIdx.x;
  sm103::pdl_wait();
  Start from, to;
  Sequence seq = {0, 0, 0, 0, 0};
  if (p.starts == nullptr) {
    find_share(p, cta, *reinterpret_cast<PlanScratch*>(s_raw), from, to, seq);
  } else {
    read_share(p, cta, *reinterpret_cast<PlanScratch*>(s_raw), from, to, seq);
  }
  // columns past the heads' width stay zero
  for (int i = tid; i < 3 * 64 * LD; i += kThreads) sQ[i] = 0.f;
  __syncthreads();
  Walk w;
  w.begin(from, to, seq);
  Segment g;
  for (; w.next(p, g); w.advance(p, g)) {
    const Sequence& s = w.seq;
    const Unit& u = g.unit;
    const int kvh = w.at.kvh, rows = u.r1 - u.r0;
    __syncthreads();  // the queries before are used up
    {
      constexpr int N = 4;
      const int vecs = p.dim / N;
      for (int x = tid; x < 64 * vecs; x += kThreads) {
        const int r = x / vecs, c = (x - r * vecs) * N;
        if (r >= rows) {
#pragma unroll
          for (int e = 0; e < N; ++e) sQ[r * LD + c + e] = 0.f;
          continue;
        }
        const int i = p.group_div(u.r0 + r), j = u.r0 + r - i * p.group;
        put16(sQ + r * LD + c, (const float*)p.q + (int64_t)(s.row0 + i) * p.q_stride +
                                   (int64_t)(kvh * p.group + j) * p.dim + c);
      }
    }
    int first[4], last[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = p.group_div(u.r0 + min(ty * 4 + a, rows - 1));
      first[a] = first_seen(p, s, i);
      last[a] = last_seen(s, i);
    }
    // positions that every row of the unit sees
    const int all0 = first_seen(p, s, p.group_div(u.r1 - 1)), all1 = last_seen(s, p.group_div(u.r0));
    const float sl2 = p.scale_log2;
    float m[4], l[4], o[4][2 * NO];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * NO; ++c) o[a][c] = 0.f;
    }
    for (int t = g.t0; t < g.t1; ++t) {
      const int pos0 = (u.tile0 + t) * kBN;
      __syncthreads();  // the tile before is used up
      {
        constexpr int N = 4;
        const int vecs = p.dim / N;
        for (int x = tid; x < 64 * vecs; x += kThreads) {
          const int r = x / vecs, c = (x - r * vecs) * N, pos = pos0 + r;
          bool have = pos >= u.lo && pos < u.hi;
          int64_t at = 0;
          if (have) {
            const int pg = p.page_div(pos);
            const int id = p.table[(int64_t)w.at.b * p.width + pg];
            if (id < 0 || id >= p.num_pages) {
              atomicCAS(&g_chunk_cores_status, 0, kBadPageSite);
              have = false;
            } else {
              at = id * p.page_stride + (int64_t)(pos - pg * p.page) * p.row_stride +
                   kvh * p.head_stride + c;
            }
          }
          if (have) {
            put16(sK + r * LD + c, (const float*)p.k + at);
            put16(sV + r * LD + c, (const float*)p.v + at);
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) sK[r * LD + c + e] = sV[r * LD + c + e] = 0.f;
          }
        }
      }
      __syncthreads();
      float x[4][4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) x[a][b] = 0.f;
#pragma unroll 4
      for (int d = 0; d < p.dim; d += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
          qv[a] = *reinterpret_cast<const float4*>(sQ + (ty * 4 + a) * LD + d);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          kv[b] = *reinterpret_cast<const float4*>(sK + (tx + 16 * b) * LD + d);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            x[a][b] = fmaf(qv[a].x, kv[b].x, x[a][b]);
            x[a][b] = fmaf(qv[a].y, kv[b].y, x[a][b]);
            x[a][b] = fmaf(qv[a].z, kv[b].z, x[a][b]);
            x[a][b] = fmaf(qv[a].w, kv[b].w, x[a][b]);
          }
      }
      const bool edge = pos0 < all0 || pos0 + kBN - 1 > all1;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int pos = pos0 + tx + 16 * b;
          x[a][b] = !edge || (pos >= first[a] && pos <= last[a]) ? x[a][b] * sl2 : -INFINITY;
          top = fmaxf(top, x[a][b]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const float mn = fmaxf(m[a], top), base = mn == -INFINITY ? 0.f : mn;
        const float f = sm103::ex2(m[a] - base);
        m[a] = mn;
        float sum = 0.f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          x[a][b] = sm103::ex2(x[a][b] - base);
          sum += x[a][b];
          sP[(ty * 4 + a) * LP + tx + 16 * b] = x[a][b];
        }
        l[a] = l[a] * f + sum;  // this thread's columns; the 16 threads' sums meet at the end
        if (f != 1.f) {
#pragma unroll
          for (int c = 0; c < 2 * NO; ++c) o[a][c] *= f;
        }
      }
      // A hidden position's weight is -0, which no exponential is (put here, behind all of
      // them, since few tiles have any: chosen where they are stored 63.4 us for 61.1).
      if (edge) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int pos = pos0 + tx + 16 * b;
            if (pos < first[a] || pos > last[a]) sP[(ty * 4 + a) * LP + tx + 16 * b] = -0.f;
          }
      }
      __syncwarp();  // a row's weights are made and used by one warp
      auto products = [&](auto masked) {
#pragma unroll 2
        for (int k = 0; k < kBN; k += 4) {
          float pw[4][4];
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const float4 y = *reinterpret_cast<const float4*>(sP + (ty * 4 + a) * LP + k);
            pw[a][0] = y.x; pw[a][1] = y.y; pw[a][2] = y.z; pw[a][3] = y.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 vv[NO];
#pragma unroll
            for (int c = 0; c < NO; ++c)
              vv[c] = *reinterpret_cast<const float2*>(sV + (k + e) * LD + 2 * tx + 32 * c);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              // a hidden position's value may be anything, also what zero times it is not zero
              // (a seen one counts, whatever its weight)
              if (decltype(masked)::value && __float_as_uint(pw[a][e]) == 0x80000000u) continue;
#pragma unroll
              for (int c = 0; c < NO; ++c) {
                o[a][2 * c] = fmaf(pw[a][e], vv[c].x, o[a][2 * c]);
                o[a][2 * c + 1] = fmaf(pw[a][e], vv[c].y, o[a][2 * c + 1]);
              }
            }
          }
        }
      };
      if (edge) products(std::true_type());
      else products(std::false_type());
      __syncwarp();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[a] += __shfl_xor_sync(~0u, l[a], d);
    }
    const bool whole = g.first && g.last;
    const int64_t slot = 2 * cta + (g.first ? 1 : 0);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = ty * 4 + a;
      if (r >= rows) continue;
      if (!whole) {
        if (tx == 0) p.part_ml[slot * kBM + r] = make_float2(m[a], l[a]);
        float* dst = p.part_o + (slot * kBM + r) * p.dp + 2 * tx;
#pragma unroll
        for (int c = 0; c < NO; ++c)
          *reinterpret_cast<float2*>(dst + 32 * c) = make_float2(o[a][2 * c], o[a][2 * c + 1]);
        continue;
      }
      const int i = p.group_div(u.r0 + r), j = u.r0 + r - i * p.group;
      const int64_t head = (int64_t)(s.row0 + i) * p.heads + kvh * p.group + j;
      const float inv = 1.f / l[a];
#pragma unroll
      for (int c = 0; c < NO; ++c) {
        const int col = 2 * tx + 32 * c;
        if (col >= p.dim) continue;
        // (weights that are all zero: the values may be no numbers)
        const float y0 = l[a] == 0.f ? 0.f : o[a][2 * c] * inv;
        const float y1 = l[a] == 0.f ? 0.f : o[a][2 * c + 1] * inv;
        *reinterpret_cast<float2*>((float*)p.out + head * p.dim + col) = make_float2(y0, y1);
      }
      if (tx == 0 && p.lse)
        p.lse[head] = l[a] == 0.f ? -INFINITY : (m[a] + log2f(l[a])) * 0.6931471805599453f;
    }
  }
}

template <int DP>
cudaError_t launch(const Params& p, int ctas, cudaStream_t stream) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto* fn = chunk_cores_kernel<DP>;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Layout<DP>::SMEM);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  KernelTimer kt("chunk_cores", stream);
  return launch_dependent(fn, dim3((unsigned)ctas), dim3(kThreads), Layout<DP>::SMEM, stream, p);
}

template <int DP>
Kernel make() {
  return {kBM, kBN, DP, Layout<DP>::OCC, kCoresCost, kCoresSnap, launch<DP>};
}

}  // namespace

Kernel kernel_cores(int dim) {
  return dim <= 64    ? make<64>()
         : dim <= 96  ? make<96>()
         : dim <= 128 ? make<128>()
         : dim <= 192 ? make<192>()
                      : make<256>();
}

}  // namespace chunk
}  // namespace mla
