// Attention of a step's new rows over a paged key/value cache on the tensor
// cores (tcgen05, accumulators in tensor memory), for bf16 and e4m3 caches.
//
// A CTA takes a unit of 128 or 256 query rows (tokens times the heads of one
// group) against tiles of 128 cached positions:
//   S = Q K^T      128 x 128, both operands in shared memory
//   P = 2^(S - m)  in registers, a thread a row, back to tensor memory over S
//   O += P V       P from tensor memory, V from shared memory
// Two streams of this keep the tensor pipe and the softmax busy in turn.  With
// more than 128 rows a stream is 128 rows, and both use the same tiles of K and
// V; with fewer both take the same rows, one the even tiles and one the odd ones,
// and their sums meet at the end.  Heads wider than 128 have room for one
// accumulator only: one stream, whose next S is made while its softmax runs.
//
// The running maximum moves only when a row's grows by more than 2^8, so O is
// rarely rescaled; sums and accumulators are fp32.  Weights enter the second
// product as bf16 beside a bf16 cache and as fp16 beside an e4m3 one, whose
// elements are exact in fp16 (queries too then, relative to their head's largest
// element, by a power of two; weights times 2^7, so that those down to 2^-31 of
// the largest count).
//
// Keys and values come through a ring of 128-position blocks:
//   kTma      one thread's TMA boxes, page by page, where pages are whole runs of
//             8 rows (page sizes with a power of two of 8 or more in them)
//   kRows     16-byte copies of single rows, for any other page size
//   kConvert  the same into a staging ring, then e4m3 -> fp16 by the same threads
// Rows that nobody sees, and elements of V that are not finite in a tile where a
// row is hidden from some query, are set to zero before P V reads them (0 times
// such an element is NaN); the latter are put back at the end, for the rows that
// see them.
#pragma once

#include <cuda_bf16.h>

#include <mutex>
#include <type_traits>

#include "chunk_attention.h"
#include "sm103_ptx.cuh"
#include "tma_host.h"

namespace mla {
namespace chunk {
namespace {
using namespace sm103;

enum Feed { kTma = 0, kRows = 1, kConvert = 2 };

static __device__ int g_status;

__device__ __forceinline__ void report(int code) { atomicCAS(&g_status, 0, code); }
__device__ __forceinline__ void wait_or_fail(bool& ok, uint32_t bar, uint32_t parity, int code) {
  if (!ok) return;
  if (!mbar_wait(bar, parity)) {
    ok = false;
    report(code);
  }
}

constexpr int kBN = 128;

template <int DP, int FEED>
struct Shape {
  static constexpr int NS = DP <= 128 ? 2 : 1;        // streams
  static constexpr int BM = 128 * NS;
  static constexpr int BW = DP < 128 ? DP : 128;      // columns of a block
  static constexpr int NBLK = (DP + 127) / 128;       // blocks of a tile of K or V
  static constexpr int QB = 128 * DP * 2;             // bytes of 128 queries
  static constexpr int SLOT = kBN * BW * 2;
  static constexpr int RAW = FEED == kConvert ? kBN * BW : 0;
  static constexpr int NB = FEED == kConvert ? (DP == 64 ? 6 : 3) : (DP == 64 ? 10 : 5);
  static constexpr int RS = FEED == kConvert ? (DP == 64 ? 6 : 3) : 0;
  static constexpr int THREADS = 128 * NS + 128;
  static constexpr int FEEDERS = FEED == kTma ? 32 : FEED == kRows ? 64 : 96;
  static constexpr uint32_t TM_S = NS * DP;           // tensor memory: O, then two of S
  static constexpr int TAIL = 1024 + (FEED == kConvert ? NS * 128 * 4 : 0);
  static constexpr int SMEM = 1024 + NS * QB + NB * SLOT + RS * RAW + TAIL;
  static_assert(SMEM <= 232448, "more shared memory than a CTA may have");
  static_assert(TM_S + 256 <= 512, "more tensor memory than there is");
  // barriers
  static constexpr int FULL = 0, EMPTY = NB, LANDED = 2 * NB, QFULL = 3 * NB, QEMPTY = QFULL + 2,
                       SFULL = QEMPTY + 1, PFULL = SFULL + 2, OFULL = PFULL + 2,
                       PVDONE = OFULL + 2, DRAIN = PVDONE + 2, BARS = DRAIN + 1;
  static_assert(BARS * 8 + 10 * 4 + 4 * NS * sizeof(Walk) <= 1024, "the barriers do not fit");
};

struct Maps {
  CUtensorMap k, v;
  int box;  // rows of a box
};

// The place of a block in the ring's order K0 K1 V0 K2 V1 .. V(n-1).
__device__ __forceinline__ int k_place(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_place(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// Positions that every row of a unit sees; a tile beyond them hides something.
struct Seen {
  int lo, hi;
  __device__ __forceinline__ Seen(const Params& p, const Sequence& s, const Unit& u)
      : lo(first_seen(p, s, p.group_div(u.r1 - 1))), hi(last_seen(s, p.group_div(u.r0))) {}
  __device__ __forceinline__ bool edge(int pos0) const { return pos0 < lo || pos0 + kBN - 1 > hi; }
};

// What the elements of V that are not finite add to one output: read again, for
// the tiles where they were set to zero.  (Slow, and for such input only.)
template <int FEED>
__device__ __noinline__ float odd_values(const Params& p, int b, int kvh, int col, int lo, int hi,
                                         int seen_lo, int seen_hi) {
  float sum = 0.f;
  for (int t = lo; t <= hi; ++t) {
    const int pos0 = t / kBN * kBN;
    if (!(pos0 < seen_lo || pos0 + kBN - 1 > seen_hi)) {
      t = pos0 + kBN - 1;  // a tile that was not touched
      continue;
    }
    const int pg = p.page_div(t);
    const int id = p.table[(int64_t)b * p.width + pg];
    if (id < 0 || id >= p.num_pages) continue;
    const int64_t at = id * p.page_stride + (int64_t)(t - pg * p.page) * p.row_stride +
                       kvh * p.head_stride + col;
    float v;
    if constexpr (FEED == kConvert) {
      const uint8_t x = ((const uint8_t*)p.v)[at];
      v = (x & 0x7F) == 0x7F ? NAN : 0.f;
    } else {
      v = __bfloat162float(((const __nv_bfloat16*)p.v)[at]);
    }
    if (!isfinite(v)) sum += v;
  }
  return sum;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int DP, int FEED>
__global__ void __launch_bounds__(Shape<DP, FEED>::THREADS, 1)
    chunk_sm103_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using C = Shape<DP, FEED>;
  constexpr int NS = C::NS, NBLK = C::NBLK, NB = C::NB;
  constexpr bool HALF = FEED == kConvert;  // fp16 operands
  constexpr float shift = HALF ? kShift : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* tail = smem + NS * C::QB + NB * C::SLOT + C::RS * C::RAW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail);
  uint32_t* slot_word = reinterpret_cast<uint32_t*>(bars + C::BARS);
  volatile int* dirty = reinterpret_cast<int*>(slot_word + 2);  // [8], by segment
  Walk* walks = reinterpret_cast<Walk*>(slot_word + 10);          // [4 * NS], a softmax warp's
  float* q_scale = reinterpret_cast<float*>(tail + 1024);       // kConvert: [NS * 128]
  const uint32_t sQ = smem_u32(smem), sRing = sQ + NS * C::QB, sRaw = sRing + NB * C::SLOT;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NB; ++i) {
      mbar_init(bar(C::FULL + i), FEED == kTma ? 1 : C::FEEDERS);
      mbar_init(bar(C::EMPTY + i), 1);
      mbar_init(bar(C::LANDED + i), FEED == kTma ? 1 : C::FEEDERS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::QFULL + i), 128);
      mbar_init(bar(C::SFULL + i), 1);
      mbar_init(bar(C::PFULL + i), 128);
      mbar_init(bar(C::OFULL + i), 1);
      mbar_init(bar(C::PVDONE + i), 1);
    }
    mbar_init(bar(C::QEMPTY), 1);
    mbar_init(bar(C::DRAIN), 1);
    for (int i = 0; i < 8; ++i) dirty[i] = -1;
    fence_mbar_init();
  }
  if (warp == 4 * NS) tmem_alloc(smem_u32(slot_word), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot_word;
  pdl_wait();
  Walk w;
  Segment g;
  w.begin(p, cta);
  bool ok = true;

  if (warp < 4 * NS) {
    // ------------------------------------------------------------- softmax
    const int s = warp >> 2;                  // stream
    const int q = (warp & 3) * 32 + lane;     // its row, and its tensor memory lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t uses[2] = {0, 0}, o_uses = 0;
    int seg = 0;                              // segments with tiles before this one
    for (; w.next(p, g); w.advance(p, g)) {
      const Sequence& sq = w.seq;
      const Unit& u = g.unit;
      const int n = g.t1 - g.t0, rows = u.r1 - u.r0, kvh = w.at.kvh;
      const bool split = NS == 2 && rows <= 128;  // both streams take the same rows
      const int r = (split ? 0 : 128 * s) + q;
      const int tok = p.group_div(u.r0 + min(r, rows - 1));
      const int first = first_seen(p, sq, tok), last = r < rows ? last_seen(sq, tok) : -1;
      const Seen seen(p, sq, u);
      float sl2 = p.scale_log2;
      float ksign = 1.f;
      if constexpr (HALF) {
        const float ks = p.k_scale ? p.k_scale[kvh] : 1.f;
        ksign = ks < 0.f ? -1.f : 1.f;
        // (a scale that is no finite number makes its heads NaN; one of zero leaves
        // hidden scores below the others)
        sl2 = isfinite(ks) ? fmaxf(sl2 * fabsf(ks), 1e-37f) : NAN;
      }
      if (n > 0 && (!split || s == 0)) {
        // ---- this stream's queries
        if (seg > 0) wait_or_fail(ok, bar(C::QEMPTY), (seg - 1) & 1, 100);
        constexpr int CH = DP / 8;  // 16-byte chunks of a row
        const uint32_t dst0 = sQ + (split ? 0 : s) * C::QB;
        const int row0 = (warp & 3) * 32;
        auto source = [&](int row, int c, bool& have) {
          const int x = (split ? 0 : 128 * s) + row;
          have = x < rows && c * 8 < p.dim;
          const int i = have ? p.group_div(u.r0 + x) : 0, j = have ? u.r0 + x - i * p.group : 0;
          return (const __nv_bfloat16*)p.q +
                 (have ? (int64_t)(sq.row0 + i) * p.q_stride +
                             (int64_t)(kvh * p.group + j) * p.dim + c * 8
                       : 0);
        };
        if constexpr (!HALF) {
#pragma unroll 4
          for (int k = 0; k < CH; ++k) {
            const int e = k * 32 + lane, row = row0 + e / CH, c = e % CH;
            bool have;
            const __nv_bfloat16* src = source(row, c, have);
            cp_async16(dst0 + (c >> 3) * 16384 + sw128_offset(row, (c & 7) * 8), src,
                       have ? 16u : 0u);
          }
          cp_async_wait_all();
        } else {
          constexpr int LPR = CH <= 8 ? 8 : CH <= 16 ? 16 : 32;  // lanes to a row
          for (int k = 0; k < LPR; ++k) {
            const int row = row0 + k * (32 / LPR) + lane / LPR, c = lane % LPR;
            bool have;
            const __nv_bfloat16* src = source(row, c, have);
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (have) x = *reinterpret_cast<const uint4*>(src);
            const uint32_t word[4] = {x.x, x.y, x.z, x.w};
            float f[8], top = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[2 * e] = __uint_as_float(word[e] << 16);
              f[2 * e + 1] = __uint_as_float(word[e] & 0xFFFF0000u);
              top = fmaxf(top, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            // 2^-exponent of the largest; the row's scores are scaled back
            float down = 1.f, up = 1.f;
            if (top > 0.f && isfinite(top)) {
              const int ex = ilogbf(top);
              down = ldexpf(1.f, -ex);
              up = ldexpf(1.f, ex);
            }
            if (c == 0) q_scale[(split ? 0 : 128 * s) + row] = up;
            down *= ksign;
            if (c < CH) {
              const uint32_t at = dst0 + (c >> 3) * 16384 + sw128_offset(row, (c & 7) * 8);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                           "r"(pack_half(f[0] * down, f[1] * down)),
                           "r"(pack_half(f[2] * down, f[3] * down)),
                           "r"(pack_half(f[4] * down, f[5] * down)),
                           "r"(pack_half(f[6] * down, f[7] * down))
                           : "memory");
            }
          }
        }
        fence_async_shared();
        mbar_arrive(bar(C::QFULL + s));
      }
      if constexpr (HALF) {
        if (n > 0) {
          if (split) named_bar_sync(1, 256);  // stream 1 reads the scales stream 0 wrote
          else __syncwarp();
          sl2 *= q_scale[r];
        }
      }
      // Where the walk stands waits in shared memory while the scores need the registers.
      if (lane == 0) walks[warp] = w;
      __syncwarp();
      // ---- tiles
      const int tile_pos = (u.tile0 + g.t0) * kBN;
      float top = -INFINITY, m = -INFINITY, l = 0.f;  // the reference, times the scale; the sum
      const int step = split ? 2 : 1;
      int i = split ? s : 0;
      const bool any = i < n;
      for (bool begun = false; i < n; i += step, begun = true) {
        const int x = NS == 2 ? s : (i & 1);
        const int pos0 = tile_pos + i * kBN;
        const uint32_t tS = tmem + lane_base + C::TM_S + 128 * x;
        wait_or_fail(ok, bar(C::SFULL + x), uses[x] & 1, 101);
        tc_fence_after();
        // The scores are read twice, for their maximum and for the weights, 32 at a time
        // with the next 32 on their way: kept in registers, 128 of them spill.
        uint32_t u0[32], u1[32];
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const bool edge = seen.edge(pos0);
        // f(scores, piece) for the four pieces; the first one is under way
        auto pieces = [&](auto f) {
          tmem_wait_ld<32>(u0);
          tmem_ld32(tS + 32, u1);
          f(u0, 0);
          tmem_wait_ld<32>(u1);
          tmem_ld32(tS + 64, u0);
          f(u1, 1);
          tmem_wait_ld<32>(u0);
          tmem_ld32(tS + 96, u1);
          f(u0, 2);
          tmem_wait_ld<32>(u1);
          f(u1, 3);
        };
        auto hide = [&](uint32_t* u, int k) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int pos = pos0 + 32 * k + j;
            if (pos < first || pos > last) u[j] = 0xFF800000u;
          }
        };
        auto highest = [&](const uint32_t* u) {
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            t4[(j >> 1) & 3] = fmaxf(t4[(j >> 1) & 3],
                                     fmaxf(__uint_as_float(u[j]), __uint_as_float(u[j + 1])));
        };
        if (edge) {
          // (few tiles: a loop, so that the code of the others stays together)
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            tmem_ld32(tS + 32 * k, u0);
            tmem_wait_ld<32>(u0);
            hide(u0, k);
            highest(u0);
          }
        } else {
          tmem_ld32(tS, u0);
          pieces([&](uint32_t* u, int) { highest(u); });
        }
        tmem_ld32(tS, u0);
        const float mx = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        const float mn = mx == -INFINITY ? -INFINITY : mx * sl2;
        const bool need = mn > m + 8.f;
        if (__any_sync(~0u, need)) {
          if (begun) {
            if constexpr (NS == 1) {
              // O must hold the tile before's products (with two streams S comes behind them)
              const int y = (i - 1) & 1;
              wait_or_fail(ok, bar(C::PVDONE + y), (uses[y] - 1) & 1, 102);
              tc_fence_after();
            }
            const float f = need ? ex2(m - mn) : 1.f;
            l *= f;
            const uint32_t tO = tmem + lane_base + (NS == 2 ? DP * s : 0);
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
              tmem_wait_ld<32>(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(tO + c, o);
            }
          }
          if (need) {
            top = mx;
            m = mn;
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        // Beyond 2^20 the rounding of m is no longer small beside 1: there the difference
        // of the scores comes first.
        const bool large = __any_sync(~0u, fabsf(base) > 1048576.f);
        const uint64_t sc2 = pack2(sl2, sl2), off2 = pack2(shift - base, shift - base);
        const float ref = m == -INFINITY ? 0.f : top;
        uint64_t sum2[2] = {0ull, 0ull};
        auto weights = [&](uint32_t* u, int k, auto careful) {
          // (step by step for 32 scores, so that no exponential waits for another)
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a = __uint_as_float(u[e]), b = __uint_as_float(u[e + 1]);
            if constexpr (decltype(careful)::value) {
              y[e] = fmaf(a - ref, sl2, shift);
              y[e + 1] = fmaf(b - ref, sl2, shift);
            } else {
              unpack2(fma2(pack2(a, b), sc2, off2), y[e], y[e + 1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = ex2(y[e]);
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            sum2[e & 1] = add2(sum2[e & 1], pack2(y[2 * e], y[2 * e + 1]));
            pk[e] = HALF ? pack_half(y[2 * e], y[2 * e + 1]) : pack_bf16(y[2 * e], y[2 * e + 1]);
          }
          tmem_st16(tS + 16 * k, pk);
        };
        if (edge || large) {
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            tmem_wait_ld<32>(u0);
            hide(u0, k);
            weights(u0, k, std::true_type());
            if (k < 3) tmem_ld32(tS + 32 * (k + 1), u0);
          }
        } else {
          pieces([&](uint32_t* u, int k) { weights(u, k, std::false_type()); });
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::PFULL + x));
        ++uses[x];
        float a, b;
        unpack2(add2(sum2[0], sum2[1]), a, b);
        l += a + b;
      }
      // ---- outputs
      w = const_cast<const Walk&>(walks[warp]);
      g = w.segment(p);
      const bool whole = g.first && g.last;
      if (any) {
        wait_or_fail(ok, bar(C::OFULL + s), o_uses & 1, 103);
        ++o_uses;
        tc_fence_after();
      }
      const bool fix = n > 0 && dirty[seg & 7] == seg;
      float f0 = 1.f, f1 = 0.f;
      int c0 = 0, c1 = DP;
      const float2* other = nullptr;
      if (split) {
        // the streams' sums meet: each half of the columns by one of them (a place of the
        // queries that are not there holds the other's maximum and sum)
        float2* sums = reinterpret_cast<float2*>(smem + C::QB);
        sums[128 * s + q] = make_float2(m, any ? l : 0.f);
        named_bar_sync(1, 256);
        tc_fence_after();
        other = sums + 128 * (s ^ 1) + q;
        const float2 z = *other;
        const float mm = fmaxf(m, z.x), ref = mm == -INFINITY ? 0.f : mm;
        f0 = ex2(m - ref);
        f1 = ex2(z.x - ref);
        l = l * f0 + z.y * f1;
        m = mm;
        c0 = s * (DP / 2);
        c1 = c0 + DP / 2;
      }
      const bool second = split && n > 1;  // stream 1 has an accumulator
      const float vs = HALF && p.v_scale ? p.v_scale[kvh] : 1.f;
      const float inv = l == 0.f ? 0.f : vs / l;
      const bool live = r < rows;
      const int i_tok = p.group_div(u.r0 + min(r, rows - 1)),
                head_in = u.r0 + min(r, rows - 1) - i_tok * p.group;
      const int64_t head = (int64_t)(sq.row0 + i_tok) * p.heads + kvh * p.group + head_in;
      const int64_t part = (int64_t)(2 * cta + (g.first ? 1 : 0)) * p.bm + r;
      // the accumulators' weights: mine and the other stream's
      const float wa = split && s == 1 ? f1 : f0, wb = split && s == 1 ? f0 : f1;
#pragma unroll 1
      for (int c = c0; c < c1; c += 16) {
        uint32_t o[16];
        __syncwarp();
        if (n > 0) {
          tmem_ld16(tmem + lane_base + (NS == 2 && !split ? DP * s : 0) + c, o);
          if (second) {
            uint32_t o1[16];
            tmem_ld16(tmem + lane_base + DP + c, o1);
            tmem_wait_ld<16>(o);
            tmem_wait_ld<16>(o1);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              // (a stream without weight may hold anything)
              const float a = wa == 0.f ? 0.f : __uint_as_float(o[e]) * wa;
              const float b = wb == 0.f ? 0.f : __uint_as_float(o1[e]) * wb;
              o[e] = __float_as_uint(a + b);
            }
          } else {
            tmem_wait_ld<16>(o);
          }
        }
        if (live) {
          if (l == 0.f) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
          } else if (fix) {
            const int lo = max(first, (u.tile0 + g.t0) * kBN),
                      hi = min(last, (u.tile0 + g.t1) * kBN - 1);
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              if (c + e >= p.dim) continue;
              const float y = odd_values<FEED>(p, w.at.b, kvh, c + e, lo, hi, seen.lo, seen.hi);
              // (the array stays in registers: no index at run time)
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (k == e) o[k] = __float_as_uint(__uint_as_float(o[k]) + y);
            }
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              if (c + e >= p.dim) continue;
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[k] = pack_bf16(__uint_as_float(o[e + 2 * k]) * inv,
                                 __uint_as_float(o[e + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>((__nv_bfloat16*)p.out + head * p.dim + c + e) =
                  make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(p.part_o + part * p.dp + c + e) =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
      }
      if (live && (!split || s == 0)) {
        if (!whole) p.part_ml[part] = make_float2(m, l);
        else if (p.lse)
          p.lse[head] = l == 0.f ? -INFINITY : (m + (log2f(l) - shift)) * 0.6931471805599453f;
      }
      if (split) {
        tc_fence_before();
        named_bar_sync(1, 256);  // both streams are through with both accumulators
      }
      if (n > 0) ++seg;
    }
  } else if (warp == 4 * NS) {
    // ----------------------------------------------------------------- MMA
    const uint32_t id_s = HALF ? idesc_f16(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0);
    const int nk = (p.dim + 15) / 16;  // steps of 16 columns
    const bool whole = nk == DP / 16;
    uint32_t at = 0;                   // blocks before this segment
    uint32_t puses[2] = {0, 0}, q_uses[2] = {0, 0};
    for (; w.next(p, g); w.advance(p, g)) {
      const int n = g.t1 - g.t0, rows = g.unit.r1 - g.unit.r0;
      if (n == 0) continue;
      const bool split = NS == 2 && rows <= 128;
      if (lane == 0) {
        auto block = [&](int place, int blk) { return at + (uint32_t)(place * NBLK + blk); };
        auto landed = [&](uint32_t pos) {
          wait_or_fail(ok, bar(C::FULL + pos % NB), (pos / NB) & 1, 110);
        };
        auto scores = [&](int x, int tile, int i, bool wait, bool free) {
          const uint64_t dq = sdesc_sw128(sQ + tile * C::QB, 16, 1024);
#pragma unroll
          for (int blk = 0; blk < NBLK; ++blk) {
            const uint32_t pos = block(k_place(i), blk);
            if (wait) landed(pos);
            if (!ok) return;
            if (FEED != kTma) fence_async_shared();
            tc_fence_after();
            const uint64_t dk = sdesc_sw128(sRing + (pos % NB) * C::SLOT, 16, 1024);
            const uint32_t dst = tmem + C::TM_S + 128 * x;
            const uint64_t dqb = dq + (uint64_t)(blk * 2048);
            // (a condition on single MMAs of the unrolled form made the compiler give some of
            // them another one's descriptor: so either all of them, or a loop)
            if (whole) {
#pragma unroll
              for (int k = 0; k < C::BW / 16; ++k)
                if (blk * (C::BW / 16) + k < DP / 16)
                  mma_bf16(dst, dqb + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                           dk + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), id_s, (blk | k) != 0);
            } else {
#pragma unroll 1
              for (int k = 0; k < C::BW / 16; ++k) {
                if (blk * (C::BW / 16) + k >= nk) break;
                const uint64_t off = (uint64_t)((k >> 2) * 1024 + (k & 3) * 2);
                mma_bf16(dst, dqb + off, dk + off, id_s, (blk | k) != 0);
              }
            }
            if (free) mma_commit(bar(C::EMPTY + pos % NB));
          }
          mma_commit(bar(C::SFULL + x));
        };
        auto products = [&](int x, int o, int i, bool begin, bool wait, bool free) {
          wait_or_fail(ok, bar(C::PFULL + x), puses[x] & 1, 111);
          ++puses[x];
#pragma unroll
          for (int blk = 0; blk < NBLK; ++blk) {
            const uint32_t pos = block(v_place(i, n), blk), sl = pos % NB;
            if (wait) landed(pos);
            if (!ok) return;
            if (FEED != kTma) fence_async_shared();
            tc_fence_after();
            const uint64_t dv = sdesc_sw128(sRing + sl * C::SLOT, 16384, 1024);
            const int cols = min(p.dim - 128 * blk, C::BW);
            const int nn = (cols + 15) & ~15;
            const uint32_t id_o = HALF ? idesc_f16(128, nn, 0, 1) : idesc_bf16(128, nn, 0, 1);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_bf16_tmem_a(tmem + o * DP + 128 * blk, tmem + C::TM_S + 128 * x + 8 * k,
                              dv + 128 * k, id_o, !begin || k > 0);
            if (free) mma_commit(bar(C::EMPTY + sl));
          }
        };
        wait_or_fail(ok, bar(C::QFULL), q_uses[0] & 1, 113);
        ++q_uses[0];
        if (NS == 2 && !split) {
          wait_or_fail(ok, bar(C::QFULL + 1), q_uses[1] & 1, 114);
          ++q_uses[1];
          scores(0, 0, 0, true, false);
          scores(1, 1, 0, false, true);
          if (n == 1) mma_commit(bar(C::QEMPTY));
          for (int i = 0; i < n && ok; ++i) {
            products(0, 0, i, i == 0, true, false);
            if (i + 1 < n) scores(0, 0, i + 1, true, false);
            else mma_commit(bar(C::OFULL));
            products(1, 1, i, i == 0, false, true);
            if (i + 1 < n) {
              scores(1, 1, i + 1, false, true);
              if (i + 2 == n) mma_commit(bar(C::QEMPTY));
            } else {
              mma_commit(bar(C::OFULL + 1));
            }
          }
        } else {
          scores(0, 0, 0, true, true);
          if (n > 1) scores(1, 0, 1, true, true);
          if (n <= 2) mma_commit(bar(C::QEMPTY));
          for (int i = 0; i < n && ok; ++i) {
            const int x = i & 1;
            products(x, NS == 2 ? x : 0, i, NS == 2 ? i < 2 : i == 0, true, true);
            if (NS == 1) mma_commit(bar(C::PVDONE + x));
            if (i + 2 < n) {
              scores(x, 0, i + 2, true, true);
              if (i + 3 == n) mma_commit(bar(C::QEMPTY));
            }
            if (NS == 2 ? i + 2 >= n : i + 1 == n) mma_commit(bar(C::OFULL + (NS == 2 ? x : 0)));
          }
        }
        at += (uint32_t)(2 * n * NBLK);
      }
      __syncwarp();
    }
    if (lane == 0) {
      // nothing this thread issued may still run when tensor memory is given back
      mma_commit(bar(C::DRAIN));
      if (!mbar_wait(bar(C::DRAIN), 0)) report(115);
    }
    __syncwarp();
  } else if (FEED == kTma && warp == 4 * NS + 1) {
    // ------------------------------------------------------------ TMA boxes
    // A lane issues one box: rows `box` of the tile, 64 columns.
    uint32_t at = 0, issued = 0;
    const int nbox = kBN / maps.box;
    const int rb = lane % nbox, ch = lane / nbox;
    for (; w.next(p, g); w.advance(p, g)) {
      const int n = g.t1 - g.t0;
      const Unit& u = g.unit;
      const int kvh = w.at.kvh;
      const Seen seen(p, w.seq, u);
      // this lane's page of tile i (num_pages, all of whose boxes read zeros, for an id
      // outside the pool) and its first row there, where somebody sees these rows
      auto look = [&](int i, int& id, int& row) {
        const int pos = (u.tile0 + g.t0 + i) * kBN + rb * maps.box;
        id = -1;
        row = 0;
        if (i >= n || pos >= u.hi || pos + maps.box <= u.lo) return;
        const int pg = p.page_div(pos);
        row = pos - pg * p.page;
        id = p.table[(int64_t)w.at.b * p.width + pg];
      };
      auto load = [&](const CUtensorMap* map, int place, int id, int row, bool have, int full) {
#pragma unroll
        for (int blk = 0; blk < NBLK; ++blk) {
          const uint32_t pos = at + (uint32_t)(place * NBLK + blk), sl = pos % NB;
          if (pos >= NB) wait_or_fail(ok, bar(C::EMPTY + sl), (pos / NB - 1) & 1, 120);
          ok = __all_sync(~0u, ok);
          if (!ok) return;
          issued = pos + 1;
          const bool mine = have && ch < (DP - 128 * blk < 128 ? (DP - 128 * blk) / 64 : C::BW / 64);
          const unsigned all = __ballot_sync(~0u, mine);
          if (lane == 0)
            mbar_arrive_expect_tx(bar(full + sl), (uint32_t)__popc(all) * maps.box * 128);
          __syncwarp();
          if (mine)
            tma_load_4d(sRing + sl * C::SLOT + ch * 16384 + rb * maps.box * 128, map,
                        bar(full + sl), 128 * blk + 64 * ch, row, kvh, id);
        }
      };
      auto visible = [&](int i) {
        const int pos = (u.tile0 + g.t0 + i) * kBN + rb * maps.box;
        return i < n && pos < u.hi && pos + maps.box > u.lo;
      };
      auto valid = [&](int id) {
        if (id >= 0 && id < p.num_pages) return id;
        report(kBadPageSite);
        return p.num_pages;
      };
      // ids are asked for two tiles ahead
      int id0, row0, id1, row1, id2, row2;
      look(0, id0, row0);
      look(1, id1, row1);
      bool have0 = visible(0);
      if (have0) id0 = valid(id0);
      if (n > 0) load(&maps.k, k_place(0), id0, row0, have0, C::FULL);
      for (int i = 0; i < n && ok; ++i) {
        look(i + 2, id2, row2);
        const bool have1 = visible(i + 1);
        if (i + 1 < n) {
          if (have1) id1 = valid(id1);
          load(&maps.k, k_place(i + 1), id1, row1, have1, C::FULL);
        }
        load(&maps.v, v_place(i, n), id0, row0, have0,
             seen.edge((u.tile0 + g.t0 + i) * kBN) ? C::LANDED : C::FULL);
        id0 = id1;
        row0 = row1;
        have0 = have1;
        id1 = id2;
        row1 = row2;
      }
      at += (uint32_t)(2 * n * NBLK);
      if (!ok) break;
    }
    // nothing may still be landing when the CTA exits
    for (uint32_t pos = issued > NB ? issued - NB : 0; pos < issued; ++pos)
      mbar_wait(bar(C::FULL + pos % NB), (pos / NB) & 1);
  } else if (FEED != kConvert && warp == 4 * NS + 2) {
    // -------------------------------------------------- V where rows are hidden
    // (its blocks arrive on a barrier of their own, the ring's is for the MMA)
    uint32_t at = 0, uses = 0;
    int seg = 0;
    for (; w.next(p, g); w.advance(p, g)) {
      const int n = g.t1 - g.t0;
      const Unit& u = g.unit;
      if (n == 0) continue;
      const Seen seen(p, w.seq, u);
      for (int i = 0; i < n && ok; ++i) {
        const int pos0 = (u.tile0 + g.t0 + i) * kBN;
        if (!seen.edge(pos0)) continue;
        for (int blk = 0; blk < NBLK && ok; ++blk) {
          const uint32_t pos = at + (uint32_t)(v_place(i, n) * NBLK + blk), sl = pos % NB;
          wait_or_fail(ok, bar(C::LANDED + sl), (uses >> sl) & 1, 130);
          uses ^= 1u << sl;
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          const int chunks = (DP - 128 * blk < 128 ? DP - 128 * blk : C::BW) / 64;
          bool met = false;
          // (a 16-byte column of 64-column part c, rows lane / 8 + 4 k: whole lines per warp)
          for (int c = 0; c < chunks; ++c) {
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
              const int row = 4 * k + (lane >> 3);
              const uint32_t a = sRing + sl * C::SLOT + c * 16384 + row * 128 + (lane & 7) * 16;
              if (pos0 + row < u.lo || pos0 + row >= u.hi) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u)
                             : "memory");
                continue;
              }
              uint32_t x[4];
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                           : "r"(a)
                           : "memory");
              uint32_t bad = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t mask = __vcmpeq2(x[e] & 0x7F807F80u, 0x7F807F80u);
                bad |= mask;
                x[e] &= ~mask;
              }
              if (bad) {
                met = true;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x[0]),
                             "r"(x[1]), "r"(x[2]), "r"(x[3])
                             : "memory");
              }
            }
          }
          if (met) dirty[seg & 7] = seg;
          fence_async_shared();
          __syncwarp();
          if constexpr (FEED == kTma) {
            if (lane == 0) mbar_arrive(bar(C::FULL + sl));
          } else {
            for (int k = 0; k < C::FEEDERS / 32; ++k) mbar_arrive(bar(C::FULL + sl));
          }
        }
      }
      ++seg;
      at += (uint32_t)(2 * n * NBLK);
    }
  } else if (FEED != kTma) {
    // ---------------------------------------------------- rows one by one
    // kRows: warps 1 and 3 behind the MMA warp; kConvert: warps 1, 2 and 3.
    const int wi = warp - 4 * NS - 1;
    const int tid = (FEED == kRows ? wi / 2 : wi) * 32 + lane;
    constexpr int EB = FEED == kConvert ? 1 : 2;  // bytes of a cached element
    // The blocks of this share in the ring's order.
    struct Blocks {
      Walk w;
      Segment g;
      int n, i, blk;
      bool value, more;
      uint32_t pos;
      int seg;
      __device__ __forceinline__ void settle(const Params& p) {
        while ((more = w.next(p, g))) {
          n = g.t1 - g.t0;
          if (n > 0) break;
          w.advance(p, g);
        }
        i = 0;
        blk = 0;
        value = false;
      }
      __device__ __forceinline__ void begin(const Params& p, int cta) {
        w.begin(p, cta);
        pos = 0;
        seg = 0;
        settle(p);
      }
      __device__ __forceinline__ void step(const Params& p) {
        ++pos;
        if (++blk < NBLK) return;
        blk = 0;
        // K0 K1 V0 K2 V1 .. V(n-1): i is the tile
        if (value) {
          if (i == n - 1) {
            w.advance(p, g);
            ++seg;
            settle(p);
            return;
          }
          if (i + 2 < n) {
            i += 2;
            value = false;
          } else {
            i += 1;
          }
        } else if (i == 0 && n > 1) {
          i = 1;
        } else {
          value = true;
          i = i == 0 ? 0 : i - 1;
        }
      }
      __device__ __forceinline__ int pos0() const { return (g.unit.tile0 + g.t0 + i) * kBN; }
    };
    // Calls f(row, chunk, element offset or -1) for this thread's 16-byte chunks of a block.
    auto chunks_of = [&](const Blocks& z, auto f) {
      constexpr int E = 16 / EB;
      const bool narrow = DP - 128 * z.blk < 128 && DP > 128;  // the 64 columns behind 128
      const int per_row = (narrow ? 64 : C::BW) / E;
      const int c = tid % per_row, step = C::FEEDERS / per_row;
      const int pos0 = z.pos0(), kvh = z.w.at.kvh, col = 128 * z.blk + c * E;
      const int64_t head = kvh * p.head_stride + col;
#pragma unroll 4
      for (int row = tid / per_row; row < kBN; row += step) {
        const int pos = pos0 + row;
        int64_t off = -1;
        if (pos >= z.g.unit.lo && pos < z.g.unit.hi && col < p.dim) {
          const int pg = p.page_div(pos);
          const int id = p.table[(int64_t)z.w.at.b * p.width + pg];
          if (id >= 0 && id < p.num_pages)
            off = id * p.page_stride + (int64_t)(pos - pg * p.page) * p.row_stride + head;
          else
            report(kBadPageSite);
        }
        f(row, c, off);
      }
    };
    if constexpr (FEED == kRows) {
      Blocks z;
      for (z.begin(p, cta); z.more && ok; z.step(p)) {
        const uint32_t sl = z.pos % NB;
        if (z.pos >= NB) wait_or_fail(ok, bar(C::EMPTY + sl), (z.pos / NB - 1) & 1, 121);
        if (!ok) break;
        const char* base = (const char*)(z.value ? p.v : p.k);
        chunks_of(z, [&](int row, int c, int64_t off) {
          cp_async16(sRing + sl * C::SLOT + (c >> 3) * 16384 + sw128_offset(row, (c & 7) * 8),
                     off >= 0 ? base + off * EB : base, off >= 0 ? 16u : 0u);
        });
        const bool edge = z.value && Seen(p, z.w.seq, z.g.unit).edge(z.pos0());
        cp_async_mbar_arrive(bar((edge ? C::LANDED : C::FULL) + sl));
      }
      cp_async_wait_all();
    } else if constexpr (FEED == kConvert) {
      // A thread converts the very chunks that it copied, so the staging ring needs no
      // barriers: its own groups of copies order it.
      constexpr int RS = C::RS;
      Blocks ahead, z;
      ahead.begin(p, cta);
      z.begin(p, cta);
      auto raw_at = [&](uint32_t pos, int row, int c) {
        return sRaw + (pos % RS) * C::RAW + row * C::BW + c * 16;
      };
      auto ask = [&]() {
        if (ahead.more) {
          const char* base = (const char*)(ahead.value ? p.v : p.k);
          chunks_of(ahead, [&](int row, int c, int64_t off) {
            cp_async16(raw_at(ahead.pos, row, c), off >= 0 ? base + off : base,
                       off >= 0 ? 16u : 0u);
          });
          ahead.step(p);
        }
        cp_async_commit();
      };
      for (int k = 0; k < RS - 1; ++k) ask();
      for (; z.more && ok; z.step(p)) {
        ask();
        cp_async_wait_group<RS - 1>();
        const uint32_t sl = z.pos % NB;
        if (z.pos >= NB) wait_or_fail(ok, bar(C::EMPTY + sl), (z.pos / NB - 1) & 1, 122);
        if (!ok) break;
        const Seen seen(p, z.w.seq, z.g.unit);
        const bool edge = z.value && seen.edge(z.pos0());
        bool met = false;
        const bool narrow = DP - 128 * z.blk < 128 && DP > 128;
        const int per_row = (narrow ? 64 : C::BW) / 16;
        const int c = tid % per_row;
#pragma unroll 4
        for (int row = tid / per_row; row < kBN; row += C::FEEDERS / per_row) {
          uint32_t x[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(raw_at(z.pos, row, c))
                       : "memory");
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t nan = __vcmpeq4(x[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              met |= nan != 0;
              x[e] &= ~nan;
            }
          }
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_half2(x[e], y[2 * e], y[2 * e + 1]);
          const uint32_t part = sRing + sl * C::SLOT + (c >> 2) * 16384;
          const int c8 = (c & 3) * 2;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           part + sw128_offset(row, c8 * 8)),
                       "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           part + sw128_offset(row, c8 * 8 + 8)),
                       "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                       : "memory");
        }
        if (met) dirty[z.seg & 7] = z.seg;
        fence_async_shared();
        mbar_arrive(bar(C::FULL + sl));
      }
      cp_async_wait_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * NS) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int DP, int FEED>
cudaError_t launch(const Params& p, int ctas, cudaStream_t stream) {
  using C = Shape<DP, FEED>;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto* fn = chunk_sm103_kernel<DP, FEED>;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  Maps maps = {};
  if (FEED == kTma) {
    maps.box = p.page & -p.page;
    if (maps.box > kBN) maps.box = kBN;
    // (the stride of a dimension of one element is not used: any multiple of 16 bytes will do)
    auto stride = [&](int64_t elements, int extent) {
      return extent > 1 ? (uint64_t)elements * 2 : (uint64_t)((p.dim * 2 + 15) / 16 * 16);
    };
    const uint64_t dims[4] = {(uint64_t)p.dim, (uint64_t)p.page, (uint64_t)p.kv_heads,
                              (uint64_t)p.num_pages};
    const uint64_t strides[3] = {stride(p.row_stride, p.page), stride(p.head_stride, p.kv_heads),
                                 stride(p.page_stride, p.num_pages)};
    const uint32_t box[4] = {64, (uint32_t)maps.box, 1, 1};
    if (!make_tmap_bf16_4d(&maps.k, p.k, dims, strides, box) ||
        !make_tmap_bf16_4d(&maps.v, p.v, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  KernelTimer kt("chunk_sm103", stream);
  return launch_dependent(fn, dim3((unsigned)ctas), dim3(C::THREADS), C::SMEM, stream, p, maps);
}

template <int FEED, int DP>
Kernel make() {
  using C = Shape<DP, FEED>;
  return {C::BM, kBN, DP, C::THREADS, C::SMEM, 1, launch<DP, FEED>};
}

template <int FEED>
Kernel pick(int dim) {
  return dim <= 64    ? make<FEED, 64>()
         : dim <= 128 ? make<FEED, 128>()
         : dim <= 192 ? make<FEED, 192>()
                      : make<FEED, 256>();
}

int read_status(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_status, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace
}  // namespace chunk
}  // namespace mla
