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
//   kTma      one warp's TMA boxes, page by page, where pages are whole runs of 8
//             rows (page sizes with a power of two of 8 or more in them)
//   kRows     16-byte copies of single rows by four warps, for any other page size
//   kConvert  e4m3: TMA boxes (of any page's rows) into a staging ring, and from there
//             as fp16 by four warps
// Rows that nobody sees, and elements of V that are not finite in a tile where a
// row is hidden from some query, are set to zero before P V reads them (0 times
// such an element is NaN); the latter are put back at the end, for the rows that
// see them.
//
// Measured in a graph, 128 wide: a causal prompt of 8192 rows, 32 heads on 8, 395 to 398 us
// = 1390 TFLOP/s (0.72 of a library product's rate; call by call 417); 24 prompts and steps
// over an e4m3 cache, 64 heads on 8, 731 us; 16 rows at 131072 positions, 32 heads on 4, 64
// us = 4.2 TB/s; 16 steps of 1 to 8 rows 33.6 us.  What bounds the long ones is the chain of
// a tile: S, its maximum (9 % of the time), its exponentials (5 %), P, O; the matrix pipe
// is busy two thirds of the time.  And a unit takes 6 to 8 tiles' time beside its tiles:
// O is waited for and written, the next queries are read, and only then its first S
// begins, nothing of which overlaps but K and V in the ring.  With 6.7 units and 219 tiles
// a CTA that is 15 to 20 % of the prompt.
// Other forms, 16 steps of 1 to 8 rows, 32 heads on 8, other inputs each time (us, share of
// the copy rate): bf16 40 (0.50), e4m3 53 (0.22), bf16 in pages of 20 by rows 119 (0.16),
// e4m3 in pages of 17, a box a row, 221 (0.05); 192 wide 65 and 94 (e4m3), 256 wide 70 and
// 80.  So a step over an e4m3 cache, half the bytes, takes longer than over a bf16 one: its
// conversion, four warps with one block at a time, is slower than the memory.
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
  static constexpr int RAW = FEED == kConvert ? kBN * 128 : 0;  // a block's bytes, 128 a row
  static constexpr int NB =
      FEED == kConvert ? (DP == 64 ? 6 : 4) : (DP == 64 ? 10 : 5);
  static constexpr int RS = FEED == kConvert ? 2 : 0;
  static_assert(NB >= (NBLK == 1 ? 3 : 2 * NBLK), "the ring is too short");
  // warps: softmax, then the MMA issuer, the TMA boxes, two for V where rows are hidden, and
  // four that copy or convert
  static constexpr int MMA = 4 * NS, TMA = MMA + 1, CLEAN = MMA + 2, FEEDER = MMA + 4;
  static constexpr int FEEDERS = FEED == kTma ? 0 : 128;
  static constexpr int THREADS = FEEDER * 32 + FEEDERS;
  // 16 warps start with 128 registers a thread: 152 for the softmax, 104 for the others
  static constexpr bool SHARES = THREADS == 512;
  static constexpr uint32_t TM_S = NS * DP;           // tensor memory: O, then two of S
  static constexpr int TAIL = 1024 + (FEED == kConvert ? NS * 128 * 4 : 0);
  static constexpr int SMEM = 1024 + NS * QB + NB * SLOT + RS * RAW + TAIL;
  static_assert(SMEM <= 232448, "more shared memory than a CTA may have");
  static_assert(TM_S + 256 <= 512, "more tensor memory than there is");
  // barriers
  static constexpr int FULL = 0, EMPTY = NB, LANDED = 2 * NB, RFULL = 3 * NB, REMPTY = RFULL + RS,
                       QFULL = REMPTY + RS, SFULL = QFULL + 1, PHALF = SFULL + 2,
                       PFULL = PHALF + 2, OFULL = PFULL + 2, PVDONE = OFULL + 2,
                       DRAIN = PVDONE + 2, BARS = DRAIN + 1;
  static_assert(BARS * 8 + 10 * 4 + 4 * NS * sizeof(Walk) <= 1024, "the barriers do not fit");
};

struct Maps {
  CUtensorMap k, v;
  int box;  // rows of a box
};

// A block of a ring of N and the phase of its barriers.
struct Slot {
  uint32_t i, phase;
  template <int N>
  __device__ __forceinline__ void move(uint32_t by) {  // by at most 2 N
    i += by;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (i >= N) {
        i -= N;
        phase ^= 1;
      }
    }
  }
  template <int N>
  __device__ __forceinline__ void move_far(uint32_t by) {
    i += by;
    phase ^= (i / N) & 1;
    i %= N;
  }
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
      mbar_init(bar(C::FULL + i), FEED == kTma ? 2 : C::FEEDERS);
      mbar_init(bar(C::EMPTY + i), 1);
      mbar_init(bar(C::LANDED + i), FEED == kTma ? 1 : C::FEEDERS);
    }
    for (int i = 0; i < C::RS; ++i) {
      mbar_init(bar(C::RFULL + i), 1);
      mbar_init(bar(C::REMPTY + i), C::FEEDERS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::SFULL + i), 1);
      mbar_init(bar(C::PHALF + i), 128);
      mbar_init(bar(C::PFULL + i), 128);
      mbar_init(bar(C::OFULL + i), 1);
      mbar_init(bar(C::PVDONE + i), 1);
    }
    mbar_init(bar(C::QFULL), 128 * NS);
    mbar_init(bar(C::DRAIN), 1);
    for (int i = 0; i < 8; ++i) dirty[i] = -1;
    fence_mbar_init();
  }
  if (warp == C::MMA) tmem_alloc(smem_u32(slot_word), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot_word;
  pdl_wait();
  Start from, to;
  Sequence seq = {0, 0, 0, 0, 0};
  if (p.starts == nullptr) {
    // (the place of the queries, which come later)
    find_share(p, cta, *reinterpret_cast<PlanScratch*>(smem), from, to, seq);
  } else {
    read_share(p, cta, *reinterpret_cast<PlanScratch*>(smem), from, to, seq);
  }
  Walk w;
  Segment g;
  w.begin(from, to, seq);
  bool ok = true;

  if (warp >= 4 * NS) {
    if constexpr (C::SHARES) regs_dec<104>();
  }
  if (warp < 4 * NS) {
    // ------------------------------------------------------------- softmax
    if constexpr (C::SHARES) regs_inc<152>();
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
        // (one that is no finite number makes its heads' queries NaN, not the scale: a hidden
        // score times that would be NaN too)
        ksign = !isfinite(ks) ? NAN : ks < 0.f ? -1.f : 1.f;
        if (isfinite(ks)) sl2 *= fabsf(ks);
      }
      // This stream's queries.  The products that read the ones before are done, and
      // with both streams' arrivals everything of the segment before is.
      if (n > 0 && (!split || s == 0)) {
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
#pragma unroll 8
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
          constexpr int AT_ONCE = 4;
#pragma unroll 1
          for (int k0 = 0; k0 < LPR; k0 += AT_ONCE) {
            uint4 x[AT_ONCE];
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
              const int row = row0 + (k0 + k) * (32 / LPR) + lane / LPR, c = lane % LPR;
              bool have;
              const __nv_bfloat16* src = source(row, c, have);
              x[k] = make_uint4(0u, 0u, 0u, 0u);
              if (have) x[k] = *reinterpret_cast<const uint4*>(src);
            }
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
              const int row = row0 + (k0 + k) * (32 / LPR) + lane / LPR, c = lane % LPR;
              const uint32_t word[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
              float f[8], most = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(word[e] << 16);
                f[2 * e + 1] = __uint_as_float(word[e] & 0xFFFF0000u);
                most = fmaxf(most, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
              }
#pragma unroll
              for (int o = LPR / 2; o > 0; o >>= 1)
                most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
              // 2^-exponent of the largest; the row's scores are scaled back.  (Both factors are
              // normal numbers: beside subnormal queries, whose few bits fp16 holds as they are,
              // and beside an infinite one, whose row's scores are no finite numbers anyway, the
              // other elements stay finite.)
              float down = 1.f, up = 1.f;
              if (most > 0.f) {
                const int ex = min(max((int)(__float_as_uint(most) >> 23) - 127, -120), 120);
                down = __uint_as_float((uint32_t)(127 - ex) << 23);
                up = __uint_as_float((uint32_t)(127 + ex) << 23);
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
        }
        fence_async_shared();
      }
      if (n > 0) mbar_arrive(bar(C::QFULL));
      if constexpr (HALF) {
        if (n > 0) {
          if (split) named_bar_sync(1, 256);  // stream 1 reads the scales stream 0 wrote
          else __syncwarp();
          sl2 *= q_scale[r];
          // (one that vanishes leaves hidden scores, minus infinity, below the others)
          if (sl2 < 1e-37f) sl2 = 1e-37f;
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
        // f(scores, piece) for the four pieces; the first one is under way.  (A loop: code
        // that stays in the instruction cache beside the MMA warp's is worth more than the
        // few instructions that an unrolled form saves.)
        auto pieces = [&](auto f) {
#pragma unroll 1
          for (int k = 0; k < 4; k += 2) {
            tmem_wait_ld<32>(u0);
            tmem_ld32(tS + 32 * (k + 1), u1);
            f(u0, k);
            tmem_wait_ld<32>(u1);
            if (k == 0) tmem_ld32(tS + 64, u0);
            f(u1, k + 1);
          }
        };
        // bit j: this row sees column j of piece k
        auto sees = [&](int k) {
          const int a = first - (pos0 + 32 * k), z = last - (pos0 + 32 * k);
          uint32_t bits = z < 0 || a > 31 ? 0u : z >= 31 ? ~0u : (2u << z) - 1u;
          if (a > 0) bits &= ~0u << (a & 31);
          return bits;
        };
        auto hide = [&](uint32_t* u, uint32_t bits) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(bits >> j & 1u)) u[j] = 0xFF800000u;
        };
        auto highest = [&](const uint32_t* u) {
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            t4[(j >> 1) & 3] = fmaxf(t4[(j >> 1) & 3],
                                     fmaxf(__uint_as_float(u[j]), __uint_as_float(u[j + 1])));
        };
        if (edge) {
          // (few tiles: a loop of its own, so that the code of the others stays together)
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            const uint32_t bits = sees(k);
            if (!__any_sync(~0u, bits != 0u)) continue;
            tmem_ld32(tS + 32 * k, u0);
            tmem_wait_ld<32>(u0);
            if (!__all_sync(~0u, bits == ~0u)) hide(u0, bits);
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
        auto store = [&](const uint32_t (&pk)[16], int k) {
          tmem_st16(tS + 16 * k, pk);
          if (k & 1) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar((k == 1 ? C::PHALF : C::PFULL) + x));
          }
        };
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
          store(pk, k);
        };
        if (edge || large) {
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            const uint32_t bits = sees(k);
            tmem_wait_ld<32>(u0);
            if (!__any_sync(~0u, bits != 0u)) {
              uint32_t none[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) none[e] = 0u;
              store(none, k);
            } else {
              if (!__all_sync(~0u, bits == ~0u)) hide(u0, bits);
              if (large) weights(u0, k, std::true_type());
              else weights(u0, k, std::false_type());
            }
            if (k < 3) tmem_ld32(tS + 32 * (k + 1), u0);
          }
        } else {
          pieces([&](uint32_t* u, int k) { weights(u, k, std::false_type()); });
        }
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
      float f0 = 1.f, f1 = 0.f;
      int c0 = 0, c1 = DP;
      if (split) {
        // The streams' sums meet, each half of the columns in one of them; a row's maximum
        // and sum go to the other stream through the scores' tensor memory.
        uint32_t z[16] = {__float_as_uint(m), __float_as_uint(any ? l : 0.f)};
        tmem_st16(tmem + lane_base + C::TM_S + 128 * s, z);
        tmem_wait_st();
        tc_fence_before();
        named_bar_sync(1, 256);
        tc_fence_after();
        tmem_ld16(tmem + lane_base + C::TM_S + 128 * (s ^ 1), z);
        tmem_wait_ld<16>(z);
        const float zm = __uint_as_float(z[0]), zl = __uint_as_float(z[1]);
        const float mm = fmaxf(m, zm), ref = mm == -INFINITY ? 0.f : mm;
        f0 = ex2(m - ref);
        f1 = ex2(zm - ref);
        l = l * f0 + zl * f1;
        m = mm;
        c0 = s * (DP / 2);
        c1 = c0 + DP / 2;
      }
      const bool second = split && n > 1;  // stream 1 has an accumulator
      // (both streams' products are done: the other's tiles may have been the odd ones)
      const bool fix = n > 0 && dirty[seg & 7] == seg;
      const float vs = HALF && p.v_scale ? p.v_scale[kvh] : 1.f;
      const float inv = l == 0.f ? 0.f : vs / l;
      const bool live = r < rows, none = __any_sync(~0u, l == 0.f);
      const int i_tok = p.group_div(u.r0 + min(r, rows - 1)),
                head_in = u.r0 + min(r, rows - 1) - i_tok * p.group;
      const int64_t head = (int64_t)(sq.row0 + i_tok) * p.heads + kvh * p.group + head_in;
      const int64_t part = (int64_t)(2 * cta + (g.first ? 1 : 0)) * p.bm + r;
      // the accumulators' weights: mine and the other stream's
      const float wa = split && s == 1 ? f1 : f0, wb = split && s == 1 ? f0 : f1;
      // 32 columns at a time through shared memory (the place of this warp's queries), so
      // that a row's columns leave side by side.
      const uint32_t stage = sQ + s * C::QB + (warp & 3) * 4096;
      const int row0 = (split ? 0 : 128 * s) + (warp & 3) * 32;
      const int rows_here = min(max(rows - row0, 0), 32);
      // where this lane's four rows go (whole: four 8-column vectors of a row side by side)
      int64_t out_at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 8 * k + (lane >> 2), x = u.r0 + row0 + row;
        const int i = p.group_div(x), j = x - i * p.group;
        out_at[k] = row < rows_here
                        ? ((int64_t)(sq.row0 + i) * p.heads + kvh * p.group + j) * p.dim +
                              8 * (lane & 3)
                        : -1;
      }
      float* part_at = p.part_o + ((int64_t)(2 * cta + (g.first ? 1 : 0)) * p.bm + row0) * p.dp;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t o[32];
        __syncwarp();
        if (n > 0) {
          tmem_ld32(tmem + lane_base + (NS == 2 && !split ? DP * s : 0) + c, o);
          if (second) {
            uint32_t o1[32];
            tmem_ld32(tmem + lane_base + DP + c, o1);
            tmem_wait_ld<32>(o);
            tmem_wait_ld<32>(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), wb, __uint_as_float(o[e]) * wa));
          } else {
            tmem_wait_ld<32>(o);
          }
        }
        if (none && whole) {  // (a part's weights may all be zero while another's are not)
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0u : o[e];
        }
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = pack_bf16(__uint_as_float(o[e + 2 * k]) * inv,
                               __uint_as_float(o[e + 2 * k + 1]) * inv);
            const uint32_t at = stage + lane * 64 + (((e / 8) ^ ((lane >> 1) & 3)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]),
                         "r"(y[1]), "r"(y[2]), "r"(y[3])
                         : "memory");
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const uint32_t at = stage + lane * 128 + (((e / 4) ^ (lane & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[e]),
                         "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3])
                         : "memory");
          }
        }
        if (fix && live && (l != 0.f || !whole)) {
          // what was set to zero, added to the staged values
          const int lo = max(first, (u.tile0 + g.t0) * kBN),
                    hi = min(last, (u.tile0 + g.t1) * kBN - 1);
#pragma unroll 1
          for (int e = 0; e < 32 && c + e < p.dim; ++e) {
            const float y = odd_values<FEED>(p, w.at.b, kvh, c + e, lo, hi, seen.lo, seen.hi);
            if (y == 0.f) continue;
            if (whole) {
              __nv_bfloat16* v = reinterpret_cast<__nv_bfloat16*>(
                  smem + (stage - sQ) + lane * 64 + (((e / 8) ^ ((lane >> 1) & 3)) << 4) +
                  (e & 7) * 2);
              *v = __float2bfloat16(__bfloat162float(*v) + y * inv);
            } else {
              float* v = reinterpret_cast<float*>(smem + (stage - sQ) + lane * 128 +
                                                  (((e / 4) ^ (lane & 7)) << 4) + (e & 3) * 4);
              *v += y;
            }
          }
        }
        __syncwarp();
        auto staged = [&](uint32_t at) {
          uint4 x;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                       : "r"(at)
                       : "memory");
          return x;
        };
        if (whole) {
          const uint32_t from = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // rows 8 k + lane / 4
            if (out_at[k] >= 0 && c + 8 * (lane & 3) < p.dim)
              *reinterpret_cast<uint4*>((__nv_bfloat16*)p.out + out_at[k] + c) =
                  staged(from + k * 512);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = 4 * k + (lane >> 3), ch = lane & 7;
            if (row < rows_here)
              *reinterpret_cast<uint4*>(part_at + row * p.dp + c + 4 * ch) =
                  staged(stage + row * 128 + ((ch ^ (row & 7)) << 4));
          }
        }
        __syncwarp();
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
  } else if (warp == C::MMA) {
    // ----------------------------------------------------------------- MMA
    // The whole warp walks and waits, so that descriptors are uniform registers, and one
    // thread of it issues for both streams in turn, O += P V of a tile and S of the next
    // one.  (An issuer for each, whose instructions the pipe takes alternately, made
    // both streams wait longer: 8192 rows 649 us against 579.)
    const uint32_t id_s = HALF ? idesc_f16(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0);
    const int nk = (p.dim + 15) / 16;  // steps of 16 columns
    const bool full_width = nk == DP / 16;
    const bool leader = elect_one();
    Slot ring = {0, 0};            // of this segment's first block
    uint32_t before[2] = {0, 0};   // tiles of each stream (or S buffer) before it
    uint32_t seg = 0;
    // (what the thread does between two tiles' instructions is what the pipe waits for:
    // few waits, and few instructions)
    const uint64_t dk0 = sdesc_sw128(sRing, 16, 1024), dv0 = sdesc_sw128(sRing, 16384, 1024);
    const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
    const uint32_t first_n = (min(p.dim, C::BW) + 15) & ~15, last_n = (p.dim - 128 + 15) & ~15;
    for (; w.next(p, g); w.advance(p, g)) {
      const int n = g.t1 - g.t0, rows = g.unit.r1 - g.unit.r0;
      if (n == 0) continue;
      const bool split = NS == 2 && rows <= 128;
      {
        auto landed = [&](const Slot& t) {
          wait_or_fail(ok, bar(C::FULL + t.i), t.phase, 110);
          if (FEED == kRows) fence_async_shared();
        };
        // S = Q K^T of the tile at `t`.  `wait`: its first use, `free`: its last one
        auto scores = [&](int x, uint64_t dq, Slot t, bool wait, bool free) {
          const uint32_t dst = tmem + C::TM_S + 128 * x;
#pragma unroll
          for (int blk = 0; blk < NBLK; ++blk) {
            if (blk > 0) t.move<NB>(1);
            if (wait) landed(t);
            if (!ok) return;
            const uint64_t dk = dk0 + (uint64_t)(t.i * (C::SLOT >> 4));
            const uint64_t dqb = dq + (uint64_t)(blk * 2048);
            // (a condition on single MMAs of the unrolled form made the compiler give some of
            // them another one's descriptor: so either all of them, or a loop)
            if (!leader) continue;
            if (full_width) {
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
            if (free) mma_commit(bar(C::EMPTY + t.i));
            if (blk == NBLK - 1) mma_commit(bar(C::SFULL + x));
          }
        };
        // O += P V of the tile at `t`, number j of its stream or S buffer.  The first half
        // of P is enough to begin with.
        auto products = [&](int x, int o, Slot t, int j, bool begin, bool wait, bool free) {
          const uint32_t parity = (before[x] + (uint32_t)j) & 1;
          if (wait) landed(t);
          wait_or_fail(ok, bar(C::PHALF + x), parity, 111);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int blk = 0; blk < NBLK; ++blk) {
            if (blk > 0) {
              t.move<NB>(1);
              if (wait) landed(t);
              if (!ok) return;
            }
            const uint64_t dv = dv0 + (uint64_t)(t.i * (C::SLOT >> 4));
            const uint32_t nn = blk == 0 ? first_n : last_n;
            const uint32_t id_o = HALF ? idesc_f16(128, nn, 0, 1) : idesc_bf16(128, nn, 0, 1);
            const uint32_t dst = tmem + o * DP + 128 * blk, from = tmem + C::TM_S + 128 * x;
            if (leader) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_bf16_tmem_a(dst, from + 8 * k, dv + 128 * k, id_o, !begin || k > 0);
            }
            if (blk == 0) {
              wait_or_fail(ok, bar(C::PFULL + x), parity, 112);
              if (!ok) return;
              tc_fence_after();
            }
            if (leader) {
#pragma unroll
              for (int k = 4; k < 8; ++k)
                mma_bf16_tmem_a(dst, from + 8 * k, dv + 128 * k, id_o, 1);
              if (free) mma_commit(bar(C::EMPTY + t.i));
            }
          }
        };
        // where the next tiles of K and V lie: K0 K1 V0 K2 V1 .. V(n-1)
        Slot kt = ring, vt = ring;
        vt.move<NB>((n == 1 ? 1 : 2) * NBLK);
        wait_or_fail(ok, bar(C::QFULL), seg & 1, 113);
        if (NS == 2 && !split) {
          constexpr uint64_t kTile = C::QB >> 4;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) scores(x, dq0 + x * kTile, kt, x == 0, x == 1);
          kt.move<NB>(NBLK);
          for (int i = 0; i < n && ok; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              products(x, x, vt, i, i == 0, x == 0, x == 1);
              if (i + 1 < n) scores(x, dq0 + x * kTile, kt, x == 0, x == 1);
              else if (leader) mma_commit(bar(C::OFULL + x));
            }
            kt.move<NB>(2 * NBLK);
            vt.move<NB>((i + 2 < n ? 2 : 1) * NBLK);
          }
        } else {
          scores(0, dq0, kt, true, true);
          kt.move<NB>(NBLK);
          if (n > 1) {
            scores(1, dq0, kt, true, true);
            kt.move<NB>(2 * NBLK);
          }
          for (int i = 0; i < n && ok; ++i) {
            const int x = i & 1;
            products(x, NS == 2 ? x : 0, vt, i >> 1, NS == 2 ? i < 2 : i == 0, true, true);
            vt.move<NB>((i + 2 < n ? 2 : 1) * NBLK);
            if (NS == 1 && leader) mma_commit(bar(C::PVDONE + x));
            if (i + 2 < n) {
              scores(x, dq0, kt, true, true);
              kt.move<NB>(2 * NBLK);
            }
            if (leader && (NS == 2 ? i + 2 >= n : i + 1 == n))
              mma_commit(bar(C::OFULL + (NS == 2 ? x : 0)));
          }
        }
        ring.move_far<NB>((uint32_t)(2 * n * NBLK));
        before[0] += (uint32_t)(NS == 2 && !split ? n : (n + 1) >> 1);
        before[1] += (uint32_t)(NS == 2 && !split ? n : n >> 1);
        ++seg;
      }
      __syncwarp();
    }
    if (leader) {
      // nothing that was issued may still run when tensor memory is given back
      mma_commit(bar(C::DRAIN));
      if (!mbar_wait(bar(C::DRAIN), 0)) report(115);
    }
    __syncwarp();
  } else if (FEED != kRows && warp == C::TMA) {
    // ------------------------------------------------------------ TMA boxes
    // A lane issues a box, `box` rows of the tile: 64 bf16 columns, or 128 bytes of e4m3
    // into the staging ring.
    constexpr int SLOTS = FEED == kTma ? NB : C::RS;
    constexpr int TO_FULL = FEED == kTma ? C::FULL : C::RFULL;
    constexpr int TO_EMPTY = FEED == kTma ? C::EMPTY : C::REMPTY;
    uint32_t at = 0, issued = 0;
    const int nbox = kBN / maps.box;
    const bool one_each = nbox <= 32;  // a lane has one box of rows at most
    const int rb = one_each ? lane % nbox : 0, ch = one_each ? lane / nbox : 0;
    for (; w.next(p, g); w.advance(p, g)) {
      const int n = g.t1 - g.t0;
      const Unit& u = g.unit;
      const int kvh = w.at.kvh;
      const Seen seen(p, w.seq, u);
      // the page of rows k of tile i (num_pages, all of whose boxes read zeros, for an id
      // outside the pool) and the first row there, where somebody sees these rows
      auto first_pos = [&](int i, int k) { return (u.tile0 + g.t0 + i) * kBN + k * maps.box; };
      auto visible = [&](int i, int k) {
        const int pos = first_pos(i, k);
        return i < n && pos < u.hi && pos + maps.box > u.lo;
      };
      auto look = [&](int i, int k, int& id, int& row) {
        id = -1;
        row = 0;
        if (!visible(i, k)) return;
        const int pos = first_pos(i, k), pg = p.page_div(pos);
        row = pos - pg * p.page;
        id = p.table[(int64_t)w.at.b * p.width + pg];
      };
      auto valid = [&](int id) {
        if (id >= 0 && id < p.num_pages) return id;
        report(kBadPageSite);
        return p.num_pages;
      };
      auto box_load = [&](const CUtensorMap* map, uint32_t sl, int full, int blk, int k, int c,
                          int row, int id) {
        if constexpr (FEED == kTma)
          tma_load_4d(sRing + sl * C::SLOT + c * 16384 + k * maps.box * 128, map, bar(full + sl),
                      128 * blk + 64 * c, row, kvh, id);
        else
          tma_load_4d(sRaw + sl * C::RAW + k * maps.box * 128, map, bar(full + sl), 128 * blk, row,
                      kvh, id);
      };
      auto load = [&](const CUtensorMap* map, int place, int i, int id, int row, bool have,
                      int full) {
#pragma unroll
        for (int blk = 0; blk < NBLK; ++blk) {
          const uint32_t pos = at + (uint32_t)(place * NBLK + blk), sl = pos % SLOTS;
          if (pos >= SLOTS) wait_or_fail(ok, bar(TO_EMPTY + sl), (pos / SLOTS - 1) & 1, 120);
          ok = __all_sync(~0u, ok);
          if (!ok) return;
          issued = pos + 1;
          const int chunks = FEED == kConvert             ? 1
                             : DP - 128 * blk < 128 ? (DP - 128 * blk) / 64
                                                    : C::BW / 64;
          if (one_each) {
            const bool mine = have && ch < chunks;
            const unsigned all = __ballot_sync(~0u, mine);
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(full + sl), (uint32_t)__popc(all) * maps.box * 128);
              if (FEED == kTma && full == C::FULL) mbar_arrive(bar(full + sl));
            }
            __syncwarp();
            if (mine) box_load(map, sl, full, blk, rb, ch, row, id);
          } else {
            int boxes = 0;
            for (int k = lane; k < nbox; k += 32) boxes += visible(i, k) ? 1 : 0;
            boxes = __reduce_add_sync(~0u, boxes);
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(full + sl), (uint32_t)boxes * maps.box * 128);
              if (FEED == kTma && full == C::FULL) mbar_arrive(bar(full + sl));
            }
            __syncwarp();
            for (int k = lane; k < nbox; k += 32) {
              int id1, row1;
              look(i, k, id1, row1);
              if (visible(i, k)) box_load(map, sl, full, blk, k, 0, row1, valid(id1));
            }
          }
        }
      };
      // ids are asked for two tiles ahead
      int id0, row0, id1, row1, id2, row2;
      look(0, rb, id0, row0);
      look(1, rb, id1, row1);
      bool have0 = visible(0, rb);
      if (have0) id0 = valid(id0);
      if (n > 0) load(&maps.k, k_place(0), 0, id0, row0, have0, TO_FULL);
      for (int i = 0; i < n && ok; ++i) {
        look(i + 2, rb, id2, row2);
        const bool have1 = visible(i + 1, rb);
        if (i + 1 < n) {
          if (have1) id1 = valid(id1);
          load(&maps.k, k_place(i + 1), i + 1, id1, row1, have1, TO_FULL);
        }
        load(&maps.v, v_place(i, n), i, id0, row0, have0,
             FEED == kTma && seen.edge(first_pos(i, 0)) ? C::LANDED : TO_FULL);
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
    for (uint32_t pos = issued > SLOTS ? issued - SLOTS : 0; pos < issued; ++pos)
      mbar_wait(bar(TO_FULL + pos % SLOTS), (pos / SLOTS) & 1);
  } else if (FEED != kConvert && (warp == C::CLEAN || warp == C::CLEAN + 1)) {
    // -------------------------------------------------- V where rows are hidden
    // (its blocks arrive on a barrier of their own, the ring's is for the MMA; two warps, half
    // of the rows each)
    const int row0 = (warp - C::CLEAN) * 64 + (lane >> 3);
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
          // (16-byte columns of whole 64-column lines, four rows of them to a warp's read)
          constexpr int AT_ONCE = 8;
#pragma unroll 1
          for (int k0 = 0; k0 < 16 * chunks; k0 += AT_ONCE) {
            const uint32_t a = sRing + sl * C::SLOT + (k0 >> 4) * 16384 + (lane & 7) * 16;
            uint32_t x[AT_ONCE][4];
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[k][0]), "=r"(x[k][1]), "=r"(x[k][2]), "=r"(x[k][3])
                           : "r"(a + (row0 + 4 * ((k0 & 15) + k)) * 128)
                           : "memory");
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
              const int row = row0 + 4 * ((k0 & 15) + k);
              const bool nobody = pos0 + row < u.lo || pos0 + row >= u.hi;
              uint32_t bad = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t mask = __vcmpeq2(x[k][e] & 0x7F807F80u, 0x7F807F80u);
                bad |= mask;
                x[k][e] = nobody ? 0u : x[k][e] & ~mask;
              }
              met |= bad != 0 && !nobody;
              if (bad != 0 || nobody)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a + row * 128),
                             "r"(x[k][0]), "r"(x[k][1]), "r"(x[k][2]), "r"(x[k][3])
                             : "memory");
            }
          }
          if (met) dirty[seg & 7] = seg;
          fence_async_shared();
          __syncwarp();
          if constexpr (FEED == kTma) {
            if (lane == 0) mbar_arrive(bar(C::FULL + sl));
          } else {
            for (int k = 0; k < C::FEEDERS / 64; ++k) mbar_arrive(bar(C::FULL + sl));
          }
        }
      }
      ++seg;
      at += (uint32_t)(2 * n * NBLK);
    }
  } else if (FEED != kTma && warp >= C::FEEDER) {
    // ------------------------------------------- rows one by one, or conversions
    const int tid = (warp - C::FEEDER) * 32 + lane;
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
      __device__ __forceinline__ void begin(const Params& p, const Walk& whole) {
        w = whole;
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
    Blocks z;
    if constexpr (FEED == kRows) {
      for (z.begin(p, w); z.more && ok; z.step(p)) {
        const uint32_t sl = z.pos % NB;
        if (z.pos >= NB) wait_or_fail(ok, bar(C::EMPTY + sl), (z.pos / NB - 1) & 1, 121);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const __nv_bfloat16* base = (const __nv_bfloat16*)(z.value ? p.v : p.k);
        // 16-byte chunk c of every `step`-th row; the block behind 128 columns may have 64
        const int per_row = DP > 128 && DP - 128 * z.blk < 128 ? 8 : C::BW / 8;
        const int c = tid % per_row, step = C::FEEDERS / per_row;
        const int pos0 = z.pos0(), kvh = z.w.at.kvh, col = 128 * z.blk + c * 8;
        const int64_t head = kvh * p.head_stride + col;
#pragma unroll 4
        for (int row = tid / per_row; row < kBN; row += step) {
          const int pos = pos0 + row;
          const __nv_bfloat16* src = nullptr;
          if (pos >= z.g.unit.lo && pos < z.g.unit.hi && col < p.dim) {
            const int pg = p.page_div(pos);
            const int id = p.table[(int64_t)z.w.at.b * p.width + pg];
            if (id >= 0 && id < p.num_pages)
              src = base + id * p.page_stride + (int64_t)(pos - pg * p.page) * p.row_stride + head;
            else
              report(kBadPageSite);
          }
          cp_async16(sRing + sl * C::SLOT + (c >> 3) * 16384 + sw128_offset(row, (c & 7) * 8),
                     src ? src : base, src ? 16u : 0u);
        }
        const bool edge = z.value && Seen(p, z.w.seq, z.g.unit).edge(pos0);
        cp_async_mbar_arrive(bar((edge ? C::LANDED : C::FULL) + sl));
      }
      cp_async_wait_all();
    } else if constexpr (FEED == kConvert) {
      for (z.begin(p, w); z.more && ok; z.step(p)) {
        const uint32_t sl = z.pos % NB, rs = z.pos % C::RS;
        wait_or_fail(ok, bar(C::RFULL + rs), (z.pos / C::RS) & 1, 123);
        if (z.pos >= NB) wait_or_fail(ok, bar(C::EMPTY + sl), (z.pos / NB - 1) & 1, 122);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        const bool edge = z.value && Seen(p, z.w.seq, z.g.unit).edge(z.pos0());
        const int lo = z.g.unit.lo - z.pos0(), hi = z.g.unit.hi - z.pos0();  // rows that are seen
        bool met = false;
        constexpr int PER_ROW = C::BW / 16;  // 16-element chunks
        const int c = tid % PER_ROW;
        const uint32_t from = sRaw + rs * C::RAW + c * 16;
        const uint32_t to = sRing + sl * C::SLOT + (c >> 2) * 16384;
        const int c8 = (c & 3) * 16;  // the chunk's first column of 64
        constexpr int STEP = C::FEEDERS / PER_ROW, ROUNDS = kBN / STEP;
        const int row0 = tid / PER_ROW;
        auto load = [&](int row, uint32_t (&x)[4]) {
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(from + row * 128)
                       : "memory");
        };
        auto put = [&](int row, const uint32_t (&x)[4]) {
          uint32_t y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_half2(x[e], y[2 * e], y[2 * e + 1]);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + sw128_offset(row, c8)),
                       "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           to + sw128_offset(row, c8 + 8)),
                       "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                       : "memory");
        };
        if (!edge) {
#pragma unroll
          for (int k0 = 0; k0 < ROUNDS; k0 += 4) {
            uint32_t x[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) load(row0 + (k0 + k) * STEP, x[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) put(row0 + (k0 + k) * STEP, x[k]);
          }
        } else {
#pragma unroll 1
          for (int row = row0; row < kBN; row += STEP) {
            uint32_t x[4];
            load(row, x);
            const bool seen_row = row >= lo && row < hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t nan = __vcmpeq4(x[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              met |= seen_row && nan != 0;
              x[e] = seen_row ? x[e] & ~nan : 0u;
            }
            put(row, x);
          }
        }
        if (met) dirty[z.seg & 7] = z.seg;
        mbar_arrive(bar(C::REMPTY + rs));
        fence_async_shared();
        mbar_arrive(bar(C::FULL + sl));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA) {
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
  if (FEED != kRows) {
    constexpr int EB = FEED == kTma ? 2 : 1;
    maps.box = p.page & -p.page;  // the largest power of two in the page size
    if (maps.box > kBN) maps.box = kBN;
    // (the stride of a dimension of one element is not used: any multiple of 16 bytes will do)
    auto stride = [&](int64_t elements, int extent) {
      return (uint64_t)(extent > 1 ? elements : p.dim) * EB;
    };
    const uint64_t dims[4] = {(uint64_t)p.dim, (uint64_t)p.page, (uint64_t)p.kv_heads,
                              (uint64_t)p.num_pages};
    const uint64_t strides[3] = {stride(p.row_stride, p.page), stride(p.head_stride, p.kv_heads),
                                 stride(p.page_stride, p.num_pages)};
    const uint32_t box[4] = {128u / EB, (uint32_t)maps.box, 1, 1};
    auto* make = FEED == kTma ? make_tmap_bf16_4d : make_tmap_u8_4d;
    if (!make(&maps.k, p.k, dims, strides, box) || !make(&maps.v, p.v, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  KernelTimer kt("chunk_sm103", stream);
  return launch_dependent(fn, dim3((unsigned)ctas), dim3(C::THREADS), C::SMEM, stream, p, maps);
}

template <int FEED, int DP>
Kernel make() {
  using C = Shape<DP, FEED>;
  return {C::BM, kBN, DP, 1, kTensorCost, kTensorSnap, launch<DP, FEED>};
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
