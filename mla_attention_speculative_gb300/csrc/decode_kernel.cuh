// Decode attention over a paged key/value cache: the kernel.
//
//   s_t = scale q . k_t,   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// One pass over the cache with a running maximum m and sum.  A key/value
// element is used by the `group` query heads that share it, 2 group flops a
// byte in bf16: far below what the matrix units would need to be the limit,
// so the kernel is built to keep the memory system full.
//
// Measured (128-wide heads, 32 query and 8 key/value heads, DRAM bytes equal to
// the cache rows read once): 32 sequences of 1024 to 32768 positions 328 us,
// 6.77 TB/s, the rate of a plain copy; 16 of up to 4099 positions 25 us, 4.1
// TB/s, of which about 10 us are the start (lengths, page ids and first rows
// are three trips to memory in a row), the merge and the join; T = 131072 49 us,
// 5.5 TB/s; e4m3, 64 sequences with groups of 8 168 us, 5.8 TB/s.
//
// Work.  The cache rows a call reads form segments (sequence, key/value head or
// a few neighbouring ones, row tile of up to ROWS query heads of each), each a
// run of tiles of positions.
// All tiles, in that order, are dealt out in equal contiguous shares to as
// many CTAs as are resident at once, whatever the lengths, so a batch of
// ragged sequences and one long sequence load the machine alike.  The lengths
// are read here, so a captured graph follows them.  A segment that falls into
// several shares leaves its parts (unnormalised sums, m, sum of weights) in
// the workspace, at most two per CTA, and a second kernel joins them in order.
//
// Loads.  Each warp owns a part of every tile and a ring of STAGES of its
// parts in shared memory, filled by 16-byte asynchronous copies (any page
// size, any strides; rows beyond the sequence are zero-filled without being
// read).  The warps share nothing until a segment ends, so there is no
// barrier in the loop, and the copies run on across segments.  The page ids
// of a tile are loaded one tile before its copies need them.
//
// Products.  The heads of a group are few, so they take the narrow side of the
// matrix instruction: S^T = K Q^T and O^T = V^T P^T with positions (head
// elements) as its 16 rows and 8 heads as its columns.  Tiles come from shared
// memory by ldmatrix (chunks of a row XORed with its number, so eight rows'
// chunks lie in different banks), and the weights P^T change from accumulator
// to operand layout by movmatrix.  tcgen05 would need 128 rows of one operand,
// its softmax a trip through tensor memory, and the loop has nothing to gain:
// it waits for DRAM.
//
// Roundings.  bf16: the products are exact in fp32, and the weights enter the
// second product as two bf16 parts, hi + lo (2^-15 relative), so that the
// output's own rounding is the only one that shows.  Both parts are above zero:
// an infinite v gives infinity and not the difference of two (hi rounded to
// nearest would halve the error and leave lo zero or negative half the time).
// e4m3: keys and values become fp16 (exact), queries fp16 scaled
// by a power of two per head (exact down to 2^-24 of the head's largest
// element), weights fp16 scaled by 2^15, so that even many weights far below
// the largest keep their sum.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_attention.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace decode {

using namespace sm103;

static __device__ int g_status;

static int read_status(bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_status, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

struct Span {  // the positions a sequence sees, and its tiles
  int lo, T, n;
};

// TILE: positions of a tile, 0: as the call says.  (A length above 0 has tiles.)
template <int TILE>
__device__ __forceinline__ Span span_of(const Params& p, int b) {
  Span s;
  s.T = (int)min((long long)max(p.lens[b], 0), (long long)p.width * p.page);
  s.lo = p.window > 0 ? max(0, s.T - p.window) : 0;
  s.n = TILE > 0 ? (s.T - s.lo + TILE - 1) / (TILE > 0 ? TILE : 1)
                 : p.tile_div(s.T - s.lo + p.tile - 1);
  return s;
}

// What a sequence's segments count for, each, when the work is dealt out.
__device__ __forceinline__ int cost_of(const Span& s) { return s.n > 0 ? s.n + kSegmentCost : 0; }

// Which blocks of `per` sequences have one with tiles, a bit each.
struct LiveBlocks {
  const uint32_t* words;
  int count, per;
};

// The first sequence behind b with tiles (p.batch: none).  The whole warp calls
// it.  Blocks without one are passed over by their bits, the sequences of a block
// 32 at a time: one by one, a run of 4094 idle slots between two sequences of
// 20064 and 25000 positions cost the CTA whose share spans it 450 us, and the
// call with it (481 us, now 27).
__device__ __forceinline__ int next_live(const Params& p, int b, const LiveBlocks& blocks) {
  const int lane = threadIdx.x & 31;
  int block = b / blocks.per;
  for (int from = b + 1;;) {
    const int to = min(p.batch, (block + 1) * blocks.per);
    for (; from < to; from += 32) {
      const uint32_t live =
          __ballot_sync(~0u, from + lane < to && p.lens[from + lane] > 0);
      if (live != 0) return from + __ffs(live) - 1;
    }
    int w = (block + 1) >> 5;
    if (w >= blocks.count) return p.batch;
    uint32_t bits = blocks.words[w] & (~0u << ((block + 1) & 31));
    while (bits == 0) {
      if (++w == blocks.count) return p.batch;
      bits = blocks.words[w];
    }
    block = w * 32 + __ffs(bits) - 1;
    from = block * blocks.per;
  }
}

// A place in the work: tile j of segment (b, kvg, rt), and its place t in the
// list in which a segment's tiles come behind kSegmentCost places without one.
template <int TILE>
struct Cursor {
  int b, kvg, rt, j;
  long long t;
  Span s;
  // To the next tile; beyond `end` the place alone is right.
  __device__ __forceinline__ void next(const Params& p, long long end, const LiveBlocks& blocks) {
    ++t;
    if (++j < s.n) return;
    t += kSegmentCost;
    if (t >= end) return;
    j = 0;
    if (++rt < p.row_tiles) return;
    rt = 0;
    if (++kvg < p.kv_groups) return;
    kvg = 0;
    if (++b < p.batch) {
      s = span_of<TILE>(p, b);
      if (s.n > 0) return;
      b = next_live(p, b, blocks);
    }
    if (b >= p.batch) {  // (lengths that another kernel changes meanwhile)
      t = end;
      return;
    }
    s = span_of<TILE>(p, b);
  }
};

// Sequences with nothing to see have no tiles: their outputs (and records),
// dealt over the CTAs.
template <int TILE, int KIND>
__device__ __forceinline__ void zero_idle(const Params& p) {
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (span_of<TILE>(p, b).n > 0) continue;
    const int64_t row = (int64_t)p.heads * p.dim * (KIND == kFp32 ? 4 : 2);
    uint4* dst = reinterpret_cast<uint4*>((char*)p.out + b * row);
    for (int i = threadIdx.x; i < row / 16; i += blockDim.x) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (int h = threadIdx.x; h < p.heads; h += blockDim.x)
        p.lse[(int64_t)b * p.heads + h] = -INFINITY;
    if (p.rec && p.by_segment) {
      const int hrs = p.kv_groups * p.row_tiles;
      for (int i = threadIdx.x; i < hrs; i += blockDim.x)
        p.rec[(int64_t)b * hrs + i].parts = 0;
    }
  }
}

// A chunk's place in its row: XORed so that the same chunk of eight successive
// rows lies in eight different 16-byte columns of the banks, whatever CH mod 8.
template <int CH>
__device__ __forceinline__ int swizzle(int row) {
  return CH % 8 == 0 ? (row & 7) : CH % 4 == 0 ? ((row >> 1) & 3) : ((row >> 2) & 1);
}

// Where a lane's row of a tile lies: the page id is loaded, not yet used.
struct RowAt {
  int64_t off;  // within the page, -1: beyond the sequence
  int id;
};

// a / b, a 32-bit division where the values allow.
__device__ __forceinline__ long long div_small(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// HEADS: a tile may hold several key/value heads (p.hg of them).
template <int DP, int KIND, int NT, bool HEADS>
__global__ void __launch_bounds__((Shape<DP, KIND, NT>::THREADS), (Shape<DP, KIND, NT>::OCC))
    decode_attn_sm103(const Params p) {
  using S = Shape<DP, KIND, NT>;
  constexpr int ROWS = S::ROWS, WP = S::WP, CH = S::CH, STAGES = S::STAGES, NW = S::NW;
  constexpr int THREADS = S::THREADS, TILE = HEADS ? 0 : NW * WP;
  const int hg = HEADS ? p.hg : 1, pw = HEADS ? p.pw : NW, tile = HEADS ? p.tile : TILE;
  extern __shared__ __align__(128) char smem[];
  float2* const s_ml = reinterpret_cast<float2*>(smem + S::RING);
  float* const s_q = reinterpret_cast<float*>(smem + S::RING + S::STATS);
  float* const s_w = reinterpret_cast<float*>(smem + S::RING + S::STATS + S::QTILE);
  __shared__ long long s_sum[NW];
  __shared__ uint32_t s_live[NW];
  __shared__ long long s_rem;
  __shared__ int s_b;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // this warp's head of the tile's, and its positions' place in the tile
  const int sub = HEADS ? warp / pw : 0, pos_in_tile = (warp - sub * pw) * WP;
  const uint32_t ring = smem_u32(smem) + warp * STAGES * S::STAGE;
  const int chunks = p.dim * S::CB / 16;  // of a row; the rest of a tile row stays zero
  if (chunks < CH) {
    char* mine = smem + warp * STAGES * S::STAGE;
    for (int i = lane * 16; i < STAGES * S::STAGE; i += 512)
      *reinterpret_cast<uint4*>(mine + i) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share of the tiles
  const int hrs = p.kv_groups * p.row_tiles;
  const int per = (p.batch + THREADS - 1) / THREADS;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  long long mine = 0;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) mine += cost_of(span_of<TILE>(p, b));
  mine *= hrs;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_sum[warp] = upto;
  const uint32_t live_here = __ballot_sync(~0u, mine > 0);
  if (lane == 0) s_live[warp] = live_here;
  const LiveBlocks blocks = {s_live, NW, per};
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) upto += s_sum[w];
    total += s_sum[w];
  }
  const int ctas = (int)min((long long)gridDim.x, total);
  const int cta = blockIdx.x;
  if (cta >= ctas) {
    if (tid == 0 && p.rec && !p.by_segment) p.rec[cta].parts = 0;
    zero_idle<TILE, KIND>(p);
    return;
  }
  // share i is places floor(total i / ctas) up to the next one's first
  const long long quot = div_small(total, ctas);
  const int left = (int)(total - quot * ctas);
  const long long t0 = quot * cta + (uint32_t)(left * cta) / (uint32_t)ctas;
  const long long t1 = quot * (cta + 1) + (uint32_t)(left * (cta + 1)) / (uint32_t)ctas;
  if (upto - mine <= t0 && t0 < upto) {
    long long at = upto - mine;
    int b = b0;
    if (per > 1) {
      for (; b < b1 - 1; ++b) {
        const long long n = (long long)cost_of(span_of<TILE>(p, b)) * hrs;
        if (t0 < at + n) break;
        at += n;
      }
    }
    s_b = b;
    s_rem = t0 - at;
  }
  __syncthreads();
  Cursor<TILE> cc;  // the tile being computed
  cc.b = s_b;
  cc.s = span_of<TILE>(p, cc.b);
  const int hr = (int)div_small(s_rem, cost_of(cc.s));
  const int place = (int)(s_rem - (long long)hr * cost_of(cc.s)) - kSegmentCost;
  cc.j = max(place, 0);
  cc.t = t0 + max(-place, 0);
  cc.kvg = hr / p.row_tiles;
  cc.rt = hr - cc.kvg * p.row_tiles;

  // ---- state of a segment, per lane
  // matrix kinds: heads 8 nt + 2 (lane % 4) + {0, 1}; fp32: all ROWS heads
  constexpr int MT = DP / 16;
  constexpr int NSTAT = KIND == kFp32 ? ROWS : 2 * NT;
  constexpr int NB = (DP + 127) / 128;
  float m[NSTAT], l[NSTAT];
  float o[KIND == kFp32 ? 1 : MT][KIND == kFp32 ? 1 : NT][4];
  float of[KIND == kFp32 ? NB : 1][KIND == kFp32 ? ROWS : 1][4];
  uint32_t qf[KIND == kFp32 ? 1 : MT][KIND == kFp32 ? 1 : NT][2];
  float sc[KIND == kE4m3 ? 2 * NT : 1];  // base-2 scale of a score, per head where it differs
  const int g = lane >> 2, quad = lane & 3;
  bool whole = false;  // the segment began in this share
  int stage = 0;
  Record rec = {0, 0, 0, 0};

  // A segment's queries: asked for while the segment before is merged (the
  // first one's before any copy), so that they do not wait behind the copies.
  // bf16 has them in the operand's layout; e4m3 converts them when the segment
  // begins; fp32 stages them in shared memory.
  constexpr int QV = KIND == kFp32 ? (ROWS * DP / 4 + THREADS - 1) / THREADS : 1;
  float4 qv[QV];
  float ks = 1.f;  // e4m3: the keys' scale
  auto load_queries = [&](const Cursor<TILE>& c) {
    const int rows = min(ROWS, p.group - c.rt * ROWS);
    const int kvh = c.kvg * hg + sub;
    const int64_t base = c.b * p.q_stride + (int64_t)(kvh * p.group + c.rt * ROWS) * p.dim;
    if constexpr (KIND == kFp32) {
#pragma unroll
      for (int i = 0; i < QV; ++i) {
        const int at = (tid + i * THREADS) * 4, r = at / DP, d = at % DP;
        qv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && d < p.dim)
          qv[i] = *reinterpret_cast<const float4*>((const float*)p.q + base + r * p.dim + d);
      }
    } else {
      const __nv_bfloat16* q = (const __nv_bfloat16*)p.q + base;
      if constexpr (KIND == kE4m3) {
        ks = p.k_scale ? p.k_scale[kvh] : 1.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = nt * 8 + g;
          if constexpr (KIND == kBf16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int d = mt * 16 + i * 8 + quad * 2;
              qf[mt][nt][i] = r < rows && d < p.dim
                                  ? *reinterpret_cast<const uint32_t*>(q + r * p.dim + d)
                                  : 0u;
            }
          } else {
            // elements 16 mt + 4 quad .. + 3: the order in which ldmatrix hands out bytes
            const int d = mt * 16 + quad * 4;
            const uint2 x = r < rows && d < p.dim
                                ? *reinterpret_cast<const uint2*>(q + r * p.dim + d)
                                : make_uint2(0u, 0u);
            qf[mt][nt][0] = x.x;
            qf[mt][nt][1] = x.y;
          }
        }
    }
  };
  load_queries(cc);

  // ---- copies
  Cursor<TILE> lc = cc;  // the tile whose page ids were last asked for
  auto locate = [&]() {
    RowAt r;
    const int pos = lc.s.lo + lc.j * tile + pos_in_tile + (lane & (WP - 1));
    r.off = -1;
    r.id = 0;
    if (pos < lc.s.T) {
      const int pg = p.div(pos);
      r.id = p.table[(int64_t)lc.b * p.width + pg];
      r.off = (int64_t)(pos - pg * p.page) * p.row_stride +
              (int64_t)(lc.kvg * hg + sub) * p.head_stride;
    }
    return r;
  };
  auto copy = [&](const RowAt& r, int stage) {
    int64_t at = -1;
    if (r.off >= 0) {
      if (r.id >= 0 && r.id < p.num_pages) at = (int64_t)r.id * p.page_stride + r.off;
      else atomicCAS(&g_status, 0, kBadPageSite);
    }
    const uint32_t base = ring + stage * S::STAGE;
#pragma unroll
    for (int i = 0; i < WP * CH / 32; ++i) {
      const int idx = lane + 32 * i, row = idx / CH, c = idx % CH;
      const int64_t src = __shfl_sync(~0u, at, row);
      if (c < chunks) {
        const uint32_t dst = base + row * S::ROWB + ((c ^ swizzle<CH>(row)) << 4);
        const int64_t off = src < 0 ? 0 : src * S::CB + c * 16;
        const uint32_t bytes = src < 0 ? 0u : 16u;
        cp_async16(dst, (const char*)p.k + off, bytes);
        cp_async16(dst + WP * S::ROWB, (const char*)p.v + off, bytes);
      }
    }
  };
  RowAt ahead;  // of the next tile to copy
  {
    RowAt first[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      first[s].off = -1;
      first[s].id = 0;
      if (s > 0 && lc.t < t1) lc.next(p, t1, blocks);
      if (lc.t < t1) first[s] = locate();
    }
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      copy(first[s], s);
      cp_async_commit();
    }
    ahead = first[STAGES - 1];
  }

  bool begin = true;  // a segment, or this share of one

  while (cc.t < t1) {
    cp_async_wait_group<STAGES - 2>();
    __syncwarp();
    if (lc.t < t1) {
      copy(ahead, stage == 0 ? STAGES - 1 : stage - 1);
      lc.next(p, t1, blocks);
      if (lc.t < t1) ahead = locate();
    }
    cp_async_commit();

    if (begin) {
      begin = false;
      whole = cc.j == 0;
#pragma unroll
      for (int i = 0; i < NSTAT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      sc[0] = p.scale_log2;
      if constexpr (KIND == kFp32) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) of[nb][r][e] = 0.f;
        // (the segment before ended with a barrier)
#pragma unroll
        for (int i = 0; i < QV; ++i) {
          const int at = (tid + i * THREADS) * 4;
          if (at < ROWS * DP) *reinterpret_cast<float4*>(s_q + at) = qv[i];
        }
        __syncthreads();
      } else {
        if constexpr (KIND == kE4m3) {
          // (a negative key scale turns the queries round, so that a score's scale is
          // positive; a zero one leaves it tiny; one that is no finite number makes
          // every score NaN)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float top = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                top = fmaxf(top, fabsf(__uint_as_float(qf[mt][nt][i] << 16)));
                top = fmaxf(top, fabsf(__uint_as_float(qf[mt][nt][i] & 0xFFFF0000u)));
              }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            // 2^e with top in [2^e, 2^(e+1)); its inverse stays a normal number
            const int e = min(max((int)((__float_as_uint(top) >> 23) & 255u) - 127, -120), 120);
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
            const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), ks);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t w = qf[mt][nt][i];
                const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * down,
                                                    __uint_as_float(w & 0xFFFF0000u) * down);
                qf[mt][nt][i] = *reinterpret_cast<const uint32_t*>(&h);
              }
            // lanes of row r know 2^e of head r; a score's columns are heads 2 quad + {0, 1}
            const float score = p.scale_log2 * fabsf(ks) * up + (ks - ks);
            const float mine_sc = score < 1e-37f ? 1e-37f : score;
            sc[2 * nt] = __shfl_sync(~0u, mine_sc, (2 * quad) * 4);
            sc[2 * nt + 1] = __shfl_sync(~0u, mine_sc, (2 * quad + 1) * 4);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      }
    }

    // ---- one tile: positions pos0 .. pos0 + WP - 1
    const int pos0 = cc.s.lo + cc.j * tile + pos_in_tile;
    const uint32_t kb = ring + stage * S::STAGE, vb = kb + WP * S::ROWB;
    if (pos0 < cc.s.T) {
      if constexpr (KIND != kFp32) {
        constexpr int SUB = WP / 16;
        float s[SUB][NT][4], s2[SUB][NT][4];  // two chains of products per score
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][nt][e] = s2[u][nt][e] = 0.f;
        const int r8 = lane & 7, mi = lane >> 3;
        const int row_k = r8 + (mi & 1) * 8;  // matrices: rows 0-7, 8-15, then the next chunk
        const int swz_k = swizzle<CH>(row_k);
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const uint32_t at = kb + (u * 16 + row_k) * S::ROWB;
          if constexpr (KIND == kBf16) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t a[4];
              ldmatrix4(at + (((2 * mt + (mi >> 1)) ^ swz_k) << 4), a);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816_bf16(mt & 1 ? s2[u][nt] : s[u][nt], a, qf[mt][nt][0], qf[mt][nt][1]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < MT; c += 2) {
              uint32_t x[4];
              ldmatrix4(at + (((c + (mi >> 1)) ^ swz_k) << 4), x);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t a[4];
                e4m3x4_to_half2(x[2 * h], a[0], a[2]);
                e4m3x4_to_half2(x[2 * h + 1], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816_f16(h ? s2[u][nt] : s[u][nt], a, qf[c + h][nt][0], qf[c + h][nt][1]);
              }
            }
          }
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][nt][e] += s2[u][nt][e];
        // scores: rows are positions u 16 + g (+ 8), columns this lane's two heads
        const int live = cc.s.T - pos0;
        if (live < WP) {
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (u * 16 + g + (e >> 1) * 8 >= live) s[u][nt][e] = -INFINITY;
        }
        float top[2 * NT];
        bool grew = false;
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
          float x = s[0][i >> 1][i & 1];
#pragma unroll
          for (int u = 0; u < SUB; ++u)
            x = fmaxf(x, fmaxf(s[u][i >> 1][i & 1], s[u][i >> 1][2 + (i & 1)]));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
          top[i] = fmaxf(m[i], x * sc[KIND == kE4m3 ? i : 0]);  // (the scale is positive)
          grew = grew || top[i] > m[i];
        }
        if (__any_sync(~0u, grew)) {
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) {
            const float f = ex2(m[i] - (top[i] == -INFINITY ? 0.f : top[i]));
            m[i] = top[i];
            l[i] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][i >> 1][i & 1] *= f;
              o[mt][i >> 1][2 + (i & 1)] *= f;
            }
          }
        }
        float base[2 * NT];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) base[i] = m[i] == -INFINITY ? 0.f : m[i];
        uint32_t hi[SUB][NT][2], lo[SUB][NT][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // (the product rounded as the maximum was, so that no difference is above
                // zero: from 2^23 on an exact one would be, by enough to leave fp16)
                const float x = __fadd_rn(
                    __fmul_rn(s[u][nt][2 * half + e], sc[KIND == kE4m3 ? 2 * nt + e : 0]),
                    -base[2 * nt + e]);
                w[e] = ex2(KIND == kE4m3 ? x + kShift : x);
                l[2 * nt + e] += w[e];
              }
              if constexpr (KIND == kBf16) {
                // (cut, not rounded, so that no second part is below zero; and none of a
                // weight is zero)
                const uint32_t h =
                    __byte_perm(__float_as_uint(w[0]), __float_as_uint(w[1]), 0x7632);
                const float low[2] = {
                    fmaxf(w[0] - __uint_as_float(h << 16), w[0] * 0x1p-20f),
                    fmaxf(w[1] - __uint_as_float(h & 0xFFFF0000u), w[1] * 0x1p-20f)};
                hi[u][nt][half] = movmatrix_trans(h);
                lo[u][nt][half] = movmatrix_trans(pack_bf16(low[0], low[1]));
              } else {
                const __half2 h = __floats2half2_rn(w[0], w[1]);
                hi[u][nt][half] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h));
              }
            }
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          if constexpr (KIND == kBf16) {
            // matrices: chunk 2 mt and 2 mt + 1 of rows 0-7, then of rows 8-15
            const int row_v = r8 + (mi >> 1) * 8;
            const int swz_v = swizzle<CH>(row_v);
            const uint32_t at = vb + (u * 16 + row_v) * S::ROWB;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t a[4];
              ldmatrix4_trans(at + (((2 * mt + (mi & 1)) ^ swz_v) << 4), a);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16816_bf16(o[mt][nt], a, hi[u][nt][0], hi[u][nt][1]);
                mma_16816_bf16(o[mt][nt], a, lo[u][nt][0], lo[u][nt][1]);
              }
            }
          } else {
            // rows 0-7 and 8-15 of chunk c, then of chunk c + 1; a 16-bit unit holds
            // elements 2g and 2g + 1 of a position: even ones are rows 0-7 of the
            // operand, odd ones rows 8-15
            const uint32_t at = vb + (u * 16 + row_k) * S::ROWB;
#pragma unroll
            for (int c = 0; c < MT; c += 2) {
              uint32_t x[4];
              ldmatrix4_trans(at + (((c + (mi >> 1)) ^ swz_k) << 4), x);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t a[4];
                e4m3x4_to_half2(__byte_perm(x[2 * h], 0, 0x3120), a[0], a[1]);
                e4m3x4_to_half2(__byte_perm(x[2 * h + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816_f16(o[c + h][nt], a, hi[u][nt][0], hi[u][nt][1]);
              }
            }
          }
        }
      } else {
        // eight positions at a time; lane: position lane % 8, every fourth chunk from lane / 8
        const int row = lane & 7, part = lane >> 3;
        float* ws = s_w + warp * 8 * ROWS;
#pragma unroll 1
        for (int u = 0; u < WP && pos0 + u < cc.s.T; u += 8) {
          const char* kp = smem + (kb - smem_u32(smem)) + (u + row) * S::ROWB;
          float s[ROWS];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) s[r] = 0.f;
#pragma unroll 4
          for (int c = part; c < chunks; c += 4) {
            const float4 x =
                *reinterpret_cast<const float4*>(kp + ((c ^ swizzle<CH>(row)) << 4));
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
              const float4 q = *reinterpret_cast<const float4*>(s_q + r * DP + c * 4);
              s[r] = fmaf(x.x, q.x, fmaf(x.y, q.y, fmaf(x.z, q.z, fmaf(x.w, q.w, s[r]))));
            }
          }
          // (one step of every row at a time: the rows' exchanges overlap)
          float top[ROWS];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) s[r] += __shfl_xor_sync(~0u, s[r], 8);
#pragma unroll
          for (int r = 0; r < ROWS; ++r) s[r] += __shfl_xor_sync(~0u, s[r], 16);
          const bool live = pos0 + u + row < cc.s.T;
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            s[r] = live ? s[r] * sc[0] : -INFINITY;
            top[r] = s[r];
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
              top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], o));
          bool grew = false;
#pragma unroll
          for (int r = 0; r < ROWS; ++r) grew = grew || top[r] > m[r];
          if (__any_sync(~0u, grew)) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
              top[r] = fmaxf(top[r], m[r]);
              const float f = ex2(m[r] - (top[r] == -INFINITY ? 0.f : top[r]));
              m[r] = top[r];
              l[r] *= f;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) of[nb][r][e] *= f;
            }
          }
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            s[r] = ex2(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
            l[r] += s[r];
            if (r / (ROWS / 4) == part) ws[row * ROWS + r] = s[r];
          }
          __syncwarp();
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            float w[ROWS];
#pragma unroll
            for (int r = 0; r < ROWS; r += 4) {
              const float4 x = *reinterpret_cast<const float4*>(ws + t * ROWS + r);
              w[r] = x.x; w[r + 1] = x.y; w[r + 2] = x.z; w[r + 3] = x.w;
            }
            const char* vp = smem + (vb - smem_u32(smem)) + (u + t) * S::ROWB;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              const int c = nb * 32 + lane;
              if (c < chunks) {
                const float4 x =
                    *reinterpret_cast<const float4*>(vp + ((c ^ swizzle<CH>(t)) << 4));
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                  of[nb][r][0] = fmaf(w[r], x.x, of[nb][r][0]);
                  of[nb][r][1] = fmaf(w[r], x.y, of[nb][r][1]);
                  of[nb][r][2] = fmaf(w[r], x.z, of[nb][r][2]);
                  of[nb][r][3] = fmaf(w[r], x.w, of[nb][r][3]);
                }
              }
            }
          }
          __syncwarp();
        }
      }
    }

    // ---- the segment ends here, or this share does
    const bool ends = cc.j == cc.s.n - 1;
    const Cursor<TILE> at = cc;
    cc.next(p, t1, blocks);
    const int used = stage;
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    if (ends || cc.t >= t1) {
      begin = true;
      if (cc.t < t1) load_queries(cc);
      const int rows = min(ROWS, p.group - at.rt * ROWS);
      // The warps' parts are merged in the tiles just used (the next copy goes
      // there after the barrier below).  Columns are XORed with 8 times the pair
      // of the row, so that the lanes of a store lie in different banks.
      float* const mine_o = reinterpret_cast<float*>(smem + (warp * STAGES + used) * S::STAGE);
      __syncwarp();
      if constexpr (KIND == kFp32) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          l[r] += __shfl_xor_sync(~0u, l[r], 1);
          l[r] += __shfl_xor_sync(~0u, l[r], 2);
          l[r] += __shfl_xor_sync(~0u, l[r], 4);
          if (lane == 0) s_ml[warp * ROWS + r] = make_float2(m[r], l[r]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int c = (nb * 32 + lane) * 4;
            if (c < DP)
              *reinterpret_cast<float4*>(mine_o + r * DP + (c ^ (((r >> 1) & 3) << 3))) =
                  make_float4(of[nb][r][0], of[nb][r][1], of[nb][r][2], of[nb][r][3]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
          l[i] += __shfl_xor_sync(~0u, l[i], 4);
          l[i] += __shfl_xor_sync(~0u, l[i], 8);
          l[i] += __shfl_xor_sync(~0u, l[i], 16);
          const int r = (i >> 1) * 8 + quad * 2 + (i & 1);
          if (g == 0) s_ml[warp * ROWS + r] = make_float2(m[i], l[i]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int d = mt * 16 + (KIND == kBf16 ? g + h * 8 : 2 * g + h);
              mine_o[r * DP + (d ^ (quad << 3))] = o[mt][i >> 1][2 * h + (i & 1)];
            }
        }
      }
      __syncthreads();
      const bool cut = !(whole && ends);
      const int slot = whole ? 2 * cta + 1 : 2 * cta;
      constexpr int C4 = DP / 4;
      for (int x = 0; x < hg; ++x) {  // the tile's heads
        const int kvh = at.kvg * hg + x;
        const float v_scale = KIND == kE4m3 && p.v_scale ? p.v_scale[kvh] : 1.f;
        const int64_t head0 = (int64_t)at.b * p.heads + kvh * p.group + at.rt * ROWS;
        const int64_t row0 = (int64_t)(slot * hg + x) * ROWS;
#pragma unroll
        for (int i = 0; i < (ROWS * C4 + THREADS - 1) / THREADS; ++i) {
          const int unit = tid + i * THREADS, rr = unit / C4, c = (unit % C4) * 4;
          if (rr >= rows || c >= p.dim) continue;
          float2 ml[NW];
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            ml[w] = make_float2(-INFINITY, 0.f);
            if (w < pw) ml[w] = s_ml[(x * pw + w) * ROWS + rr];
            M = fmaxf(M, ml[w].x);
          }
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if (w >= pw) continue;
            const float f = ex2(ml[w].x - (M == -INFINITY ? 0.f : M));
            const float4 y = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(
                    smem + ((x * pw + w) * STAGES + used) * S::STAGE) +
                rr * DP + (c ^ (((rr >> 1) & 3) << 3)));
            L = fmaf(f, ml[w].y, L);
            a.x = fmaf(f, y.x, a.x);
            a.y = fmaf(f, y.y, a.y);
            a.z = fmaf(f, y.z, a.z);
            a.w = fmaf(f, y.w, a.w);
          }
          if (cut) {
            *reinterpret_cast<float4*>(p.part_o + (row0 + rr) * DP + c) = a;
            if (c == 0) p.part_ml[row0 + rr] = make_float2(M, L);
          } else {
            const int64_t head = head0 + rr;
            const float inv = L == 0.f ? 0.f : v_scale / L;
            if constexpr (KIND == kFp32)
              *reinterpret_cast<float4*>((float*)p.out + head * p.dim + c) =
                  make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
            else
              *reinterpret_cast<uint2*>((__nv_bfloat16*)p.out + head * p.dim + c) =
                  make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
            if (c == 0 && p.lse)
              p.lse[head] = L == 0.f ? -INFINITY
                                     : (M + log2f(L) - (KIND == kE4m3 ? kShift : 0.f)) *
                                           0.6931471805599453f;
          }
        }
      }
      __syncthreads();
      if (chunks < CH) {
        // the rows' ends are zeros again (a zero query times anything but a number is none)
        for (int i = lane; i < 2 * WP * CH; i += 32) {
          const int row = i / CH, c = i % CH;
          if ((c ^ swizzle<CH>(row)) >= chunks)
            *reinterpret_cast<uint4*>(smem + (warp * STAGES + used) * S::STAGE + i * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      if (whole && !ends) {
        // the segment's last tile lies in CTA ((te + 1) ctas - 1) / total
        const long long te = at.t + (at.s.n - 1 - at.j);
        rec.cta = cta;
        rec.b = at.b;
        rec.hr = at.kvg * p.row_tiles + at.rt;
        rec.parts = (int)(((te + 1) * ctas - 1) / total) - cta + 1;
      }
      // (the CTA in which a segment begins writes its record)
      if (tid == 0 && p.rec && p.by_segment && whole)
        p.rec[(int64_t)at.b * hrs + at.kvg * p.row_tiles + at.rt] = rec;
    }
  }
  if (tid == 0 && p.rec && !p.by_segment) p.rec[cta] = rec;
  zero_idle<TILE, KIND>(p);
}

template <int DP, int KIND, int NT>
Kernel kernel_of() {
  using S = Shape<DP, KIND, NT>;
  // (fp32 keeps a segment's queries per CTA, for one head)
  void (*heads)(Params) = nullptr;
  if constexpr (KIND != kFp32) heads = decode_attn_sm103<DP, KIND, NT, true>;
  return {decode_attn_sm103<DP, KIND, NT, false>, heads, S::SMEM, S::NW, S::OCC, S::WP, S::ROWS,
          DP};
}

template <int KIND, int NT>
Kernel kernel_for(int dim) {
  return dim <= 64    ? kernel_of<64, KIND, NT>()
         : dim <= 96  ? kernel_of<96, KIND, NT>()
         : dim <= 128 ? kernel_of<128, KIND, NT>()
         : dim <= 192 ? kernel_of<192, KIND, NT>()
                      : kernel_of<256, KIND, NT>();
}

template <int KIND>
Kernel kernel_for(int dim, int nt) {
  return nt == 1 ? kernel_for<KIND, 1>(dim) : kernel_for<KIND, 2>(dim);
}

}  // namespace decode
}  // namespace mla
