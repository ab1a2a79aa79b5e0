// Interface between the decode attention's entry point and its kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "mla_internal.h"

namespace mla {
namespace decode {

// Element types of a call: q/out and cache bf16; q/out bf16 beside an e4m3
// cache; all fp32.
enum Kind { kBf16 = 0, kE4m3 = 1, kFp32 = 2 };

constexpr int kMaxCtas = 512;  // the join holds one weight per CTA

// A segment counts as this many tiles more than it has when the work is dealt
// out: its queries, its merge and its outputs take about as long as one tile.
constexpr int kSegmentCost = 1;

// Weights beside an e4m3 cache are scaled by 2^kShift.
constexpr float kShift = 15.f;

// Shape of one kernel: everything that follows from the padded head width DP,
// the element types and the row multiple NT.
template <int DP, int KIND, int NT>
struct Shape {
  static constexpr int CB = KIND == kBf16 ? 2 : KIND == kE4m3 ? 1 : 4;  // bytes of an element
  static constexpr int ROWB = DP * CB;                                  // bytes of a tile row
  static constexpr int CH = ROWB / 16;                                  // its 16-byte chunks
  // warps of a CTA, each with its own ring of tiles: four, more for the wide
  // heads whose CTA has an SM to itself and is short of warps, not of bytes on
  // their way (16 sequences of 4000 to 16000, 256 wide: fp32 511 us against
  // 622, bf16 with groups of 16 304 against 393)
  static constexpr bool WIDE = DP >= 192 && (KIND == kFp32 || NT == 2);
  static constexpr int NW = !WIDE ? 4 : DP == 192 ? 8 : 6;
  static constexpr int THREADS = NW * 32;
  // positions of a warp's tile: its K and V are 4 to 16 KB
  static constexpr int WP = KIND == kFp32                            ? (DP <= 64 ? 16 : 8)
                            : ROWB >= 192 && !(KIND == kE4m3 && NT == 2) ? 16
                                                                      : 32;
  static constexpr int ROWS = KIND == kFp32 ? 4 * NT : 8 * NT;  // query heads of a row tile
  static constexpr int STAGE = 2 * WP * ROWB;  // K, then V
  // Three CTAs per SM with rings of two tiles per warp where the registers of
  // 168 a thread suffice (up to 128 elements; beside 16-bit products one row
  // multiple): the third CTA's warps cover more latency than a third tile in
  // each ring would (bf16, 32 sequences of up to 32768: 327 us against 340;
  // e4m3, 64 sequences: 170 against 181; fp32, 16 sequences, groups of 8: 322
  // against 383).  Else two CTAs, or one with the whole shared memory.
  static constexpr int OCC = WIDE                                              ? 1
                             : DP <= 128 && (NT == 1 || KIND == kFp32)         ? 3
                             : 98304 / (NW * STAGE) >= 3                       ? 2
                                                                               : 1;
  static constexpr int FIT = 196608 / OCC / (NW * STAGE);
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int RING = NW * STAGES * STAGE;
  static constexpr int STATS = NW * ROWS * 8;
  // fp32: the row tile's queries, and each warp's weights
  static constexpr int QTILE = KIND == kFp32 ? ROWS * DP * 4 : 0;
  static constexpr int WEIGHTS = KIND == kFp32 ? NW * 8 * ROWS * 4 : 0;
  static constexpr int SMEM = RING + STATS + QTILE + WEIGHTS;
  static_assert(ROWS * DP * 4 <= STAGE, "a segment's sums are merged in the tile just used");
  static_assert(STAGES >= 2, "a warp's ring needs two tiles");
  // 228 KB of an SM, 1 KB of which each CTA costs besides (and a little static)
  static_assert(OCC * (SMEM + 1024 + 256) <= 228 * 1024, "OCC CTAs do not fit an SM");
};

// What is left for the join of a segment: the CTA whose share it begins in, as
// its last segment, and how many shares hold a part of it, that one and the
// next ones (0: nothing to join).
struct Record {
  int cta, parts, b, hr;
};

struct Params {
  const void* q;
  int64_t q_stride;
  const void *k, *v;
  int64_t page_stride, row_stride, head_stride;
  const float *k_scale, *v_scale;
  const int32_t* lens;
  const int32_t* table;
  void* out;
  float* lse;
  Record* rec;     // by segment or by CTA; NULL: no sequence is cut
  int by_segment;
  float2* part_ml; // [2 * ctas][hg][ROWS] running maximum (base 2) and sum
  float* part_o;   // [2 * ctas][hg][ROWS][DP] unnormalised
  int heads, group, row_tiles, dim, batch, page, width, num_pages, window;
  // a tile: `hg` neighbouring key/value heads, each taken by `pw` warps side by
  // side, `tile` positions in all; kv_groups such groups of heads
  int kv_groups, hg, pw, tile;
  PageDiv tile_div;
  PageDiv div;  // by `page`
  float scale_log2;  // softmax scale * log2(e)
};

struct Kernel {
  void (*fn)(Params);        // one key/value head to a tile
  void (*fn_heads)(Params);  // several (NULL: none)
  int smem, warps, occupancy, wp, rows, dp;
};

// The kernel for a head width and row multiple nt (1, 2).
Kernel kernel_bf16(int dp, int nt);
Kernel kernel_e4m3(int dp, int nt);
Kernel kernel_fp32(int dp, int nt);

int bf16_status(bool clear);
int e4m3_status(bool clear);
int fp32_status(bool clear);

}  // namespace decode
}  // namespace mla
