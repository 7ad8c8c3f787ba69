// Device code shared by the quantisers and the experts' products.
#pragma once

#include "experts_internal.h"

namespace eplb {

// A run of rows of one group that a workgroup works on.
struct Tile {
  int32_t g;                 // group; G and G + 1: rows of no group; -1: none
  int32_t row, rows;         // its rows
};

__host__ __device__ __forceinline__ int32_t clamp_row(int32_t v, int32_t R) { return v < 0 ? 0 : v > R ? R : v; }

// Rows lo .. hi - 1.
struct Span {
  int32_t lo, hi;
};

// Rows of group g; G: those behind the last group, G + 1: those before the first.
__host__ __device__ __forceinline__ Span group_span(const int32_t* offsets, int32_t g, int32_t G, int32_t R) {
  if (g < G) return {clamp_row(offsets[g], R), clamp_row(offsets[g + 1], R)};
  if (g == G) return {clamp_row(offsets[G], R), R};
  return {0, clamp_row(offsets[0], R)};
}

__host__ __device__ __forceinline__ int32_t tiles_of(Span s, int32_t size) {
  return s.hi > s.lo ? (int32_t)(((int64_t)s.hi - s.lo + size - 1) / size) : 0;
}

// Sum of two tile counts, at most 2^31 - 1: groups of decreasing offsets
// overlap, and together may have more tiles than that.
__host__ __device__ __forceinline__ int32_t add_tiles(int32_t a, int32_t b) {
  const uint32_t sum = (uint32_t)a + (uint32_t)b;
  return sum > 0x7FFFFFFFu ? 0x7FFFFFFF : (int32_t)sum;
}

// Tile `want` when every group's rows are cut into tiles of `size` rows, in
// the order of the groups; with `rest`, the rows behind the last group and
// those before the first one follow as groups G and G + 1.  Each wave looks
// at 64 groups at a time.
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int32_t G, int32_t R, int32_t size, int32_t want,
                                          bool rest) {
  const int lane = threadIdx.x & 63;
  const int32_t n = rest ? G + 2 : G;
  int32_t carry = 0;
  for (int32_t g0 = 0; g0 < n; g0 += 64) {
    const int32_t g = g0 + lane;
    const Span rows = g < n ? group_span(offsets, g, G, R) : Span{0, 0};
    const int32_t lo = rows.lo, hi = rows.hi, tiles = tiles_of(rows, size);
    int32_t incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t v = __shfl_up(incl, d);
      if (lane >= d) incl = add_tiles(incl, v);
    }
    const int32_t before = add_tiles(carry, incl - tiles);
    const u64 here = __ballot(want >= before && want - before < tiles);
    if (here != 0) {
      const int src = __ffsll((unsigned long long)here) - 1;
      Tile t;
      t.g = __shfl(g, src);
      t.row = __shfl(lo, src) + (want - __shfl(before, src)) * size;
      const int32_t left = __shfl(hi, src) - t.row;
      t.rows = left < size ? left : size;
      t.g = __builtin_amdgcn_readfirstlane(t.g);
      t.row = __builtin_amdgcn_readfirstlane(t.row);
      t.rows = __builtin_amdgcn_readfirstlane(t.rows);
      return t;
    }
    carry = __builtin_amdgcn_readfirstlane(__shfl(add_tiles(carry, incl), 63));
  }
  return Tile{-1, 0, 0};
}

// Number of tiles of all groups and, with `rest`, of the rows of no group.
__device__ __forceinline__ int32_t count_tiles(const int32_t* offsets, int32_t G, int32_t R, int32_t size, bool rest) {
  const int lane = threadIdx.x & 63;
  const int32_t n = rest ? G + 2 : G;
  int32_t mine = 0;
  for (int32_t g = lane; g < n; g += 64) mine = add_tiles(mine, tiles_of(group_span(offsets, g, G, R), size));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) mine = add_tiles(mine, __shfl_xor(mine, d));
  return __builtin_amdgcn_readfirstlane(mine);
}

// Workgroup `id` of `total` on a chip of 8 dies (workgroups go round the dies
// in turn): each die gets a run of neighbouring tiles, which share operands in
// its L2.
__device__ __forceinline__ int32_t die_order(int32_t id, int32_t total) {
  const int32_t per = total >> 3;
  return id < per * 8 ? (id & 7) * per + (id >> 3) : id;
}

// Tile `id` of rows x columns tiles taken in bands of four rows, column by
// column: the 32 tiles that a die works on at once are 4 x 8, which read 12
// different operand tiles (one row after the other: 18 of 2 x 16).  Bands of
// one, two, four and eight rows, 16384 x 8192 x 2048: 635, 600, 589 and 590 us;
// 16384 rows on 9, 4096 x 4096: 682, 686, 676, 672; weight gradient of 16384 rows
// on 9, 2048 x 4096: 364, 364, 350, 368.
__device__ __forceinline__ void band_order(int32_t id, int32_t rows, int32_t columns, int32_t& row, int32_t& column) {
  const int32_t band = id / (4 * columns), at = id - band * 4 * columns;
  const int32_t high = rows - band * 4 < 4 ? rows - band * 4 : 4;
  column = at / high;
  row = band * 4 + at - column * high;
}

// Scale of a block whose largest magnitude is amax (NaN: the block holds an
// infinity or a NaN) and the factor its elements are multiplied with.
__device__ __forceinline__ float block_scale(float amax, float& factor) {
  const float a = fmaxf(amax, kAmaxMin);
  factor = (1.0f / a) * kF8Max;
  return a * (1.0f / kF8Max);
}

// Four 32-bit values to 8 bits, nearest, ties to even.
__device__ __forceinline__ uint32_t pack_f8(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

}  // namespace eplb
