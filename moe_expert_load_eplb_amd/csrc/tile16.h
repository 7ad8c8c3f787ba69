// Tiles of a product of 16-bit operands with 32-bit sums: what the experts'
// products and the weight gradient have in common.
//
// out[o][i] = sum over k of O(o, k) * I(i, k).  A workgroup of WI x WO waves
// computes (WI IT 32) inner x (WO OT 32) outer values, a wave IT x OT tiles of
// 32 x 32.  The inner index is contiguous in the output; its operand is the
// matrix instruction's first, whose rows are taken in an order that leaves a
// lane with 16 consecutive inner values of one outer row for every tile.
//
// Operands go from memory to LDS without passing through registers, a block of
// 64 of k at a time, into one of two stages.  An operand lies in memory (and in
// LDS) one of two ways:
//   along    a row of the operand is contiguous in k: 128 bytes of a block for
//            each row, its eight 16-byte parts permuted by bits 1 to 3 of the row
//   across   k runs over rows of memory: 2 ROWS bytes for each k, the 16-byte
//            parts permuted by the lowest bits of k; fragments are read with
//            the transposing LDS read
// in both so that the lanes of a read reach all banks.
#pragma once

#include "experts_device.h"
#include "layer_internal.h"

namespace eplb {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

constexpr int kTileK = 64;                 // k of a block

__device__ __attribute__((aligned(16))) static const uint8_t g_zero_part[16] = {};   // read in place of what lies outside

// 16 bytes of every lane to 1 KiB of LDS from `to` (the same for the wave).  Written out, as the compiler lets the
// transposing reads wait for every such load in flight, whatever part of LDS it goes to: the waits for these loads are
// the tile's own.  No register is written but M0, which nothing else in these kernels uses (it cannot be named as
// clobbered) and which is read two instructions after it is set.
__device__ __forceinline__ void part_to_lds(const uint8_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from));
}

// The address of a byte of LDS as those loads take it.
__device__ __forceinline__ uint32_t lds_address(uint8_t* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)p);
}

// What the two operands hold.  kSplit: the first bfloat16, the second half precision, which is taken as two bfloat16
// values that sum to it exactly (11 significant bits are 8 and 3).
enum Mode { kBothBf16, kBothF16, kSplit };

__device__ __forceinline__ f32x16 mfma_bf16(i32x4 a, i32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight half-precision values as bfloat16: the nearest ones, and what they leave (0 of an infinity).
__device__ __forceinline__ void split_f16(i32x4 v, i32x4& high, i32x4& low) {
  const half8 x = __builtin_bit_cast(half8, v);
  bf16x8 h, l;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = (float)x[j];
    h[j] = (__bf16)f;
    const float left = f - (float)h[j];
    l[j] = (__bf16)(fabsf(f) <= 65504.0f ? left : 0.0f);
  }
  high = __builtin_bit_cast(i32x4, h);
  low = __builtin_bit_cast(i32x4, l);
}

// Four consecutive values of one output row; `left` of them are inside.
__device__ __forceinline__ void store_four(void* p, int32_t dtype, int64_t at, int left, bool vec, const float* v) {
  if (vec && left >= 4) {
    if (dtype == kF32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
      u16 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = dtype == kBf16 ? float_to_bf16(v[j]) : float_to_f16(v[j]);
      *reinterpret_cast<uint2*>(static_cast<u16*>(p) + at) =
          uint2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) store_float(p, dtype, at + j, v[j]);
}

// Eight consecutive values of one output row.
__device__ __forceinline__ void store_eight(void* p, int32_t dtype, int64_t at, int left, int64_t width,
                                            const float* v) {
  if (dtype != kF32 && left >= 8 && width % 8 == 0) {
    u16 h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = dtype == kBf16 ? float_to_bf16(v[j]) : float_to_f16(v[j]);
    *reinterpret_cast<uint4*>(static_cast<u16*>(p) + at) =
        uint4{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
              h[6] | (uint32_t)h[7] << 16};
    return;
  }
  store_four(p, dtype, at, left, width % 4 == 0, v);
  if (left > 4) store_four(p, dtype, at + 4, left - 4, width % 4 == 0, v + 4);
}

// Eight 4-bit values times a power of two as bfloat16.  Of the scale only the exponent counts; all bits of it set (255
// of a scale byte): NaN.
__device__ __forceinline__ i32x4 four_bit_values(int codes, float scale) {
  i32x4 v;
  v[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)codes, scale, 0));
  v[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)codes, scale, 1));
  v[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)codes, scale, 2));
  v[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)codes, scale, 3));
  return v;
}

// ---------------------------------------------------------------- operands
// ROWS rows of an operand loaded by W waves; T tiles of 32 rows to a wave;
// INNER: the rows of a wave in the inner operand's order.

// The row of the operand, counted from the wave's first, that index `a` (0 .. 31) of tile t stands for.
template <int T, bool INNER>
__device__ __forceinline__ int tile_row(int a, int t) {
  return INNER ? (a >> 2 & 1) * (16 * T) + 16 * t + (a >> 3) * 4 + (a & 3) : t * 32 + a;
}

template <int ROWS, int W, int T, bool INNER>
struct Along {
  static constexpr bool kThroughRegisters = false;
  static constexpr int kLoads = ROWS / 8 / W;
  static constexpr int kBytes = ROWS * 128;
  static_assert(ROWS % (8 * W) == 0 && W % 2 == 0, "whole loads, and the same part of every load's rows");

  const uint8_t* row[kLoads];              // where this lane's part of block 0 lies
  int part;                                // its first k within a block
  int at[4];                               // where the four steps' parts of this lane's row lie in LDS

  // start(r): where row r of the tile begins (any valid row for one that is not stored)
  template <typename Start>
  __device__ __forceinline__ void init(int lane, int wave, int first, Start start) {
    part = ((lane & 7) ^ ((wave * 8 + (lane >> 3)) >> 1 & 7)) * 8;
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
      row[p] = start((p * W + wave) * 8 + (lane >> 3)) + part * 2;
    }
    const int r = tile_row<T, INNER>(lane & 31, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) at[s] = (first + r) * 128 + (((s * 2 + (lane >> 5)) ^ (r >> 1 & 7)) << 4);
  }
  // load p of block blk, of K elements in all, to LDS
  __device__ __forceinline__ void load(int p, int blk, int K, int wave, uint32_t lds) const {
    const bool in = blk * kTileK + part < K;
    part_to_lds(in ? row[p] + (int64_t)blk * 128 : g_zero_part, lds + (p * W + wave) * 1024);
  }
  __device__ __forceinline__ i32x4 fragment(const uint8_t* lds, int t, int s) const {
    return *reinterpret_cast<const i32x4*>(lds + at[s] + (INNER ? 16 : 32) * 128 * t);
  }
};

// Memory rows are k; rows of the operand are columns there.
template <int ROWS, int W, int T, bool INNER>
struct Across {
  static constexpr bool kThroughRegisters = false;
  static constexpr int kParts = ROWS / 8;            // 16-byte parts of a memory row
  static constexpr int kEach = 64 / kParts;          // memory rows of one load of a wave
  static constexpr int kLoads = kTileK / kEach / W;
  static constexpr int kBytes = ROWS * 128;
  static_assert(kParts <= 64 && kParts >= 16 && kTileK % (kEach * W) == 0, "whole loads");
  static_assert(kEach * W % 4 == 0, "k & 3 is the same for every load of a lane");

  const uint8_t* base;                     // this lane's column of memory row 0 (one it has, if its own is outside)
  int64_t ld;                              // bytes between memory rows
  int first;                               // k within a block of this lane's first load; the next ones are kEach W on
  bool inside;
  int at[T];

  // How the parts of memory row k are permuted: four consecutive k reach different banks.  The inner order reads parts
  // {0, 1} and {2 T, 2 T + 1} from a tile's start at once, the outer order {0 .. 3}.
  static __device__ __forceinline__ int key(int k) {
    return !INNER ? (k & 3) << 2 : T == 4 ? (k & 3) << 1 : (k & 1) << 1 | (k & 2) << 2;
  }
  __device__ __forceinline__ uint32_t k_of(int p, int blk) const {
    return (uint32_t)blk * kTileK + first + p * (kEach * W);
  }

  // `columns` of the tile's columns are inside
  __device__ __forceinline__ void init(int lane, int wave, int first_row, const uint8_t* start, int64_t ld_bytes,
                                       int columns) {
    first = wave * kEach + lane / kParts;
    const int part = lane % kParts ^ key(first);
    inside = part * 8 < columns;
    base = start + (inside ? part * 16 : 0);
    ld = ld_bytes;
    const int kr = lane >> 2 & 3, half = lane >> 5, c = (lane >> 4 & 1) * 4 + (lane & 3);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int r = first_row + tile_row<T, INNER>(c * 4, t);      // four consecutive columns
      at[t] = (half * 8 + kr) * (ROWS * 2) + (((r >> 3) ^ key(kr)) << 4) + (r >> 2 & 1) * 8;
    }
  }
  // load p of a block: memory row `row`, -1: zeros
  __device__ __forceinline__ void load_row(int p, int row, int wave, uint32_t lds) const {
    part_to_lds(inside && row >= 0 ? base + row * ld : g_zero_part, lds + (p * W + wave) * 1024);
  }
  __device__ __forceinline__ void load(int p, int blk, int K, int wave, uint32_t lds) const {
    const uint32_t k = k_of(p, blk);
    load_row(p, k < (uint32_t)K ? (int)k : -1, wave, lds);
  }
  __device__ __forceinline__ i32x4 fragment(const uint8_t* lds, int t, int s) const {
    typedef __attribute__((address_space(3))) s16x4* Ptr;
    const uint8_t* from = lds + at[t] + s * 16 * (ROWS * 2);
    union {
      s16x4 h[2];
      i32x4 v;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)from);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(from + 4 * (ROWS * 2)));
    return u.v;
  }
};

// An operand of 4-bit values along k, its blocks of 32 scaled by powers of two: from memory to registers a block ahead,
// and to LDS as bfloat16 (exactly), in the layout of Along.
template <int ROWS, int W, int T, bool INNER>
struct FourBit {
  static constexpr bool kThroughRegisters = true;
  static constexpr int kLoads = ROWS / 32 / W;       // of 32 rows and both halves of a block
  static constexpr int kBytes = ROWS * 128;
  static_assert(ROWS % (32 * W) == 0, "whole loads");

  const uint8_t* codes;                    // this lane's part of block 0 of its first row
  const uint8_t* scales;
  int32_t ld_codes, ld_scales;             // bytes from one load's row to the next one's, which is 32 W rows on
  int half, own, last;                     // half of a block, first row, last row inside
  i32x4 raw[kLoads];
  uint32_t scale[kLoads];
  int at[4];

  __device__ __forceinline__ void init(int lane, int wave, int first, const uint8_t* q, const uint8_t* s, int C, int n) {
    half = lane & 1;
    own = wave * 32 + (lane >> 1);
    last = n - 1;
    codes = q + half * 16;
    scales = s + half;
    ld_codes = C / 2;
    ld_scales = C / kScaleGroup;
    const int r = tile_row<T, INNER>(lane & 31, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = (first + r) * 128 + (((j * 2 + (lane >> 5)) ^ (r >> 1 & 7)) << 4);
  }
  // block blk of K elements in all; past the end of a row: zeros
  __device__ __forceinline__ void fetch(int blk, int K) {
    const bool in = blk * kTileK + half * kScaleGroup < K;
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
      const int64_t r = min(own + p * 32 * W, last);
      raw[p] = i32x4{0, 0, 0, 0};
      scale[p] = 127;
      if (in) {
        raw[p] = *reinterpret_cast<const i32x4*>(codes + r * ld_codes + blk * 32);
        scale[p] = scales[r * ld_scales + blk * 2];
      }
    }
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int p = 0; p < kLoads; ++p) asm volatile("" : "+v"(raw[p]), "+v"(scale[p]));
  }
  // load p of the block that was fetched last
  __device__ __forceinline__ void load(int p, uint8_t* lds) const {
    const int r = own + p * 32 * W;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<i32x4*>(lds + r * 128 + (((half * 4 + j) ^ (r >> 1 & 7)) << 4)) =
          four_bit_values(raw[p][j], __uint_as_float(scale[p] << 23));
  }
  __device__ __forceinline__ i32x4 fragment(const uint8_t* lds, int t, int s) const {
    return *reinterpret_cast<const i32x4*>(lds + at[s] + (INNER ? 16 : 32) * 128 * t);
  }
};

// ---------------------------------------------------------------- a tile
template <Mode MODE, int WI, int WO, int IT, int OT, typename Inner, typename Outer>
struct Tile16 {
  typedef Inner Inner_;
  typedef Outer Outer_;
  static constexpr int kWaves = WI * WO, kThreads = kWaves * 64;
  static constexpr int kInner = WI * IT * 32, kOuter = WO * OT * 32;
  static constexpr int kStageBytes = Inner::kBytes + Outer::kBytes;
  static constexpr int kLdsBytes = 2 * kStageBytes;

  static __device__ __forceinline__ int inner_first(int wave) { return wave % WI * (IT * 32); }
  static __device__ __forceinline__ int outer_first(int wave) { return wave / WI * (OT * 32); }

  // loads.issue(i, blk, stage): one of the loads.kLoads loads of block blk to LDS, in order; loads.fetch(blk): what they
  // need in registers; loads.settle(): waits for that
  template <typename Loads>
  static __device__ __forceinline__ void run(const Inner& in, const Outer& out, Loads& loads, int K, uint8_t* lds,
                                             f32x16 (&acc)[OT][IT]) {
    constexpr int kTiles = IT * OT, kReads = IT + OT;
    const int blocks = (K - 1) / kTileK + 1;
    i32x4 fi[2][IT], fo[2][OT];
#pragma unroll
    for (int o = 0; o < OT; ++o)
#pragma unroll
      for (int t = 0; t < IT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[o][t][i] = 0.0f;
    // fragment u of step s of a stage
    auto read = [&](const uint8_t* stage, int s, int u) {
      if (u < IT) fi[s & 1][u] = in.fragment(stage, u, s);
      else fo[s & 1][u - IT] = out.fragment(stage + Inner::kBytes, u - IT, s);
    };
    // the products of step s, the next step's fragments read under them (and after the last step of a block, which leaves
    // its stage free, the loads of a later block)
    auto step = [&](int s, const uint8_t* stage, int blk, uint32_t slot) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        const int o = j / IT, t = j % IT;
        multiply(fi[s & 1][t], fo[s & 1][o], acc[o][t]);
#pragma unroll
        for (int u = j * kReads / kTiles; u < (j + 1) * kReads / kTiles; ++u) read(stage, (s + 1) & 3, u);
        if (s == 3) {
#pragma unroll
          for (int i = j * Loads::kLoads / kTiles; i < (j + 1) * Loads::kLoads / kTiles; ++i) loads.issue(i, blk, slot);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto wait = [&] {
      // this wave's loads have arrived and its reads are done; then those of all waves
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      loads.settle();
    };
    loads.fetch(0);
    loads.settle();
#pragma unroll
    for (int i = 0; i < Loads::kLoads; ++i) loads.issue(i, 0, 0);
    loads.fetch(1);
    wait();
#pragma unroll
    for (int i = 0; i < Loads::kLoads; ++i) loads.issue(i, 1, kStageBytes);
    loads.fetch(2);
#pragma unroll
    for (int u = 0; u < kReads; ++u) read(lds, 0, u);
    for (int b = 0; b < blocks; ++b) {
      const uint32_t slot = (b & 1) * kStageBytes;
      const uint8_t* stage = lds + slot;
      step(0, stage, 0, 0);
      step(1, stage, 0, 0);
      step(2, stage, 0, 0);
      wait();                              // the next block is there, and all are done with this one
      step(3, lds + (kStageBytes - slot), b + 2, slot);
      loads.fetch(b + 3);
    }
    wait();                                // none may land in LDS that is no longer this workgroup's
  }

  static __device__ __forceinline__ void multiply(i32x4 a, i32x4 b, f32x16& acc) {
    if constexpr (MODE == kBothBf16) {
      acc = mfma_bf16(a, b, acc);
    } else if constexpr (MODE == kBothF16) {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), acc, 0, 0,
                                                   0);
    } else {
      i32x4 high, low;
      split_f16(b, high, low);
      acc = mfma_bf16(a, high, acc);
      acc = mfma_bf16(a, low, acc);
    }
  }

  // Stores the wave's values: row(r) is outer row r's first element in the
  // output or -1, some(r) whether it has values (else zeros), `left` the inner
  // values from the tile's start on.
  template <typename Row, typename Some>
  static __device__ __forceinline__ void store(const f32x16 (&acc)[OT][IT], void* out, int32_t dtype, int64_t width,
                                               int64_t left, Row row, Some some) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = inner_first(wave) + (lane >> 5) * (16 * IT), wo = outer_first(wave);
#pragma unroll
    for (int o = 0; o < OT; ++o) {
      const int r = wo + o * 32 + (lane & 31);
      const int64_t at = row(r);
      if (at < 0) continue;
      const bool in = some(r);
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = in ? acc[o][t][i] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          const int64_t n = wi + 16 * t + i;
          if (n < left) store_eight(out, dtype, at + n, left - n < 8 ? (int)(left - n) : 8, width, v + i);
        }
      }
    }
  }
};

// ---------------------------------------------------------------- a product
__device__ __forceinline__ int32_t source_of(const int32_t* rows, FastDiv topk, int64_t X, int32_t r) {
  int32_t from = r;
  if (rows != nullptr) {
    from = rows[r];
    from = from < 0 ? -1 : (int32_t)fastdiv_apply((uint32_t)from, topk);
  }
  return from < X ? from : -1;
}

enum Weights { kWeights, kWeightsTransposed, kWeights4 };

template <int WI, int WO, int IT, Weights FORM>
struct InnerOperand {
  typedef Along<WI * IT * 32, WI * WO, IT, true> Type;
};
template <int WI, int WO, int IT>
struct InnerOperand<WI, WO, IT, kWeightsTransposed> {
  typedef Across<WI * IT * 32, WI * WO, IT, true> Type;
};
template <int WI, int WO, int IT>
struct InnerOperand<WI, WO, IT, kWeights4> {
  typedef FourBit<WI * IT * 32, WI * WO, IT, true> Type;
};

template <Mode MODE, int WI, int WO, int IT, int OT, Weights FORM>
using LinearTile = Tile16<MODE, WI, WO, IT, OT, typename InnerOperand<WI, WO, IT, FORM>::Type,
                          Along<WO * OT * 32, WI * WO, OT, false>>;

// The loads of a product's tile.
template <typename Inner, typename Outer>
struct LinearLoads {
  static constexpr int kLoads = Inner::kLoads + Outer::kLoads;
  Inner& in;
  const Outer& out;
  uint8_t* lds;
  uint32_t at;
  int K, wave;

  // what goes through registers first: it was waited for, and nothing that was issued since is waited for with it
  __device__ __forceinline__ void issue(int i, int blk, uint32_t slot) const {
    if (i < Inner::kLoads) {
      if constexpr (Inner::kThroughRegisters) in.load(i, lds + slot);
      else in.load(i, blk, K, wave, at + slot);
    } else {
      out.load(i - Inner::kLoads, blk, K, wave, at + slot + Inner::kBytes);
    }
  }
  __device__ __forceinline__ void fetch(int blk) {
    if constexpr (Inner::kThroughRegisters) in.fetch(blk, K);
  }
  __device__ __forceinline__ void settle() {
    if constexpr (Inner::kThroughRegisters) in.settle();
  }
};

template <Mode MODE, int WI, int WO, int IT, int OT, Weights FORM>
__global__ __launch_bounds__(WI* WO * 64) void linear_tile_kernel(Linear16Args a, int32_t columns) {
  typedef LinearTile<MODE, WI, WO, IT, OT, FORM> Tile_;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int32_t src[Tile_::kOuter];
  const int32_t row_tiles = count_tiles(a.offsets, a.G, a.R, Tile_::kOuter, true);
  const int64_t tiles = min((int64_t)row_tiles * columns, (int64_t)gridDim.x);    // less where offsets decrease
  if (blockIdx.x >= tiles) return;
  int32_t row, column;
  band_order(die_order(blockIdx.x, (int32_t)tiles), row_tiles, columns, row, column);
  const Tile t = find_tile(a.offsets, a.G, a.R, Tile_::kOuter, row, true);
  if (t.g < 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = FORM == kWeightsTransposed ? a.C : a.N, K = FORM == kWeightsTransposed ? a.N : a.C;
  const int i0 = column * Tile_::kInner;
  for (int r = threadIdx.x; r < Tile_::kOuter; r += Tile_::kThreads)
    src[r] = r < t.rows && t.g < a.G ? source_of(a.rows, a.fd_topk, a.X, t.row + r) : -1;
  __syncthreads();
  f32x16 acc[OT][IT];
  if (t.g < a.G && a.X > 0) {
    typename Tile_::Inner_ in;
    typename Tile_::Outer_ out;
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + (int64_t)t.g * a.N * a.C * 2;
    // a row that has no source reads one that is there, and is not stored
    out.init(lane, wave, Tile_::outer_first(wave),
             [&](int r) { return static_cast<const uint8_t*>(a.x) + max(src[r], 0) * a.ld * 2; });
    if constexpr (FORM == kWeightsTransposed) {
      in.init(lane, wave, Tile_::inner_first(wave), w + i0 * 2, (int64_t)a.C * 2, width - i0);
    } else if constexpr (FORM == kWeights) {
      in.init(lane, wave, Tile_::inner_first(wave),
              [&](int r) { return w + (int64_t)min(i0 + r, width - 1) * K * 2; });
    } else {
      const int64_t n = (int64_t)t.g * a.N + i0;
      in.init(lane, wave, Tile_::inner_first(wave), a.q + n * (K / 2), a.scale + n * (K / kScaleGroup), K, width - i0);
    }
    LinearLoads<typename Tile_::Inner_, typename Tile_::Outer_> loads{in, out, lds, lds_address(lds), K, wave};
    Tile_::run(in, out, loads, K, lds, acc);
  }
  Tile_::store(acc, a.y, a.y_dtype, width, width - i0,
               [&](int r) -> int64_t { return r < t.rows ? (int64_t)(t.row + r) * width + i0 : -1; },
               [&](int r) { return src[r] >= 0; });
}

}  // namespace eplb
