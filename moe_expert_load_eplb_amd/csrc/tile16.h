// Tiles of a product of 16-bit operands with 32-bit sums: what the experts'
// products and the weight gradient have in common.
//
// out[o][i] = sum over k of O(o, k) * I(i, k).  A workgroup of WI x WO waves
// computes (WI IT 32) inner x (WO OT 32) outer values, a wave IT 32 x OT 32 of
// them, as tiles of the matrix instruction (16 x 16).  The inner index is
// contiguous in the output; its operand is the matrix instruction's first, so
// that a lane ends up with runs of four inner values of one outer row.
//
// Operands go from memory to LDS without passing through registers, a block of
// 64 of k at a time, into one of two stages.  An operand lies in memory (and in
// LDS) one of two ways:
//   along    a row of the operand is contiguous in k: 128 bytes of a block for
//            each row, its eight 16-byte parts permuted by bits 1 to 3 of the row
//   across   k runs over rows of memory: 2 ROWS bytes for each k, the 16-byte
//            parts permuted by bits of k; fragments are read with the transposing
//            LDS read
// in both so that the lanes of a read reach all banks.
//
// The loads take a buffer descriptor and 32-bit offsets: what is past the
// descriptor's end, or marked by the offset's highest bit, arrives as zeros.
#pragma once

#include "experts_device.h"
#include "layer_internal.h"

namespace eplb {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

constexpr int kTileK = 64;                 // k of a block
constexpr uint32_t kOutside = 0x80000000u; // an offset that no descriptor reaches

__device__ __attribute__((aligned(16))) static const uint8_t g_zero_part[16] = {};

// A descriptor of `bytes` bytes (2^31 at most) from p on.  The same for the wave.
__device__ __forceinline__ i32x4 describe(const void* p, uint64_t bytes) {
  const uint64_t at = (uint64_t)p;
  i32x4 d;
  d[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)at);
  d[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
  d[2] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(bytes < kOutside ? bytes : kOutside));
  d[3] = 0x00020000;                       // raw, 32-bit elements
  return d;
}

// The same for the compiler's own loads.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(i32x4 d) {
  const uint64_t at = (uint64_t)(uint32_t)d[0] | (uint64_t)(uint32_t)d[1] << 32;
  return __builtin_amdgcn_make_buffer_rsrc((void*)at, 0, d[2], d[3]);
}

// 16 bytes of every lane to 1 KiB of LDS from `to` (the same for the wave).  Written out, as the compiler lets the
// transposing reads wait for every such load in flight, whatever part of LDS it goes to: the waits for these loads are
// the tile's own.  No register is written but M0, which nothing else in these kernels uses (it cannot be named as
// clobbered) and which is read two instructions after it is set.
__device__ __forceinline__ void part_to_lds(i32x4 from, uint32_t offset, uint32_t shift, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(offset), "s"(from),
               "s"(shift));
}

// The same from an address of each lane.
__device__ __forceinline__ void part_to_lds(const uint8_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from));
}

// The address of a byte of LDS as those loads take it.
__device__ __forceinline__ uint32_t lds_address(uint8_t* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)p);
}

// What the two operands hold.  kScaled: the first 4-bit values without their scales, as half precision, the second half
// precision; what an instruction adds up, 32 of k, is multiplied by the scales then.  (A value times its scale is a
// bfloat16 number, but not one of half precision; with the rows as two bfloat16 numbers each, 16384 rows on 9, 4096 x
// 4096, took 1210 us, so 778.)
enum Mode { kBothBf16, kBothF16, kScaled };

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

// Eight 4-bit values as half precision.
__device__ __forceinline__ i32x4 four_bit_halves(int codes) {
  i32x4 v;
  v[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)codes, 1.0f, 0));
  v[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)codes, 1.0f, 1));
  v[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)codes, 1.0f, 2));
  v[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4((uint32_t)codes, 1.0f, 3));
  return v;
}

// What a scale byte stands for, 2^(byte - 127) or NaN (255), as a float whose lower half is zeros.
__device__ __forceinline__ uint32_t scale_bits(uint32_t byte) {
  return byte << 23 | (byte == 0 || byte == 255 ? 0x00400000u : 0);
}

// ---------------------------------------------------------------- the matrix instruction
constexpr int kM = 16;                     // its rows and columns; a lane has four rows' sums, from 4 (lane / kM) on
constexpr int kInstrK = 32;                // its k: lane / kM takes eight of them

__device__ __forceinline__ f32x4 multiply_bf16(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 multiply_f16(i32x4 a, i32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------- operands
// ROWS rows of an operand loaded by W waves.

// How the parts of row r are permuted where k lies along: two rows make one turn of the banks.
__device__ __forceinline__ int along_key(int r) { return r >> 1 & 7; }

// Where the fragments of a wave lie, in a stage of rows along k.
struct AlongFragments {
  static constexpr int kSteps = kTileK / kInstrK;
  int at[kSteps];
  __device__ __forceinline__ void init(int lane, int first_row) {
    const int r = first_row + lane % kM;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) at[s] = r * 128 + (((s * (kInstrK / 8) + lane / kM) ^ along_key(r)) << 4);
  }
  __device__ __forceinline__ i32x4 read(const uint8_t* lds, int t, int s) const {
    return *reinterpret_cast<const i32x4*>(lds + at[s] + kM * 128 * t);
  }
};

// Rows that lie one after the other.
template <int ROWS, int W>
struct Along {
  static constexpr int kLoads = ROWS / 8 / W;
  static constexpr int kBytes = ROWS * 128;
  static_assert(ROWS % (8 * W) == 0 && W % 2 == 0, "whole loads, and the same part of every load's rows");

  i32x4 from;
  uint32_t offset, step;                   // of this lane's part, from one load's rows to the next one's
  int part;                                // its first k within a block

  // `rows` rows of `ld` bytes from `start` on; those past them read as zeros
  __device__ __forceinline__ void init(int lane, int wave, const uint8_t* start, uint32_t ld, int rows) {
    from = describe(start, (uint64_t)min(rows, ROWS) * ld);
    part = ((lane & 7) ^ along_key(wave * 8 + (lane >> 3))) * 8;
    offset = (wave * 8 + (lane >> 3)) * ld + part * 2;
    step = W * 8 * ld;
  }
  // load p of block blk, of K elements in all, to LDS
  __device__ __forceinline__ void load(int p, int blk, int K, int wave, uint32_t lds) const {
    part_to_lds(from, part < K - blk * kTileK ? offset : kOutside, p * step + blk * 128, lds + (p * W + wave) * 1024);
  }
};

// Rows that lie anywhere.  FAR: they span 2^31 bytes or more.
template <int ROWS, int W, bool FAR>
struct Gathered {
  static constexpr int kLoads = ROWS / 8 / W;
  static constexpr int kBytes = ROWS * 128;
  static_assert(ROWS % (8 * W) == 0 && W % 2 == 0, "whole loads, and the same part of every load's rows");

  i32x4 from;
  uint32_t offset[FAR ? 1 : kLoads];
  const uint8_t* row[FAR ? kLoads : 1];
  int part;

  // row(r): the row of memory that row r of the tile is, or -1 (what is read for it is not used)
  template <typename Row>
  __device__ __forceinline__ void init(int lane, int wave, const uint8_t* start, int64_t ld, int64_t rows, Row of) {
    part = ((lane & 7) ^ along_key(wave * 8 + (lane >> 3))) * 8;
    if (!FAR) from = describe(start, rows * ld);
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
      const int32_t r = of((p * W + wave) * 8 + (lane >> 3));
      if (FAR) row[p] = start + max(r, 0) * ld + part * 2;
      else offset[p] = r < 0 ? kOutside : (uint32_t)r * (uint32_t)ld + part * 2;
    }
  }
  __device__ __forceinline__ void load(int p, int blk, int K, int wave, uint32_t lds) const {
    const bool in = part < K - blk * kTileK;
    if (FAR) part_to_lds(in ? row[p] + (int64_t)blk * 128 : g_zero_part, lds + (p * W + wave) * 1024);
    else part_to_lds(from, offset[p] | (in ? 0 : kOutside), blk * 128, lds + (p * W + wave) * 1024);
  }
};

// Memory rows are k; rows of the operand are columns there.
template <int ROWS, int W>
struct Across {
  static constexpr int kParts = ROWS / 8;            // 16-byte parts of a memory row
  static constexpr int kEach = 64 / kParts;          // memory rows of one load of a wave
  static constexpr int kLoads = kTileK / kEach / W;
  static constexpr int kBytes = ROWS * 128;
  static_assert(kParts <= 64 && kParts >= 16 && kTileK % (kEach * W) == 0, "whole loads");
  // a lane's loads are kEach W memory rows apart: permutations that they have
  static constexpr int kKinds = kEach * W % 16 == 0 ? 1 : 2;
  static_assert(kEach * W % 8 == 0, "not more of them");

  const uint8_t* base;                     // column 0 of the tile in memory row 0
  uint32_t ld;                             // bytes between memory rows
  uint32_t offset[kKinds];                 // of this lane's part of load p, from the first memory row of load 0's on

  // How the parts of memory row k are permuted.  What 32 lanes read at once is twice four consecutive k, eight apart, of
  // 32 bytes.
  static __device__ __forceinline__ int key(int k) { return (k & 3) << 1 | (k & 8); }

  // `columns` of the tile's columns are inside
  __device__ __forceinline__ void init(int lane, int wave, const uint8_t* start, int64_t ld_bytes, int columns) {
    base = start;
    ld = (uint32_t)ld_bytes;
    const int k = wave * kEach + lane / kParts;
#pragma unroll
    for (int i = 0; i < kKinds; ++i) {
      const uint32_t c = column(lane, wave, i, columns);
      offset[i] = c == kOutside ? c : k * ld + c;
    }
  }
  // where in a memory row this lane's part of load p lies
  static __device__ __forceinline__ uint32_t column(int lane, int wave, int p, int columns) {
    const int part = lane % kParts ^ key((p * W + wave) * kEach + lane / kParts);
    return part * 8 < columns ? part * 16 : kOutside;
  }
  // of block blk, with memory rows up to K
  __device__ __forceinline__ i32x4 describe_block(int blk, int K) const {
    const uint32_t k = (uint32_t)blk * kTileK;
    return describe(base + (uint64_t)k * ld, k < (uint32_t)K ? (uint64_t)((uint32_t)K - k) * ld : 0);
  }
  __device__ __forceinline__ void load(int p, const i32x4& from, int wave, uint32_t lds) const {
    part_to_lds(from, offset[p % kKinds], p * (kEach * W) * ld, lds + (p * W + wave) * 1024);
  }
};

template <int ROWS>
struct AcrossFragments {
  static constexpr int kKinds = 8;         // tiles that the permutation tells apart
  int at[kKinds];
  __device__ __forceinline__ void init(int lane, int first_row) {
    const int k = lane / kM * 8 + (lane >> 2 & 3), c = (lane & 3) * 4;   // four consecutive columns
#pragma unroll
    for (int t = 0; t < kKinds; ++t) {
      const int r = first_row + t * kM + c;
      at[t] = k * (ROWS * 2) + (((r >> 3) ^ Across<ROWS, 16>::key(k)) << 4) + (r >> 2 & 1) * 8;
    }
  }
  __device__ __forceinline__ i32x4 read(const uint8_t* lds, int t, int s) const {
    typedef __attribute__((address_space(3))) s16x4* Ptr;
    const uint8_t* from = lds + at[t] + s * kInstrK * (ROWS * 2);
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
// and to LDS as bfloat16 (exactly), in the layout of rows along k.  SCALED: without the scales, as half precision; the
// scales follow the block, in bfloat16, those of all rows' first half and then those of the second.
template <int ROWS, int W, bool SCALED>
struct FourBit {
  static constexpr int kActive = ROWS / 32 < W ? ROWS / 32 : W;    // waves that load
  static constexpr int kLoads = ROWS / 32 / kActive; // of 32 rows and both halves of a block
  static constexpr int kBytes = ROWS * 128;
  static_assert(ROWS % (32 * kActive) == 0, "whole loads");

  const uint8_t* codes;                    // this lane's part of block 0 of its first row
  const uint8_t* scales;
  int32_t ld_codes, ld_scales;
  int half, own, last;                     // half of a block, first row, last row inside
  i32x4 raw[kLoads];
  uint32_t scale[kLoads];

  __device__ __forceinline__ void init(int lane, int wave, const uint8_t* q, const uint8_t* s, int C, int n) {
    half = lane & 1;
    own = wave * 32 + (lane >> 1);
    last = n - 1;
    codes = q + half * 16;
    scales = s + half;
    ld_codes = C / 2;
    ld_scales = C / kScaleGroup;
  }
  // block blk of K elements in all; past the end of a row: zeros
  __device__ __forceinline__ void fetch(int blk, int K) {
    const bool in = blk * kTileK + half * kScaleGroup < K;
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
      const int64_t r = min(own + p * 32 * kActive, last);
      raw[p] = i32x4{0, 0, 0, 0};
      scale[p] = 127;
      if (in && own < ROWS) {
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
  __device__ __forceinline__ void load(int p, uint8_t* lds, uint8_t* lds_scales) const {
    const int r = own + p * 32 * kActive;
    if (kActive < W && own >= ROWS) return;          // the same for a wave
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<i32x4*>(lds + r * 128 + (((half * 4 + j) ^ along_key(r)) << 4)) =
          SCALED ? four_bit_halves(raw[p][j]) : four_bit_values(raw[p][j], __uint_as_float(scale[p] << 23));
    if (SCALED) reinterpret_cast<u16*>(lds_scales)[half * ROWS + r] = (u16)(scale_bits(scale[p]) >> 16);
  }
};

// ---------------------------------------------------------------- a tile
template <Mode MODE, int WI, int WO, int IT, int OT, typename InnerFragments, typename OuterFragments>
struct Tile16 {
  typedef f32x4 Sum;
  static constexpr int kWaves = WI * WO, kThreads = kWaves * 64;
  static constexpr int kInner = WI * IT * 32, kOuter = WO * OT * 32;
  static constexpr int kInnerBytes = kInner * 128, kScales = kInnerBytes + kOuter * 128;
  static constexpr int kStageBytes = kScales + (MODE == kScaled ? kInner * 4 : 0);
  static constexpr int kOutBytes = 4096;             // of a wave, to bring its values into the output's order
  static constexpr int kLdsBytes = 2 * kStageBytes;  // the same bytes, after the last block
  static_assert(kLdsBytes >= kWaves * kOutBytes && kLdsBytes + kOuter * 4 <= 160 * 1024, "fits a compute unit");
  static constexpr int kI = IT * 32 / kM, kO = OT * 32 / kM, kSteps = kTileK / kInstrK;

  static __device__ __forceinline__ int inner_first(int wave) { return wave % WI * (IT * 32); }
  static __device__ __forceinline__ int outer_first(int wave) { return wave / WI * (OT * 32); }

  // Blocks 0 and 1 of a tile on their way.
  template <typename Loads>
  static __device__ __forceinline__ void start(Loads& loads) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      loads.fetch(b);
      loads.begin(b);
#pragma unroll
      for (int i = 0; i < Loads::kLoads; ++i) loads.issue(i, b * kStageBytes);
    }
  }

  // The products, after start().
  //
  // loads.issue(i, stage): one of the loads.kLoads loads of a block to LDS, in order.  What they need in registers
  // is asked for by loads.fetch(blk), early, and waited for by loads.begin(blk), right before the first of them.
  //
  // A block is four quarters.  All its fragments are in registers after its first one: the last quarter (of the block
  // before) and the first read those of half a block each, under the matrix instructions.  Its stage is then free for the
  // block after the next one, whose loads go out in the second and third quarter, at half the rate the memory units take
  // them, and have until the end of the next block's third, so that the last of them has a block's time.  A wait for all
  // loads but the last block's, once a block, leaves the rest in flight.
  template <typename Loads>
  static __device__ __forceinline__ void run(const InnerFragments& in, const OuterFragments& out, Loads& loads, int K,
                                             const uint8_t* lds, Sum (&acc)[kO][kI]) {
    constexpr int kLoads = Loads::kLoads, kReads = kSteps / 2 * (kI + kO), kSlots = kSteps * kI * kO / 4;
    const int blocks = (K - 1) / kTileK + 1;
    i32x4 fi[kSteps][kI], fo[kSteps][kO];
    // kScaled: the scales of a lane's four inner values of each tile, two to a register; those of the current tile; and the
    // products of the instruction before
    const int at_scales = kScales + (inner_first(threadIdx.x >> 6) + 4 * ((threadIdx.x & 63) / kM)) * 2;
    uint2 scales[kSteps][kI];
    f32x4 scale, before;
#pragma unroll
    for (int o = 0; o < kO; ++o)
#pragma unroll
      for (int t = 0; t < kI; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[o][t][i] = 0.0f;
    // fragment u of half `half` of a stage, in the order they are needed
    auto read = [&](const uint8_t* stage, int half, int u) {
      const int s = half * (kSteps / 2) + u / (kI + kO);
      u %= kI + kO;
      if (u == 0) fo[s][0] = out.read(stage + kInnerBytes, 0, s);
      else if (u <= kI) fi[s][u - 1] = in.read(stage, u - 1, s);
      else fo[s][u - kI] = out.read(stage + kInnerBytes, u - kI, s);
      if (MODE == kScaled && u < kI)
        scales[s][u] = *reinterpret_cast<const uint2*>(stage + at_scales + (s * kInner + u * kM) * 2);
    };
    // the products of quarter q; under them the fragments of half `half` of a stage, or a part of the loads
    auto quarter = [&](int q, const uint8_t* stage, int half, int part, uint32_t slot) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const int m = q * kSlots + j, s = m / (kI * kO);
        if constexpr (MODE == kScaled) {
          static_assert(kSlots % kO == 0 && kInstrK == kScaleGroup, "a tile's scale is looked up within the quarter");
          const int t = m % (kI * kO) / kO, o = j % kO;
          const f32x4 products = multiply_f16(fi[s][t], fo[s][o], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
          if (j > 0) add_scaled(acc[(j - 1) % kO][(m - 1) % (kI * kO) / kO], scale, before);
          if (o == 0)
            scale = f32x4{__uint_as_float(scales[s][t].x << 16), __uint_as_float(scales[s][t].x & 0xFFFF0000u),
                          __uint_as_float(scales[s][t].y << 16), __uint_as_float(scales[s][t].y & 0xFFFF0000u)};
          before = products;
          if (j == kSlots - 1) add_scaled(acc[o][t], scale, before);
        } else {
          const int o = m % (kI * kO) / kI, t = m % kI;
          acc[o][t] = MODE == kBothF16 ? multiply_f16(fi[s][t], fo[s][o], acc[o][t])
                                       : multiply_bf16(fi[s][t], fo[s][o], acc[o][t]);
        }
        if (half >= 0) {
          // all are under way three quarters through
          constexpr int kEnd = kSlots * 3 / 4;
#pragma unroll
          for (int u = j * kReads / kEnd; u < (j + 1) * kReads / kEnd && u < kReads; ++u) read(stage, half, u);
        }
        if (part >= 0) {
          const int at = part * kSlots + j;
#pragma unroll
          for (int i = at * kLoads / (2 * kSlots); i < (at + 1) * kLoads / (2 * kSlots); ++i) loads.issue(i, slot);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    wait_for_loads<Loads::kDirect>();
    loads.fetch(2);
#pragma unroll
    for (int u = 0; u < kReads; ++u) read(lds, 0, u);
    for (int b = 0; b < blocks; ++b) {
      const uint32_t slot = (b & 1) * kStageBytes;
      quarter(0, lds + slot, 1, -1, 0);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");     // all are done with this stage
      loads.begin(b + 2);
      quarter(1, nullptr, -1, 0, slot);
      quarter(2, nullptr, -1, 1, slot);
      wait_for_loads<Loads::kDirect>();    // the next block is there
      loads.fetch(b + 3);
      quarter(3, lds + (kStageBytes - slot), 0, -1, 0);
    }
    wait_for_loads<0>();                   // both stages are free again, and none lands in LDS after the end
  }

  static __device__ __forceinline__ void add_scaled(Sum& to, const f32x4& scale, const f32x4& products) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = fmaf(scale[i], products[i], to[i]);
  }

  // Waits for all but the last N loads of every wave.
  template <int N>
  static __device__ __forceinline__ void wait_for_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
  }

  // Stores the wave's values: row(r) is outer row r's first element in the output or -1, some(r) whether it has values
  // (else zeros), `left` the inner values from the tile's start on.  Runs of 32 rows and 128 bytes pass through a part of
  // LDS that is the wave's own, so that memory gets whole lines.
  template <typename Row, typename Some>
  static __device__ __forceinline__ void store(const Sum (&acc)[kO][kI], uint8_t* lds, void* out, int32_t dtype,
                                               int64_t width, int64_t left, Row row, Some some) {
    if (dtype == kF32) store_as<kF32>(acc, lds, out, width, left, row, some);
    else if (dtype == kBf16) store_as<kBf16>(acc, lds, out, width, left, row, some);
    else store_as<kF16>(acc, lds, out, width, left, row, some);
  }

  template <int DTYPE, typename Row, typename Some>
  static __device__ __forceinline__ void store_as(const Sum (&acc)[kO][kI], uint8_t* lds, void* out, int64_t width,
                                                  int64_t left, Row row, Some some) {
    constexpr int kSize = DTYPE == kF32 ? 4 : 2, kPart = 16 / kSize;
    constexpr int kRun = IT * 32 * kSize < 128 ? IT * 32 : 128 / kSize;    // inner values of a run
    constexpr int kParts = kRun * kSize / 16, kAtOnce = 64 / kParts;       // 16-byte parts of its rows, rows of a store
    static_assert(kRun % 32 == 0 && IT * 32 % kRun == 0 && (kParts == 8 || kParts == 4), "whole runs");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint8_t* own = lds + wave * kOutBytes;
    auto place = [](int r, int part) { return r * (kParts * 16) + ((part ^ (kParts == 8 ? r >> 1 & 7 : r >> 2 & 3)) << 4); };
    const bool whole = width % kPart == 0;
#pragma unroll
    for (int o = 0; o < OT; ++o) {
      int64_t at[32 / kAtOnce];
      bool in[32 / kAtOnce];
#pragma unroll
      for (int j = 0; j < 32 / kAtOnce; ++j) {
        const int r = outer_first(wave) + o * 32 + j * kAtOnce + lane / kParts;
        at[j] = row(r);
        in[j] = some(r);
      }
#pragma unroll
      for (int run = 0; run < IT * 32 / kRun; ++run) {
        // the run's values of 32 rows, four at a time
#pragma unroll
        for (int oo = 0; oo < 32 / kM; ++oo)
#pragma unroll
          for (int tt = 0; tt < kRun / kM; ++tt) {
            const Sum& v = acc[o * (32 / kM) + oo][run * (kRun / kM) + tt];
            const int i = tt * kM + 4 * (lane / kM);
            uint8_t* to = own + place(oo * kM + lane % kM, i / kPart);
            if constexpr (DTYPE == kF32) {
              *reinterpret_cast<f32x4*>(to) = v;
            } else {
              u16 h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) h[j] = DTYPE == kBf16 ? float_to_bf16(v[j]) : float_to_f16(v[j]);
              *reinterpret_cast<uint2*>(to + (i & 4) * 2) = uint2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
            }
          }
        const int64_t n = inner_first(wave) + run * kRun + lane % kParts * kPart;
#pragma unroll
        for (int j = 0; j < 32 / kAtOnce; ++j) {
          i32x4 v = *reinterpret_cast<const i32x4*>(own + place(j * kAtOnce + lane / kParts, lane % kParts));
          if (!in[j]) v = i32x4{0, 0, 0, 0};
          if (at[j] < 0 || n >= left) continue;
          uint8_t* to = static_cast<uint8_t*>(out) + (at[j] + n) * kSize;
          if (whole && left - n >= kPart) {
            *reinterpret_cast<i32x4*>(to) = v;
          } else {
#pragma unroll
            for (int e = 0; e < kPart; ++e)
              if (e < left - n) {
                if constexpr (DTYPE == kF32) reinterpret_cast<int*>(to)[e] = v[e];
                else reinterpret_cast<u16*>(to)[e] = (u16)((uint32_t)v[e / 2] >> e % 2 * 16);
              }
          }
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

template <int ROWS, int W, Weights FORM, Mode MODE>
struct InnerOperand {
  typedef Along<ROWS, W> Loader;
  typedef AlongFragments Fragments;
};
template <int ROWS, int W, Mode MODE>
struct InnerOperand<ROWS, W, kWeightsTransposed, MODE> {
  typedef Across<ROWS, W> Loader;
  typedef AcrossFragments<ROWS> Fragments;
};
template <int ROWS, int W, Mode MODE>
struct InnerOperand<ROWS, W, kWeights4, MODE> {
  typedef FourBit<ROWS, W, MODE == kScaled> Loader;
  typedef AlongFragments Fragments;
};

// The loads of a product's tile.
template <typename Inner, typename Outer, Weights FORM>
struct LinearLoads {
  static constexpr int kLoads = Inner::kLoads + Outer::kLoads;
  static constexpr int kDirect = FORM == kWeights4 ? Outer::kLoads : kLoads;     // those to LDS directly
  Inner in;
  Outer out;
  uint8_t* lds;
  uint32_t at;
  int K, wave, blk;
  i32x4 from;

  __device__ __forceinline__ void fetch(int b) {
    if constexpr (FORM == kWeights4) in.fetch(b, K);
  }
  __device__ __forceinline__ void begin(int b) {
    blk = b;
    if constexpr (FORM == kWeights4) in.settle();
    if constexpr (FORM == kWeightsTransposed) from = in.describe_block(b, K);
  }
  // what goes through registers first: it was waited for, and nothing that was issued since is waited for with it
  __device__ __forceinline__ void issue(int i, uint32_t slot) const {
    if (i < Inner::kLoads) {
      if constexpr (FORM == kWeights4) in.load(i, lds + slot, lds + slot + Inner::kBytes + Outer::kBytes);
      else if constexpr (FORM == kWeightsTransposed) in.load(i, from, wave, at + slot);
      else in.load(i, blk, K, wave, at + slot);
    } else {
      out.load(i - Inner::kLoads, blk, K, wave, at + slot + Inner::kBytes);
    }
  }
};

// WI IT 32 outputs of WO OT 32 rows.
template <Mode MODE, int WI, int WO, int IT, int OT, Weights FORM, bool FAR>
struct LinearUnit {
  typedef InnerOperand<WI * IT * 32, WI * WO, FORM, MODE> Inner;
  typedef Gathered<WO * OT * 32, WI * WO, FAR> Outer;
  typedef Tile16<MODE, WI, WO, IT, OT, typename Inner::Fragments, AlongFragments> Tile_;

  // rows t.row .. of group t.g, outputs i0 ..
  static __device__ __forceinline__ void run(const Linear16Args& a, const Tile& t, int i0, uint8_t* lds, int32_t* src) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int width = FORM == kWeightsTransposed ? a.C : a.N, K = FORM == kWeightsTransposed ? a.N : a.C;
    for (int r = threadIdx.x; r < Tile_::kOuter; r += Tile_::kThreads)
      src[r] = r < t.rows && t.g < a.G ? source_of(a.rows, a.fd_topk, a.X, t.row + r) : -1;
    __syncthreads();
    typename Tile_::Sum acc[Tile_::kO][Tile_::kI];
    if (t.g < a.G && a.X > 0) {
      LinearLoads<typename Inner::Loader, Outer, FORM> loads;
      loads.lds = lds;
      loads.at = lds_address(lds);
      loads.K = K;
      loads.wave = wave;
      const int64_t n = (int64_t)t.g * a.N;
      if constexpr (FORM == kWeightsTransposed)
        loads.in.init(lane, wave, static_cast<const uint8_t*>(a.w) + (n * a.C + i0) * 2, (int64_t)a.C * 2, width - i0);
      else if constexpr (FORM == kWeights)
        loads.in.init(lane, wave, static_cast<const uint8_t*>(a.w) + (n + i0) * K * 2, (uint32_t)K * 2, width - i0);
      else
        loads.in.init(lane, wave, a.q + (n + i0) * (K / 2), a.scale + (n + i0) * (K / kScaleGroup), K, width - i0);
      loads.out.init(lane, wave, static_cast<const uint8_t*>(a.x), a.ld * 2, a.X, [&](int r) { return src[r]; });
      typename Inner::Fragments in;
      AlongFragments out;
      in.init(lane, Tile_::inner_first(wave));
      out.init(lane, Tile_::outer_first(wave));
      Tile_::start(loads);
      Tile_::run(in, out, loads, K, lds, acc);
    }
    Tile_::store(acc, lds, a.y, a.y_dtype, width, width - i0,
                 [&](int r) -> int64_t { return r < t.rows ? (int64_t)(t.row + r) * width + i0 : -1; },
                 [&](int r) { return src[r] >= 0; });
  }
};

// Tiles of 128 x 128, four waves, two workgroups to a compute unit.
template <Mode MODE, Weights FORM, bool FAR>
__global__ __launch_bounds__(256, 2) void linear_small_kernel(Linear16Args a, int32_t columns) {
  typedef LinearUnit<MODE, 2, 2, 2, 2, FORM, FAR> Unit;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int32_t src[128];
  const int32_t row_tiles = count_tiles(a.offsets, a.G, a.R, 128, true);
  const int64_t tiles = min((int64_t)row_tiles * columns, (int64_t)gridDim.x);    // less where offsets decrease
  if (blockIdx.x >= tiles) return;
  int32_t row, column;
  band_order(die_order(blockIdx.x, (int32_t)tiles), row_tiles, columns, row, column);
  const Tile t = find_tile(a.offsets, a.G, a.R, 128, row, true);
  if (t.g < 0) return;
  Unit::run(a, t, column * 128, lds, src);
}

// Tiles of 256 x 256, eight waves, one workgroup to a compute unit.  The chip takes 256 at a time, so what does not fill a
// round of them is given out in smaller pieces at the end: full tiles past the last whole round as two of 256 x 128 each
// (where that makes one round of half the time), and what a group has behind its last 256 rows as 256 x 128 or, for 128
// rows or fewer, 128 x 128.
constexpr int kUnits = 256;                // compute units

struct LargePlan {
  int32_t full_rows, part_rows;            // row tiles of 256 rows; groups with rows behind them
  int64_t whole, split;                    // tiles given out whole, and in two pieces
  int64_t blocks;
};

__host__ __device__ __forceinline__ LargePlan plan_large(int32_t full_rows, int32_t part_rows, int64_t columns) {
  LargePlan p;
  p.full_rows = full_rows;
  p.part_rows = part_rows;
  const int64_t full = full_rows * columns, over = full % kUnits;
  p.split = over <= kUnits / 2 ? over : 0;
  p.whole = full - p.split;
  p.blocks = p.whole + 2 * p.split + 2 * columns * part_rows;
  return p;
}

// Row tile `want` of 256 rows of all groups in order, or (want past them) what is behind the last one of a group.
__device__ __forceinline__ Tile find_large(const int32_t* offsets, int32_t G, int32_t R, int32_t want, bool part) {
  const int lane = threadIdx.x & 63;
  int32_t carry = 0;
  for (int32_t g0 = 0; g0 < G + 2; g0 += 64) {
    const int32_t g = g0 + lane;
    const Span s = g < G + 2 ? group_span(offsets, g, G, R) : Span{0, 0};
    const int32_t rows = s.hi > s.lo ? s.hi - s.lo : 0, tiles = part ? rows % 256 != 0 : rows / 256;
    int32_t incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t v = __shfl_up(incl, d);
      if (lane >= d) incl = add_tiles(incl, v);
    }
    const int32_t before = add_tiles(carry, incl - tiles);
    const u64 here = __ballot(want >= before && want - before < tiles);
    if (here != 0) {
      const int at = __ffsll((unsigned long long)here) - 1;
      const int32_t skip = part ? __shfl(rows, at) / 256 : want - __shfl(before, at);
      Tile t;
      t.g = __builtin_amdgcn_readfirstlane(g0 + at);
      t.row = __builtin_amdgcn_readfirstlane(__shfl(s.lo, at) + skip * 256);
      t.rows = __builtin_amdgcn_readfirstlane(part ? __shfl(rows, at) % 256 : 256);
      return t;
    }
    carry = __builtin_amdgcn_readfirstlane(__shfl(add_tiles(carry, incl), 63));
  }
  return Tile{-1, 0, 0};
}

__device__ __forceinline__ LargePlan plan_large(const int32_t* offsets, int32_t G, int32_t R, int64_t columns) {
  const int lane = threadIdx.x & 63;
  int32_t full = 0, part = 0;
  for (int32_t g = lane; g < G + 2; g += 64) {
    const Span s = group_span(offsets, g, G, R);
    const int32_t rows = s.hi > s.lo ? s.hi - s.lo : 0;
    full = add_tiles(full, rows / 256);
    part += rows % 256 != 0;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    full = add_tiles(full, __shfl_xor(full, d));
    part += __shfl_xor(part, d);
  }
  return plan_large(__builtin_amdgcn_readfirstlane(full), __builtin_amdgcn_readfirstlane(part), columns);
}

template <Mode MODE, Weights FORM>
__global__ __launch_bounds__(512) void linear_large_kernel(Linear16Args a, int32_t columns) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int32_t src[256];
  const LargePlan p = plan_large(a.offsets, a.G, a.R, columns);
  int64_t id = blockIdx.x;
  if (id < p.whole) {
    int32_t row, column;
    band_order(die_order((int32_t)id, (int32_t)min(p.whole, (int64_t)gridDim.x)), p.full_rows, columns, row, column);
    const Tile t = find_large(a.offsets, a.G, a.R, row, false);
    if (t.g < 0) return;
    if constexpr (MODE == kScaled) {
      // scales take the registers that the sums of half the rows would: one half after the other
      LinearUnit<MODE, 4, 2, 2, 2, FORM, false>::run(a, Tile{t.g, t.row, 128}, column * 256, lds, src);
      __syncthreads();
      LinearUnit<MODE, 4, 2, 2, 2, FORM, false>::run(a, Tile{t.g, t.row + 128, 128}, column * 256, lds, src);
    } else {
      LinearUnit<MODE, 4, 2, 2, 4, FORM, false>::run(a, t, column * 256, lds, src);
    }
    return;
  }
  id -= p.whole;
  const int32_t width = FORM == kWeightsTransposed ? a.C : a.N;
  int32_t row, column;
  Tile t;
  if (id < 2 * p.split) {
    band_order((int32_t)(p.whole + id / 2), p.full_rows, columns, row, column);
    t = find_large(a.offsets, a.G, a.R, row, false);
    column = column * 256 + (int32_t)(id & 1) * 128;
  } else {
    id -= 2 * p.split;
    t = find_large(a.offsets, a.G, a.R, (int32_t)min(id / (2 * columns), (int64_t)0x7FFFFFFF), true);
    column = (int32_t)(id % (2 * columns)) * 128;
  }
  if (t.g < 0 || column >= width) return;
  if (t.rows > 128) LinearUnit<MODE, 4, 2, 1, 4, FORM, false>::run(a, t, column, lds, src);
  else LinearUnit<MODE, 4, 2, 1, 2, FORM, false>::run(a, t, column, lds, src);
}

inline int64_t small_blocks(int64_t R, int64_t width, int32_t G) {
  // every group adds at most one tile that is not full, and a tile has a row
  return (std::min(R, R / 128 + G) + 2) * ceil_div(width, 128);
}

inline int64_t large_blocks(int64_t R, int64_t width, int32_t G) {
  const int64_t columns = ceil_div(width, 256);
  return R / 256 * columns + kUnits / 2 + 2 * columns * std::min(R, (int64_t)G + 2);
}

// Large tiles where there are enough of them for the chip: 16-bit weights, 256 tiles: 120 us in small ones, 100 in large ones
// (4096 rows of one group, 4096 x 4096), 288: 139 and 142 (8192 rows on 9, 2048 x 4096), 160: 82 and 105 (4096 rows), 192: 49
// and 69 (8192 rows on 32, 1024 x 2048).  4-bit weights are converted once for twice the rows there: 224 tiles: 126 and 113
// (6144 rows on 9), 160: 111 and 111, 128: 36 and 34 (4096 rows on 32, 1024 x 2048; 36 and 53 where the largest group has
// three times the mean: nearly every group ends in a rest of its own), 48: 29 and 32.
inline bool large_suits(int64_t R, int64_t width, int32_t G, bool four) {
  return R >= 128 * (int64_t)G && (R / 256 + G / 2) * ceil_div(width, 256) >= (four ? 128 : 256);
}

// Two stages of a block of both operands, and of scales where they are apart.
constexpr unsigned lds_bytes(Mode mode, int side) { return 2 * (2 * side * 128 + (mode == kScaled ? side * 4 : 0)); }

template <Mode MODE, Weights FORM>
hipError_t launch_tiles(const Linear16Args& a, hipStream_t stream) {
  const int64_t width = FORM == kWeightsTransposed ? a.C : a.N;
  const bool far = a.X * a.ld * 2 >= (int64_t)kOutside;
  if (!far && large_suits(a.R, width, a.G, FORM == kWeights4)) {
    linear_large_kernel<MODE, FORM><<<dim3((unsigned)large_blocks(a.R, width, a.G)), dim3(512), lds_bytes(MODE, 256), stream>>>(a, (int32_t)ceil_div(width, 256));
    return hipGetLastError();
  }
  const dim3 grid((unsigned)small_blocks(a.R, width, a.G));
  const int32_t columns = (int32_t)ceil_div(width, 128);
  if (far) linear_small_kernel<MODE, FORM, true><<<grid, dim3(256), lds_bytes(MODE, 128), stream>>>(a, columns);
  else linear_small_kernel<MODE, FORM, false><<<grid, dim3(256), lds_bytes(MODE, 128), stream>>>(a, columns);
  return hipGetLastError();
}

// Workgroups of whichever form a product takes.
inline int64_t tile_blocks(int64_t R, int64_t width, int32_t G, bool four) {
  return std::max(small_blocks(R, width, G), large_suits(R, width, G, four) ? large_blocks(R, width, G) : 0);
}

}  // namespace eplb
