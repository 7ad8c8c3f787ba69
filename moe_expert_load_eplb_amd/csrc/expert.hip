// The experts' products in 8-bit floating point with a scale for each block
// of 128.
//
// Both products have the same shape: out[o][i] = sum over blocks b of 128 of
// so[o][b] * si[i][b] * (sum over j in b of O[o][j] * I[i][j]), with the
// inner index i contiguous in the output (matmul: o = row, i = n, j = k;
// weight gradient: o = n, i = k, j = row).  The sum within a block is what its
// scales multiply; the sum over blocks is kept in 32-bit registers.  The inner
// operand is the matrix instruction's first, which leaves consecutive i of one
// o in each lane.
//
// Sums within a block.  All products are taken by the 16-bit matrix
// instruction, whose sums keep 32 bits (measured: 7e-8 of a typical sum); the
// 8-bit values become 16-bit ones exactly on the way from LDS, two per vector
// instruction.  The 8-bit matrix instruction has twice its rate, but aligns each
// 8 consecutive products to the largest of them and drops what lies below 2^-13
// of it: where large products cancel, nothing is left of the small ones beside
// them, in an output of any type.
#include "experts_device.h"

namespace eplb {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Half h of 16 8-bit values as 16-bit ones.
__device__ __forceinline__ f16x8 half_of(i32x4 v, int h) {
  const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * h], 1.0f, false);
  const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * h], 1.0f, true);
  const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * h + 1], 1.0f, false);
  const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * h + 1], 1.0f, true);
  return f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// 16 x 16 sums over 128: a lane's 32 values of each operand, in two parts.
__device__ __forceinline__ f32x4 mfma_block(const i32x4 (&a)[2], const i32x4 (&b)[2]) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s)
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(half_of(a[s >> 1], s & 1), half_of(b[s >> 1], s & 1), d, 0, 0, 0);
  return d;
}

// Four consecutive values of one output row; `left` of them are inside.
__device__ __forceinline__ void store4(void* p, int32_t dtype, int64_t at, int left, bool vec, f32x4 v) {
  if (vec && left >= 4) {
    if (dtype == kF32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = v;
    } else {
      uint2 w;
      if (dtype == kBf16) {
        w.x = float_to_bf16(v[0]) | (uint32_t)float_to_bf16(v[1]) << 16;
        w.y = float_to_bf16(v[2]) | (uint32_t)float_to_bf16(v[3]) << 16;
      } else {
        w.x = float_to_f16(v[0]) | (uint32_t)float_to_f16(v[1]) << 16;
        w.y = float_to_f16(v[2]) | (uint32_t)float_to_f16(v[3]) << 16;
      }
      *reinterpret_cast<uint2*>(static_cast<u16*>(p) + at) = w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) store_float(p, dtype, at + j, v[j]);
}

// ---------------------------------------------------------------- few rows
// The streaming form, for groups of few rows: the weights are read once, from
// memory to registers, and bound the time.  A wave takes 16 n of one group
// through K; both operands of eight blocks of 128 are in flight at once (2 KiB
// each).  With the memory as the bound, 16-bit products cost nothing and keep
// 32-bit sums.  No load stands behind a branch (rows and blocks past
// the end are clamped to the last ones and not used): a load that may or may
// not have been issued makes every wait behind it wait for all of them.
constexpr int kStreamThreads = 256;
constexpr int kStream16N = 64;             // n of a workgroup: 16 of each wave

// The two 16-byte parts of block kb that a lane of `quad` holds; at the end of
// a row that has no such part, its first ones (the caller zeroes the other
// operand there).
__device__ __forceinline__ void load_parts(const uint8_t* row, int kb, int quad, int K, i32x4& lo, i32x4& hi) {
  const int k0 = kb * kBlock + quad * 16, k1 = k0 + 64;
  lo = *reinterpret_cast<const i32x4*>(row + (k0 < K ? k0 : 0));
  hi = *reinterpret_cast<const i32x4*>(row + (k1 < K ? k1 : 0));
}

// The row of the operand that grouped row `r` reads, or -1.
__device__ __forceinline__ int32_t source_row(const MatmulArgs& a, int32_t r) {
  int32_t from = r;
  if (a.rows != nullptr) {
    from = a.rows[r];
    from = from < 0 ? -1 : (int32_t)fastdiv_apply((uint32_t)from, a.fd_topk);
  }
  return from < a.X ? from : -1;
}

// A row of per-block scales that is the same for the whole wave: lane i holds
// the scale of the i-th block from one on, for two runs of blocks (this one,
// the next).
struct ScaleRow {
  const float* p;
  int n;
  float now, next;
  __device__ __forceinline__ ScaleRow(const float* row, int blocks) : p(row), n(blocks), next(0.0f) {
    now = p[min((int)(threadIdx.x & 63), n - 1)];
  }
  __device__ __forceinline__ void load_next(int from) { next = p[min(from + (int)(threadIdx.x & 63), n - 1)]; }
  __device__ __forceinline__ void advance() { now = next; }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(now), i));
  }
};

constexpr int kAhead16 = 8;                // blocks in flight

__global__ __launch_bounds__(kStreamThreads) void expert_stream16_kernel(MatmulArgs a, int32_t n_tiles) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, quad = lane >> 4, col = lane & 15;
  const int n0 = (int)(blockIdx.x % n_tiles) * kStream16N + wave * 16;
  const Tile t = find_tile(a.offsets, a.G, a.R, 16, (int32_t)(blockIdx.x / n_tiles), true);
  if (t.g < 0 || n0 >= a.N) return;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  if (t.g < a.G && a.X > 0) {
    const int n = n0 + col < a.N ? n0 + col : a.N - 1;
    const uint8_t* w = a.w + ((int64_t)t.g * a.N + n) * a.K;
    i32x4 rw[kAhead16][2], rx[kAhead16][2];
    float sx[kAhead16];
    // loads return in order: the short ones that the next addresses need go first
    const int32_t from = col < t.rows ? source_row(a, t.row + col) : -1;
#pragma unroll
    for (int p = 0; p < kAhead16; ++p) load_parts(w, min(p, a.KB - 1), quad, a.K, rw[p][0], rw[p][1]);
    ScaleRow ws(a.w_scale + ((int64_t)t.g * a.NB + n0 / kBlock) * a.KB, a.KB);
    const uint8_t* x = a.q + (int64_t)(from < 0 ? 0 : from) * a.K;
    const float* xs = a.scale + (int64_t)(from < 0 ? 0 : from) * a.KB;
#pragma unroll
    for (int p = 0; p < kAhead16; ++p) {
      const int kb = min(p, a.KB - 1);
      load_parts(x, kb, quad, a.K, rx[p][0], rx[p][1]);
      sx[p] = xs[kb];
    }
    for (int kb0 = 0; kb0 < a.KB; kb0 += kAhead16) {
      ws.load_next(kb0 + kAhead16);
#pragma unroll
      for (int p = 0; p < kAhead16; ++p) {
        const int i = kb0 + p;               // past the end: not added
        const i32x4 zero = {0, 0, 0, 0};
        const int k = i * kBlock + quad * 16;
        const i32x4 fw[2] = {rw[p][0], rw[p][1]};
        const i32x4 fx[2] = {k < a.K ? rx[p][0] : zero, k + 64 < a.K ? rx[p][1] : zero};
        const float sc = ws.get(p) * sx[p];
        const int next = min(i + kAhead16, a.KB - 1);
        load_parts(w, next, quad, a.K, rw[p][0], rw[p][1]);
        load_parts(x, next, quad, a.K, rx[p][0], rx[p][1]);
        sx[p] = xs[next];
        const f32x4 d = mfma_block(fw, fx);
        if (i < a.KB) {
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] += d[j] * sc;
        }
      }
      ws.advance();
    }
    if (from < 0) acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int n = n0 + quad * 4;
  if (col < t.rows) store4(a.y, a.dtype, (int64_t)(t.row + col) * a.N + n, a.N - n, a.N % 4 == 0, acc);
}

// ---------------------------------------------------------------- tiles
// Tiles of the output, for many rows.  A workgroup of WI x WO waves computes
// (WI IT 32) inner x (WO OT 32) outer values, a wave IT x OT tiles of 32 x 32
// (32 x 32 x 64 reaches 4.4 POPS on its own, 16 x 16 x 128 4.0).  The operands
// of a block of 128 (rows of 128 bytes) and its scales go from memory to LDS
// without passing through registers, STAGES - 1 blocks ahead; one barrier per
// block.  Every wave issues the same number of such loads per block, so that
// waiting for all but the later blocks' is waiting for this one's.
//
// A row's eight 16-byte parts are permuted (on the way in, by the address a
// lane loads from) so that eight lanes that read one part of eight rows reach
// all banks.  The inner rows of a wave are taken in an order that leaves a
// lane with 16 IT consecutive inner values of one outer row.
//
// Measured, weights not in any cache.  Low tiles, 8 rows on 8 of 32 experts,
// 4096 x 2048 (67 MB): 18.7 us, 3.6 TB/s.  Small tiles, 56 rows to a group, 2048 x
// 4096: a block takes a workgroup 0.7 us as long as each has a compute unit to
// itself (64 workgroups 22.3 us, 256 23.4): a wave, alone on its SIMD, issues
// about 160 vector and 8 matrix instructions for two thirds of it and waits for
// loads and LDS the rest.  So a second workgroup on a unit adds half of the first
// one's time and more (512: 38.8 us, 3.5 TB/s), also where few units have two (288,
// which is 9 groups: 34.6 us, 2.2 TB/s).  Wide tiles, 16384 rows on 9, 4096 x 4096,
// bfloat16 output: 622 to 654 us, 0.84 to 0.88 PFLOP/s: the matrix units are busy
// for 47 % of the time and the vector units for 44 %, with 7.6 instructions to a
// matrix instruction (conversions to 16 bits, and 16 multiply-adds a lane and tile
// for the scales, which the matrix unit's output has to pass through); two waves
// to a SIMD overlap little of the two.  Weight gradient, 16384 rows on 9, 2048 x
// 4096, 32-bit output: 375 to 402 us, 0.68 to 0.73 PFLOP/s, with two scales to each
// product: 37 % and 46 %; it stores 302 MB.
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __attribute__((aligned(16))) uint8_t g_zeros[16];   // read in place of what lies past the end of K

__device__ __forceinline__ void load_to_lds16(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

__device__ __forceinline__ void load_to_lds4(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 4, 0, 0);
}

// Waits until at most N of this wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Eight consecutive values of one output row; `left` of them are inside.
__device__ __forceinline__ void store8(void* p, int32_t dtype, int64_t at, int left, int64_t width, const float* v) {
  if (dtype != kF32 && left >= 8 && width % 8 == 0) {
    u16 h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = dtype == kBf16 ? float_to_bf16(v[j]) : float_to_f16(v[j]);
    uint4 w;
    w.x = h[0] | (uint32_t)h[1] << 16;
    w.y = h[2] | (uint32_t)h[3] << 16;
    w.z = h[4] | (uint32_t)h[5] << 16;
    w.w = h[6] | (uint32_t)h[7] << 16;
    *reinterpret_cast<uint4*>(static_cast<u16*>(p) + at) = w;
    return;
  }
  store4(p, dtype, at, left, width % 4 == 0, f32x4{v[0], v[1], v[2], v[3]});
  if (left > 4) store4(p, dtype, at + 4, left - 4, width % 4 == 0, f32x4{v[4], v[5], v[6], v[7]});
}

// What a workgroup multiplies: both products in one form.
struct TileJob {
  const uint8_t* inner;      // first inner row of the tile
  int64_t inner_ld;
  int inner_rows;            // rows inside (the others read the last one and are not stored)
  // scale i of block b: inner_scale[i * inner_scale_ld + b * inner_step], i < inner_scales.  Matmul: one for each 128
  // inner rows, the tile's first row being row inner_first of its 128; weight gradient: one for each row
  const float* inner_scale;
  int64_t inner_scale_ld, inner_step;
  int inner_scales, inner_first;
  int64_t outer_step;        // from one block's scale of an outer row to the next one's
  int64_t K;                 // elements of a row (matmul: past it zeros)
  int block0, blocks;        // first block, number of blocks
};

template <int WI, int WO, int IT, int OT, int STAGES, bool WGRAD>
struct TileKernel {
  static constexpr int kWaves = WI * WO, kThreads = kWaves * 64;
  static constexpr int kInner = WI * IT * 32, kOuter = WO * OT * 32;
  static constexpr int kInnerLoads = kInner / 8 / kWaves, kOuterLoads = kOuter / 8 / kWaves;   // of 8 rows, per wave
  static constexpr int kOuterScaleWaves = (kOuter + 63) / 64, kInnerScaleWaves = WGRAD ? (kInner + 63) / 64 : 1;
  static constexpr int kLoads = kInnerLoads + kOuterLoads + 1;
  static constexpr int kScaleWords = (kOuterScaleWaves + kInnerScaleWaves + 1) * 64;
  static constexpr int kStageBytes = (kInner + kOuter) * kBlock + kScaleWords * 4;
  static constexpr int kLdsBytes = STAGES * kStageBytes;
  static_assert(kInner % (8 * kWaves) == 0 && kOuter % (8 * kWaves) == 0, "whole loads");
  static_assert(kOuterScaleWaves + kInnerScaleWaves <= kWaves, "one load of scales per wave");

  // How the parts of row r are permuted: by bits 1 to 3 of the row, as two
  // rows make one turn of the banks.
  static __device__ __forceinline__ int key(int r) { return r >> 1 & 7; }

  // The element of a block that this lane's load p starts at.
  static __device__ __forceinline__ int inner_part(int p, int wave, int lane) {
    return ((lane & 7) ^ key((wave * kInnerLoads + p) * 8 + (lane >> 3))) * 16;
  }
  static __device__ __forceinline__ int outer_part(int p, int wave, int lane) {
    return ((lane & 7) ^ key((wave * kOuterLoads + p) * 8 + (lane >> 3))) * 16;
  }

  // `outer_row(r)`: pointer to outer row r of the tile (any valid row where it has none).
  template <typename OuterRow, typename OuterScale>
  static __device__ __forceinline__ void run(const TileJob& job, uint8_t* lds, OuterRow outer_row,
                                             OuterScale outer_scale, f32x16 (&acc)[OT][IT]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int wi = wave % WI * (IT * 32), wo = wave / WI * (OT * 32);
#pragma unroll
    for (int o = 0; o < OT; ++o)
#pragma unroll
      for (int t = 0; t < IT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[o][t][i] = 0.0f;

    // what this lane loads of every block
    // from the tile's start: matmul below 2^32, as there are at most 256 rows of at most 2^24 bytes; a row of padded
    // rows may be longer
    typedef typename std::conditional<WGRAD, int64_t, uint32_t>::type Offset;
    static_assert(kInner <= 256, "inner offsets in 32 bits");
    Offset ip[kInnerLoads];
    const uint8_t* op[kOuterLoads];
#pragma unroll
    for (int p = 0; p < kInnerLoads; ++p) {
      const int r = (wave * kInnerLoads + p) * 8 + (lane >> 3);
      ip[p] = (Offset)min(r, job.inner_rows - 1) * (Offset)job.inner_ld + (Offset)inner_part(p, wave, lane);
    }
#pragma unroll
    for (int p = 0; p < kOuterLoads; ++p)
      op[p] = outer_row((wave * kOuterLoads + p) * 8 + (lane >> 3)) + outer_part(p, wave, lane);
    const float* sp;
    int64_t s_step = job.outer_step;
    int s_at = wave * 64;
    if (wave < kOuterScaleWaves) {
      sp = outer_scale(wave * 64 + lane);
    } else if (wave < kOuterScaleWaves + kInnerScaleWaves) {
      sp = job.inner_scale + min((wave - kOuterScaleWaves) * 64 + lane, job.inner_scales - 1) * job.inner_scale_ld;
      s_step = job.inner_step;
    } else {
      sp = outer_scale(0);                   // keeps the count of loads equal; its place is not read
      s_at = (kOuterScaleWaves + kInnerScaleWaves) * 64;
    }
    // block b of the job to stage `slot`; past the end the last one again
    auto load = [&](int b, int slot) {
      const int64_t blk = job.block0 + min(b, job.blocks - 1);
      uint8_t* stage = lds + slot * kStageBytes;
      uint8_t* si = stage + wave * kInnerLoads * 1024;
      uint8_t* so = stage + kInner * kBlock + wave * kOuterLoads * 1024;
      const uint8_t* inner = job.inner + blk * kBlock;
      if (WGRAD || (blk + 1) * kBlock <= job.K) {
#pragma unroll
        for (int p = 0; p < kInnerLoads; ++p) load_to_lds16(inner + ip[p], si + p * 1024);
#pragma unroll
        for (int p = 0; p < kOuterLoads; ++p) load_to_lds16(op[p] + blk * kBlock, so + p * 1024);
      } else {                               // the end of K: the row's first inner part against zeros
        const int left = (int)(job.K - blk * kBlock);
#pragma unroll
        for (int p = 0; p < kInnerLoads; ++p) {
          const int k = inner_part(p, wave, lane);
          load_to_lds16(k < left ? inner + ip[p] : job.inner + (ip[p] - k), si + p * 1024);
        }
#pragma unroll
        for (int p = 0; p < kOuterLoads; ++p)
          load_to_lds16(outer_part(p, wave, lane) < left ? op[p] + blk * kBlock : g_zeros, so + p * 1024);
      }
      load_to_lds4(sp + blk * s_step, stage + (kInner + kOuter) * kBlock + s_at * 4);
    };
#pragma unroll
    for (int p = 0; p < STAGES - 1; ++p) load(p, p);
    int slot = 0;
    for (int b = 0; b < job.blocks; ++b) {
      wait_loads<kLoads * (STAGES - 2)>();   // this block's have arrived, of this wave
      // of all waves; and all are done with the block before (a barrier that
      // does not wait for the later blocks' loads)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      load(b + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
      const uint8_t* it = lds + slot * kStageBytes;
      slot = slot + 1 == STAGES ? 0 : slot + 1;
      const uint8_t* ot = it + kInner * kBlock;
      const float* scales = reinterpret_cast<const float*>(ot + kOuter * kBlock);
      const float one = WGRAD ? 1.0f : scales[kOuterScaleWaves * 64 + (job.inner_first + wi) / kBlock];
      auto part = [&](const uint8_t* tile, int row, int g) {
        return *reinterpret_cast<const i32x4*>(tile + row * kBlock + ((g ^ key(row)) << 4));
      };
      // a lane's 64 of the block's 128 elements, the same of both operands
      i32x4 fi[IT][4];
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int r = wi + (col >> 2 & 1) * (16 * IT) + 16 * t + (col >> 3) * 4 + (col & 3);
#pragma unroll
        for (int g = 0; g < 4; ++g) fi[t][g] = part(it, r, (g >> 1) * 4 + half * 2 + (g & 1));
      }
      f32x4 si[IT][4];
      if (WGRAD) {
#pragma unroll
        for (int t = 0; t < IT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            si[t][j] = *reinterpret_cast<const f32x4*>(scales + kOuterScaleWaves * 64 + wi + half * (16 * IT) + 16 * t +
                                                       j * 4);
      }
      // a tile's scales are applied while the next tile's products are in the
      // matrix pipeline
      f32x16 d[2];
      float sc[2];
      auto apply = [&](int j) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[j / IT][j % IT][i] += d[j & 1][i] * (WGRAD ? sc[j / IT & 1] * si[j % IT][i >> 2][i & 3] : sc[j / IT & 1]);
      };
      i32x4 fo[2][4];                        // outer fragments, one set ahead of the matrix instructions
      auto outer = [&](int o) {
#pragma unroll
        for (int g = 0; g < 4; ++g) fo[o & 1][g] = part(ot, wo + o * 32 + col, (g >> 1) * 4 + half * 2 + (g & 1));
        sc[o & 1] = scales[wo + o * 32 + col] * one;
      };
      outer(0);
#pragma unroll
      for (int o = 0; o < OT; ++o) {
#pragma unroll
        for (int t = 0; t < IT; ++t) {
          const int j = o * IT + t;
#pragma unroll
          for (int i = 0; i < 16; ++i) d[j & 1][i] = 0.0f;
          if (IT * OT == 1) {        // no other tile to fill the pipeline with: two sums side by side
#pragma unroll
            for (int i = 0; i < 16; ++i) d[1][i] = 0.0f;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                d[h] = __builtin_amdgcn_mfma_f32_32x32x16_f16(half_of(fi[t][g], h), half_of(fo[o & 1][g], h), d[h],
                                                            0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; ++i) d[0][i] += d[1][i];
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                d[j & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(half_of(fi[t][g], h), half_of(fo[o & 1][g], h),
                                                                  d[j & 1], 0, 0, 0);
          }
          if (j > 0) apply(j - 1);
          // the tile before has had its scale by now
          if (t == 0 && o + 1 < OT) outer(o + 1);
        }
      }
      apply(OT * IT - 1);
    }
    wait_loads<0>();                         // none may land in LDS that is no longer this workgroup's
  }

  // Stores the wave's values: row(r) is outer row r's first element in the
  // output or -1, some(r) whether it has values (else zeros), `left` the inner
  // values from the tile's start on.
  template <typename Row, typename Some>
  static __device__ __forceinline__ void store(const f32x16 (&acc)[OT][IT], void* out, int32_t dtype, int64_t width,
                                               int64_t left, Row row, Some some) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int wi = wave % WI * (IT * 32) + half * (16 * IT), wo = wave / WI * (OT * 32);
#pragma unroll
    for (int o = 0; o < OT; ++o) {
      const int64_t at = row(wo + o * 32 + col);
      if (at < 0) continue;
      const bool in = some(wo + o * 32 + col);
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = in ? acc[o][t][i] : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          const int64_t n = wi + 16 * t + i;
          if (n < left) store8(out, dtype, at + n, left - n < 8 ? (int)(left - n) : 8, width, v + i);
        }
      }
    }
  }
};

template <int WI, int WO, int IT, int OT, int STAGES>
__global__ __launch_bounds__(WI* WO * 64) void expert_tile_kernel(MatmulArgs a, int32_t n_tiles) {
  typedef TileKernel<WI, WO, IT, OT, STAGES, false> K;
  // Large tiles: the workgroups of one die take neighbouring tiles, which share operands in its cache.  Small tiles
  // run where the weights are read once or few, and are found without counting them all first.
  constexpr bool kOrdered = IT * OT > 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t tile_lds[];
  __shared__ int32_t src[K::kOuter];
  int32_t row = blockIdx.x / n_tiles, column = blockIdx.x % n_tiles;
  if (kOrdered) {
    const int32_t row_tiles = count_tiles(a.offsets, a.G, a.R, K::kOuter, true);
    const int64_t tiles = min((int64_t)row_tiles * n_tiles, (int64_t)gridDim.x);    // less where offsets decrease
    if (blockIdx.x >= tiles) return;
    band_order(die_order(blockIdx.x, (int32_t)tiles), row_tiles, n_tiles, row, column);
  }
  const Tile t = find_tile(a.offsets, a.G, a.R, K::kOuter, row, true);
  if (t.g < 0) return;
  const int64_t n0 = (int64_t)column * K::kInner;
  for (int r = threadIdx.x; r < K::kOuter; r += K::kThreads)
    src[r] = r < t.rows && t.g < a.G ? source_row(a, t.row + r) : -1;
  __syncthreads();
  f32x16 acc[OT][IT];
  if (t.g < a.G && a.X > 0) {
    TileJob job;
    job.inner = a.w + ((int64_t)t.g * a.N + n0) * a.K;
    job.inner_ld = a.K;
    job.inner_rows = (int)(a.N - n0 < K::kInner ? a.N - n0 : K::kInner);
    job.inner_scale = a.w_scale + ((int64_t)t.g * a.NB + n0 / kBlock) * a.KB;
    job.inner_scale_ld = a.KB;
    job.inner_step = job.outer_step = 1;
    job.inner_scales = a.NB - (int)(n0 / kBlock);
    job.inner_first = (int)(n0 % kBlock);
    job.block0 = 0;
    job.blocks = a.KB;
    job.K = a.K;
    K::run(job, tile_lds, [&](int r) { return a.q + (int64_t)max(src[r], 0) * a.K; },
           [&](int r) { return a.scale + (int64_t)max(src[r < K::kOuter ? r : 0], 0) * a.KB; }, acc);
  }
  K::store(acc, a.y, a.dtype, a.N, a.N - n0,
           [&](int r) -> int64_t { return r < t.rows ? (int64_t)(t.row + r) * a.N + n0 : -1; },
           [&](int r) { return src[r] >= 0; });
}

template <int WI, int WO, int IT, int OT, int STAGES>
__global__ __launch_bounds__(WI* WO * 64) void expert_wgrad_kernel(WgradArgs a, int32_t ni, int32_t no) {
  typedef TileKernel<WI, WO, IT, OT, STAGES, true> K;
  extern __shared__ __attribute__((aligned(16))) uint8_t tile_lds[];
  const int32_t id = die_order(blockIdx.x, gridDim.x);
  const int32_t g = id / (ni * no);
  int32_t row, column;
  band_order(id - g * (ni * no), no, ni, row, column);
  const int64_t i0 = (int64_t)column * K::kInner, o0 = (int64_t)row * K::kOuter;
  // the group's blocks of 128 rows
  const int32_t before = count_tiles(a.offsets, g, a.R, kBlock, false);
  TileJob job;
  job.block0 = before;
  job.blocks = tiles_of(group_span(a.offsets, g, a.G, a.R), kBlock);
  if ((int64_t)job.block0 + job.blocks > a.Rp / kBlock) job.blocks = (int)(a.Rp / kBlock) - job.block0;
  job.inner = a.x + i0 * a.Rp;
  job.inner_ld = a.Rp;
  job.inner_rows = (int)(a.K - i0 < K::kInner ? a.K - i0 : K::kInner);
  job.inner_scale = a.x_scale + i0;
  job.inner_scale_ld = 1;
  job.inner_step = a.K;
  job.inner_scales = job.inner_rows;
  job.inner_first = 0;
  job.outer_step = a.N;
  job.K = a.Rp;
  const int64_t last = a.N - 1 - o0;
  f32x16 acc[OT][IT];
  const bool some = job.blocks > 0;
  if (some)
    K::run(job, tile_lds, [&](int r) { return a.dy + (o0 + (r < last ? r : last)) * a.Rp; },
           [&](int r) { return a.dy_scale + o0 + (r < last ? r : last); }, acc);
  K::store(acc, a.dw, a.dtype, a.K, a.K - i0,
           [&](int r) -> int64_t { return r <= last ? ((int64_t)g * a.N + o0 + r) * a.K + i0 : -1; },
           [&](int) { return some; });
}

// The form of a product, with its rows to a tile and n to a workgroup.
//
// kStream16: one row to a group at most, and too few tiles for their loads in
// flight to cover the memory's latency (a streaming workgroup has 64 KiB in
// flight, a small tile's 24).  Weights of 8-bit values not in any cache, 8 rows
// of 64 groups, N = 2048, K = 4096 (256 tiles): 17.9 us, 21.9 with low tiles;
// 1 row, N = 4096, K = 2048: 10.1 and 12.6.  Twice the tiles: 20.5 and 18.7.
// 16 groups of about one row, 2048 x 2048: 22.5 and 19.0.  K = 512: 7.8 and 6.0.
//
// kLowTiles (32 x 64, two waves) against kSmallTiles, up to 16 rows to a group:
// half the rows' bytes and products beside the same weights.  72 rows of 9
// groups, 4096 x 2048: 22.9 us, 28.4 with small tiles; 16, 64, 128 and 192 rows
// of 16, 2048 x 2048: 19.0, 19.2, 19.1 and 19.4, small 20.7, 20.8, 20.2 and
// 20.3; 128 of 32, 1024 x 4096: 37.3 and 36.7.  512 of 9, 2048 x 4096: 36.8 and
// 35.0, as most groups then take two.
//
// kSmallTiles (64 x 64, two workgroups to a compute unit) against kWideTiles
// (128 x 256, half the bytes through LDS per product): the wide ones win where
// there are more of them than half the compute units and the groups fill them.
// G = 1, K = 4096, N = 4096, 2048 rows (256 wide tiles): 76.5 us against 119.3;
// 1024 rows (128): 122 at K = 8192 against 114; 8 groups of 1024 rows, 2048 x
// 2048: 105 against 128; 32 groups of 128, 2048 x 2048: 78 against 88; 32
// groups of 64: 215 against 210 (4096 x 4096).  At K = 128 they are equal, at K
// = 256 wide tiles take 309 us of 361 (16384 x 8192, 32-bit output).
enum MatmulForm { kStream16, kLowTiles, kSmallTiles, kWideTiles };

struct MatmulPlan {
  MatmulForm form;
  int rows, n;
};

// Tiles of R rows and N columns, every second group with one that is not full.
int64_t about_tiles(int64_t R, int64_t N, int32_t G, int rows, int n) {
  return (R / rows + G / 2) * ceil_div(N, n);
}

MatmulPlan plan_matmul(int64_t R, int64_t N, int64_t K, int32_t G) {
  if (R <= G && K >= 1024 && R * ceil_div(N, 64) <= 256) return {kStream16, 16, kStream16N};
  if (R <= 16 * (int64_t)G) return {kLowTiles, 32, 64};
  if (R >= 128 * (int64_t)G && K >= 256 && about_tiles(R, N, G, 128, 256) > 128) return {kWideTiles, 128, 256};
  return {kSmallTiles, 64, 64};
}

// The form of a weight gradient.
struct WgradPlan {
  bool large;
  int32_t ni, no;            // tiles along K and N
};

// Large tiles (128 x 256 against 64 x 64) take half the bytes through LDS per
// product, but there have to be enough of them: G = 8, 1024 x 1024 (256 large
// tiles), 4096 rows: 18.0 us against 26.0 (16-bit output); 8 groups of 8 rows,
// 32-bit output: 18.2 against 23.0; 700 x 600, G = 9 (162): 13.2 and 13.1; 2048
// x 2048, G = 1 (128): 39.3 and 38.8; 1024 x 1024, G = 1 (32), 8192 rows: 112
// and 45.
WgradPlan plan_wgrad(int64_t N, int64_t K, int32_t G) {
  const bool large = G * ceil_div(N, 128) * ceil_div(K, 256) >= 160;
  return {large, (int32_t)ceil_div(K, large ? 256 : 64), (int32_t)ceil_div(N, large ? 128 : 64)};
}

}  // namespace

int64_t matmul_tiles(int64_t R, int64_t N, int64_t K, int32_t G) {
  const MatmulPlan p = plan_matmul(R, N, K, G);
  // every group adds at most one tile that is not full, and a tile has a row
  return (std::min(R, R / p.rows + G) + 2) * ceil_div(N, p.n);
}

int64_t wgrad_tiles(int64_t N, int64_t K, int32_t G) {
  const WgradPlan p = plan_wgrad(N, K, G);
  return (int64_t)G * p.ni * p.no;
}

hipError_t launch_expert_matmul(const MatmulArgs& a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  const MatmulPlan p = plan_matmul(a.R, a.N, a.K, a.G);
  const dim3 grid((unsigned)matmul_tiles(a.R, a.N, a.K, a.G));
  const int32_t n_tiles = (int32_t)ceil_div(a.N, p.n);
  switch (p.form) {
    case kStream16:
      expert_stream16_kernel<<<grid, dim3(kStreamThreads), 0, stream>>>(a, n_tiles);
      break;
    case kLowTiles:
      expert_tile_kernel<2, 1, 1, 1, 4><<<grid, dim3(128), TileKernel<2, 1, 1, 1, 4, false>::kLdsBytes, stream>>>(
          a, n_tiles);
      break;
    case kSmallTiles:
      expert_tile_kernel<2, 2, 1, 1, 4><<<grid, dim3(256), TileKernel<2, 2, 1, 1, 4, false>::kLdsBytes, stream>>>(
          a, n_tiles);
      break;
    case kWideTiles:
      expert_tile_kernel<4, 2, 2, 2, 3><<<grid, dim3(512), TileKernel<4, 2, 2, 2, 3, false>::kLdsBytes, stream>>>(
          a, n_tiles);
      break;
  }
  return hipGetLastError();
}

hipError_t launch_expert_wgrad(const WgradArgs& a, hipStream_t stream) {
  const WgradPlan p = plan_wgrad(a.N, a.K, a.G);
  const dim3 grid((unsigned)wgrad_tiles(a.N, a.K, a.G));
  if (p.large)
    expert_wgrad_kernel<4, 2, 2, 2, 3><<<grid, dim3(512), TileKernel<4, 2, 2, 2, 3, true>::kLdsBytes, stream>>>(
        a, p.ni, p.no);
  else
    expert_wgrad_kernel<2, 2, 1, 1, 4><<<grid, dim3(256), TileKernel<2, 2, 1, 1, 4, true>::kLdsBytes, stream>>>(
        a, p.ni, p.no);
  return hipGetLastError();
}

}  // namespace eplb
