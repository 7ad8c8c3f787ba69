// The experts' products for few rows to a group: the weights are read once, from
// memory to registers, and bound the time.
//
// A workgroup of eight waves takes 16 MT rows of a group; KS waves share K, a run
// of chunks each in turn, and each of the 8 / KS sets of them has 16 outputs.  The
// rows pass through LDS, in two stages of 32 KiB that all waves share: read from
// memory by every wave for itself they would be several times the weights' bytes.
// The weights of D chunks are in flight at once, in registers, whatever the stages
// do, in whole cache lines: what a compute unit can have under way is the lines of
// its first-level cache, 32 KiB, however little of a line is wanted.  No load stands
// behind a branch: what lies past the end of a row, a group or the outputs has an
// offset outside its descriptor and arrives as zeros.
//
// Measured, launches back to back with the weights of many calls in rotation, so
// that none is in a cache: a token's 8 rows on 32 groups, 4096 x 2048: 23.2 us, 5.8
// TB/s (4-bit weights 13.4; traced among others 28.1 and 13.9); 512 uneven rows on
// 9, 2048 x 4096: 43 us (30); tiles of 128 x 128: 24.2 (28) and 46 (54).
//
// What is not there is multiplied all the same, as zeros: the sets of waves past a
// workgroup's outputs, the rows of a tile past its group's last, and the rounds of
// stages past the end of K (`kStages` at a time).
#pragma once

#include <cmath>

#include "tile16.h"

namespace eplb {

constexpr int kStreamWaves = 8;
constexpr int kStreamStage = 32 * 1024;    // bytes of rows in a stage

template <int DTYPE>
__device__ __forceinline__ void store_four(void* p, int64_t at, int left, bool vec, f32x4 v) {
  if (vec && left >= 4) {
    if (DTYPE == kF32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = v;
    } else {
      u16 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = DTYPE == kBf16 ? float_to_bf16(v[j]) : float_to_f16(v[j]);
      *reinterpret_cast<uint2*>(static_cast<u16*>(p) + at) =
          uint2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < left) store_float(p, DTYPE, at + j, v[j]);
}

template <bool FOUR, int MT, int KS>
struct StreamShape {
  static constexpr int kRows = 16 * MT;
  static constexpr int kChunk = FOUR ? 256 : 64;                   // k of a chunk: 128 bytes of each row of weights
  static constexpr int kStageK = kStreamStage / (kRows * 2);       // k of a stage
  static constexpr int kEach = kStageK / (kChunk * KS);            // chunks of a wave in a stage
};

// What a lane holds of a chunk's weights: with 16-bit ones two instructions' operands; with 4-bit ones twice four
// instructions', a block of 32 of k each.
struct StreamChunk {
  i32x4 w[2];
};

// Lane 16 q + c holds M[q][s] in element s: from now on M[s][q].
__device__ __forceinline__ void turn_quads(i32x4& v) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const auto p = __builtin_amdgcn_permlane32_swap((uint32_t)v[s], (uint32_t)v[s + 2], false, false);
    v[s] = (int)p[0];
    v[s + 2] = (int)p[1];
  }
#pragma unroll
  for (int s = 0; s < 4; s += 2) {
    const auto p = __builtin_amdgcn_permlane16_swap((uint32_t)v[s], (uint32_t)v[s + 1], false, false);
    v[s] = (int)p[0];
    v[s + 1] = (int)p[1];
  }
}

// `each` sets of 16 outputs to a workgroup, `columns` workgroups to a row of tiles
template <Mode MODE, bool FOUR, int MT, int KS, int D>
__global__ __launch_bounds__(kStreamWaves * 64, 4) void linear_stream_kernel(Linear16Args a, int32_t columns, int32_t each) {
  typedef StreamShape<FOUR, MT, KS> Shape;
  constexpr int kBlockBytes = Shape::kRows * 128, kOctets = Shape::kRows / 8;
  constexpr int kXLoads = kStreamStage / 1024 / kStreamWaves;      // of a wave and stage
  constexpr int kWLoads = 2;                                       // of a chunk
  constexpr int kBatch = 4;                                        // chunks whose scales are asked for together
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStreamStage];
  __shared__ int32_t src[Shape::kRows];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, col = lane & 15, share = wave % KS, set = wave / KS;
  const int n0 = ((int)(blockIdx.x % columns) * each + set) * 16;
  const Tile t = find_tile(a.offsets, a.G, a.R, Shape::kRows, (int32_t)(blockIdx.x / columns), true);
  if (t.g < 0) return;
  const bool some = t.g < a.G && a.X > 0;
  const int outputs = set < each ? max(min(a.N - n0, 16), 0) : 0;
  const int64_t first = some && outputs > 0 ? (int64_t)t.g * a.N + n0 : 0;
  const int rows = some ? outputs : 0;
  const uint32_t ld = FOUR ? a.C / 2 : a.C * 2, ld_s = a.C / kScaleGroup;
  const i32x4 from_w = FOUR ? describe(a.q + first * ld, (uint64_t)rows * ld)
                            : describe(static_cast<const uint8_t*>(a.w) + first * ld, (uint64_t)rows * ld);
  const i32x4 from_s = FOUR ? describe(a.scale + first * ld_s, (uint64_t)rows * ld_s) : from_w;
  // Where a part of 16 bytes lies in a row's 128.  Quads 0 and 1, 2 and 3 read together, without conflicts where their parts
  // are 1 apart: parts that are 4 apart, as with 4-bit values (which are 32 of k to a lane), become neighbours.
  constexpr bool kFours = FOUR && MODE != kScaled;
  auto place_of = [](int part) { return kFours ? (part & 3) << 1 | part >> 2 : part; };
  auto part_at = [](int place) { return kFours ? (place & 1) << 2 | place >> 1 : place; };
  const uint32_t at_w = col * ld + quad * 16, at_s = col * ld_s + quad;
  auto load_w = [&](int c, StreamChunk& p) {
    const int k = c * Shape::kChunk + quad * (FOUR ? 32 : 8);      // this lane's first; half a chunk on its second
#pragma unroll
    for (int s = 0; s < 2; ++s)
      p.w[s] = __builtin_amdgcn_raw_buffer_load_b128(
          resource(from_w), (at_w + s * 64) | (k + s * (Shape::kChunk / 2) < a.C ? 0 : kOutside), c * 128, 0);
  };
  // This wave's chunk i.  A stage's are shared out in runs, so that what lies next to each other is asked for together.
  // Rows of weights are often a power of two apart, and then their chunks of one place all lie in one channel of a die's
  // cache: each workgroup of a die (every eighth) starts with another stage, and each set of waves with another chunk of
  // its run.
  const int stages = (a.C - 1) / Shape::kStageK + 1, turn = (int)((blockIdx.x >> 3) % stages),
            chunk_turn = set + (int)((blockIdx.x >> 3) / stages % Shape::kEach);
  auto stage_of = [&](int stage) { return stage >= stages ? stages : stage + turn < stages ? stage + turn : stage + turn - stages; };
  auto chunk = [&](int i) {
    return (stage_of(i / Shape::kEach) * KS + share) * Shape::kEach + (i + chunk_turn) % Shape::kEach;
  };
  // What rows names is asked for first, and the weights before it is looked at: loads return in order.
  static_assert(Shape::kRows <= kStreamWaves * 64, "a thread to a row");
  const int mine = threadIdx.x;
  int32_t named = t.row + mine;
  if (a.rows != nullptr && mine < t.rows) named = a.rows[t.row + mine];
  // scales of chunks i .. i + 3, a byte to a lane and half a chunk
  uint32_t scale[2][kBatch][2];
  auto load_s = [&](int i, uint32_t (&to)[kBatch][2]) {
    if constexpr (FOUR) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int c = chunk(i + j), k = c * Shape::kChunk + s * 128 + quad * 32;
          to[j][s] = __builtin_amdgcn_raw_buffer_load_b8(resource(from_s), (at_s + s * 4) | (k < a.C ? 0 : kOutside), c * 8, 0);
        }
    }
  };
  StreamChunk part[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load_w(chunk(d), part[d]);
  load_s(0, scale[0]);
  __builtin_amdgcn_sched_barrier(0);
  if (mine < Shape::kRows) {
    if (a.rows != nullptr) named = named < 0 ? -1 : (int32_t)fastdiv_apply((uint32_t)named, a.fd_topk);
    src[mine] = mine < t.rows && t.g < a.G && named < a.X ? named : -1;
  }
  // a barrier that does not wait for the weights
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  f32x4 acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (some) {
    const i32x4 from_x = describe(a.x, (uint64_t)a.X * a.ld * 2);
    uint32_t at_x[kXLoads];
    int part_x[kXLoads];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int r = (wave * kXLoads + i) % kOctets * 8 + (lane >> 3);
      part_x[i] = part_at((lane & 7) ^ along_key(r)) * 8;
      at_x[i] = src[r] < 0 ? kOutside : (uint32_t)src[r] * (uint32_t)a.ld * 2 + part_x[i] * 2;
    }
    const uint32_t lds_at = lds_address(lds);
    auto load_x = [&](int stage) {
#pragma unroll
      for (int i = 0; i < kXLoads; ++i) {
        const int j = wave * kXLoads + i, block = stage_of(stage) * (Shape::kStageK / kTileK) + j / kOctets;
        part_to_lds(from_x, at_x[i] | (part_x[i] < a.C - block * kTileK ? 0 : kOutside), block * 128,
                    lds_at + (stage & 1) * kStreamStage + j * 1024);
      }
    };
    // until all loads but the last `n` of every wave are there, and all waves are here
    auto wait = [](auto n) {
      constexpr int kLeft = decltype(n)::value < 63 ? decltype(n)::value : 63;
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
    };
    load_x(0);
    load_x(1);
    constexpr int kLeast = FOUR ? 2 * kBatch : D, kMost = D > Shape::kEach ? D : Shape::kEach;
    constexpr int kUnroll = kMost > kLeast ? kMost : kLeast, kStages = kUnroll / Shape::kEach;
    static_assert(kUnroll % D == 0 && kUnroll % Shape::kEach == 0, "whole stages and whole rounds of chunks");
    for (int st = 0; st < stages; st += kStages) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int stage = st + u / Shape::kEach, i = st * Shape::kEach + u;
        if (u % Shape::kEach == 0) {
          // this stage's rows have arrived (after them: the next one's, or a stage's weights), and all waves are done with
          // the one before, whose place the one after this takes
          if (stage == 0) {
            wait(std::integral_constant<int, kXLoads>());
          } else {
            wait(std::integral_constant<int, Shape::kEach * kWLoads>());
            load_x(stage + 1);
          }
        }
        const uint8_t* rows_at = lds + (stage & 1) * kStreamStage;
        const int c_in = share * Shape::kEach + (i + chunk_turn) % Shape::kEach;    // its place in the stage
        if (FOUR && u % kBatch == 0) load_s(i + kBatch, scale[u / kBatch + 1 & 1]);
        auto rows_of = [&](int m, int at) {       // eight of k, part `at` of the chunk, of row `col` of tile m
          const int block = c_in * (Shape::kChunk / kTileK) + (at >> 3), r = m * 16 + col;
          return *reinterpret_cast<const i32x4*>(rows_at + block * kBlockBytes + r * 128 + ((place_of(at & 7) ^ along_key(r)) << 4));
        };
        if constexpr (MODE == kScaled) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // An instruction's k has to be one block of 32: quad s has block s, and register q becomes part of quad q.
            i32x4 w = part[u % D].w[h], scales;
            turn_quads(w);
            const int mine = (int)scale_bits(scale[u / kBatch & 1][u % kBatch][h]);
            scales = i32x4{mine, mine, mine, mine};
            turn_quads(scales);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const i32x4 values = four_bit_halves(w[s]);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                // the rows first: a lane's sums are of one output then, and have one scale
                const f32x4 products =
                    multiply_f16(rows_of(m, h * 16 + s * 4 + quad), values, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = fmaf(__int_as_float(scales[s]), products[j], acc[m][j]);
              }
            }
          }
        } else {
#pragma unroll
          for (int s = 0; s < (FOUR ? 8 : 2); ++s) {
            i32x4 w = part[u % D].w[FOUR ? s >> 2 : s];
            if constexpr (FOUR)
              w = four_bit_values(w[s & 3], __uint_as_float(scale[u / kBatch & 1][u % kBatch][s >> 2] << 23));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              // which eight of the chunk's k the weights are of
              const i32x4 x = rows_of(m, FOUR ? (s >> 2) * 16 + quad * 4 + (s & 3) : s * 4 + quad);
              acc[m] = MODE == kBothF16 ? multiply_f16(w, x, acc[m]) : multiply_bf16(w, x, acc[m]);
            }
          }
        }
        load_w(chunk(i + D), part[u % D]);                           // past the last chunk: nothing is read
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");      // LDS is free
  }
  if constexpr (KS > 1) {
    // the shares of K, added up in order
    f32x4(*sums)[MT][64] = reinterpret_cast<f32x4(*)[MT][64]>(lds);
    static_assert(kStreamWaves * MT * 1024 <= 2 * kStreamStage, "sums fit");
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[wave][m][lane] = acc[m];
    __syncthreads();
    if (share != 0) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 1; s < KS; ++s) acc[m] += sums[wave + s][m][lane];
  }
  auto store = [&](auto type) {
    constexpr int kType = decltype(type)::value;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (MODE == kScaled) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = m * 16 + quad * 4 + j;
          if (r < t.rows && col < outputs)
            store_float(a.y, kType, (int64_t)(t.row + r) * a.N + n0 + col, src[r] >= 0 ? acc[m][j] : 0.0f);
        }
      } else {
        const int r = m * 16 + col;
        if (r < t.rows)
          store_four<kType>(a.y, (int64_t)(t.row + r) * a.N + n0 + quad * 4, outputs - quad * 4, a.N % 4 == 0,
                            src[r] >= 0 ? acc[m] : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
      }
    }
  };
  if (a.y_dtype == kF32) store(std::integral_constant<int, kF32>());
  else if (a.y_dtype == kBf16) store(std::integral_constant<int, kBf16>());
  else store(std::integral_constant<int, kF16>());
}

// How a product of few rows is taken: tiles of 16 mt rows, `share` waves to 16 outputs, `each` such to a workgroup.
struct StreamPlan {
  int mt, share, each;
};

// Tiles of `tile` rows: every group adds at most one that is not full, and a tile has a row.
inline int64_t row_tiles(int64_t R, int32_t G, int tile) { return std::min(R, R / tile + G) + 2; }

// Few rows.  Uneven groups (the largest has one and a half times the mean on 9, three times on 32 and 64), here and in
// tiles, us, at 47, 64, 71, 80 and 95 rows to a group.  16-bit weights:
//   2048 x 4096 on 9   39 43 43 45 49 | 45 46 47 47 48      4096 x 2048 on 9   40 44 44 45 50 | 50 51 51 52 51
//   1024 x 2048 on 32  49 56 53 58 62 | 49 49 48 50 48      on 64              62 79 78 88 97 | 64 72 73 73 72
// 4-bit weights:
//   2048 x 4096 on 9   29 31 39 44 44 | 53 55 55 55 55      4096 x 2048 on 9   28 31 39 40 42 | 39 39 39 40 40
//   1024 x 2048 on 32  36 39 31 31 40 | 31 39 39 39 39      on 64              51 54 61 57 67 | 40 64 65 64 70
// One limit for both: no mean tells all of these apart.  What it costs most: 4-bit weights of long rows on few groups, a
// third just past it.
inline bool stream_suits(int64_t R, int32_t G) { return R <= 64 * (int64_t)G; }

// The busiest compute unit ends last, and what it can have in flight is the same whatever is on it: the form is the one
// for which ceil(workgroups / compute units) times what a workgroup costs, its sets of outputs and its start and end, is
// least.  512 rows on 9, 2048 outputs, K 4096, 5 sets to a workgroup: 37 us in tiles of 64 rows and 42 in those of 128
// where every group has 57 rows; where groups have up to 84, some two tiles of 64, 61 and 43.
inline StreamPlan plan_stream(int64_t R, int64_t N, int32_t G, bool four) {
  constexpr int kUnits = 256;
  // rows to a group: as chance deals them out, and a fifth of the mean besides, which a balanced placement leaves
  const double mean = (double)R / G, spread = std::sqrt(mean + 0.04 * mean * mean);
  StreamPlan best{};
  double least = 0;
  for (int mt = 1; mt <= (four ? 4 : 8); mt *= 2) {
    // what an output of a tile costs, against one of a tile of 16 rows: the weights are the same, but more is multiplied
    const double weight = four ? (mt == 1 ? 1 : mt == 2 ? 1.15 : 1.6) : (mt == 1 ? 1 : mt == 2 ? 1.02 : mt == 4 ? 1.06 : 1.25);
    double tiles = G, more_of_them = 0;    // and how many groups have another one; what chance may add
    for (int t = 1; t <= 64 && 16 * mt * t < mean + 3 * spread; ++t) {
      const double more = 0.5 * std::erfc((16 * mt * t - mean) / (spread * std::sqrt(2.0)));
      tiles += G * more;
      more_of_them += std::sqrt(G * more * (1 - more));
    }
    for (int each = 1; each <= kStreamWaves; ++each) {
      auto turns = [&](double t) { return std::ceil(std::min((double)R, t) * ceil_div(N, 16 * each) / kUnits); };
      const double cost = (weight * each + 1 + 0.25 * mt) * (turns(tiles) + turns(tiles + more_of_them));
      if (best.mt == 0 || cost < least || (cost == least && mt == best.mt)) {
        least = cost;
        best = StreamPlan{mt, 1, each};
      }
    }
  }
  const int most = four ? 4 / best.mt : 16 / best.mt;    // every wave has a chunk in every stage
  while (best.share * 2 * best.each <= kStreamWaves && best.share * 2 <= most) best.share *= 2;
  return best;
}

inline int64_t stream_blocks(int64_t R, int64_t N, int32_t G, bool four) {
  const StreamPlan p = plan_stream(R, N, G, four);
  return row_tiles(R, G, 16 * p.mt) * ceil_div(N, 16 * p.each);
}

template <Mode MODE, bool FOUR, int MT, int KS, int D>
hipError_t launch_stream(const Linear16Args& a, int32_t each, hipStream_t stream) {
  const int64_t columns = ceil_div(a.N, 16 * each);
  linear_stream_kernel<MODE, FOUR, MT, KS, D>
      <<<dim3((unsigned)(row_tiles(a.R, a.G, 16 * MT) * columns)), dim3(kStreamWaves * 64), 0, stream>>>(a, (int32_t)columns, each);
  return hipGetLastError();
}

template <Mode MODE, bool FOUR, int MT>
hipError_t launch_stream(const Linear16Args& a, const StreamPlan& p, hipStream_t stream) {
  // chunks in flight.  16-bit weights, 2 and 4: 43 and 37 us (252 rows on 9, 2048 x 4096), 55 and 45 (512 rows); 4-bit
  // weights (a chunk is four times the k): 13.8 and 14.3 (a token's 8 rows, 4096 x 2048), but 24.1 and 23.2 (252 rows)
  constexpr int kAhead = FOUR && MT == 1 ? 2 : 4, kMost = FOUR ? 4 / MT : 16 / MT;
  if constexpr (kMost >= 8)
    if (p.share == 8) return launch_stream<MODE, FOUR, MT, 8, kAhead>(a, p.each, stream);
  if constexpr (kMost >= 4)
    if (p.share == 4) return launch_stream<MODE, FOUR, MT, 4, kAhead>(a, p.each, stream);
  if constexpr (kMost >= 2)
    if (p.share == 2) return launch_stream<MODE, FOUR, MT, 2, kAhead>(a, p.each, stream);
  return launch_stream<MODE, FOUR, MT, 1, kAhead>(a, p.each, stream);
}

template <Mode MODE, bool FOUR>
hipError_t launch_stream(const Linear16Args& a, hipStream_t stream) {
  const StreamPlan p = plan_stream(a.R, a.N, a.G, FOUR);
  if constexpr (!FOUR)
    if (p.mt == 8) return launch_stream<MODE, FOUR, 8>(a, p, stream);
  return p.mt == 1 ? launch_stream<MODE, FOUR, 1>(a, p, stream)
                   : p.mt == 2 ? launch_stream<MODE, FOUR, 2>(a, p, stream) : launch_stream<MODE, FOUR, 4>(a, p, stream);
}

}  // namespace eplb
