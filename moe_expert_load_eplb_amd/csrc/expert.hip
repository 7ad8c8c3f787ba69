// The experts' products in 8-bit floating point with a scale for each block
// of 128.
//
// Both products have the same shape: out[o][i] = sum over blocks b of 128 of
// so[o][b] * si[i][b] * (sum over j in b of O[o][j] * I[i][j]), with the
// inner index i contiguous in the output (matmul: o = row, i = n, j = k;
// weight gradient: o = n, i = k, j = row).  One matrix instruction takes a
// 16 x 16 tile through a whole block (128 products per element), so its
// result is what the block's scales multiply; the sum over blocks is kept in
// 32-bit registers.  The inner operand is the instruction's first, which
// leaves four consecutive i of one o in each lane.
#include "experts_device.h"

namespace eplb {

namespace {

constexpr int kTile = 128;                   // rows of each operand per workgroup
constexpr int kMmThreads = 256;              // four waves, 64 x 64 of the tile each

// Whether the matrix cores' rate bounds a product, rather than its bytes or
// the launch: then 16-bit outputs come from the 8-bit matrix instruction.
// out rows x in columns over a contraction of `inner`, and the bytes of its
// operands and output.
bool matrix_bound(double out, double in, double inner, double bytes) {
  const double ops = 2.0 * out * in * inner;
  return ops >= 0x1p34 && ops >= 256.0 * bytes;
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 16 x 16 sums over a block of 128.  The 8-bit matrix instruction adds its
// products with less than 32 bits (measured: 5e-5 of a typical sum of values
// spread over the format's whole range, 1.6e-5 of normally distributed ones),
// far below the rounding of a 16-bit output.  For 32-bit outputs the values
// become 16-bit ones, exactly, and go through the 16-bit matrix instruction,
// whose sums keep 32 bits (measured: 7e-8), at half the rate or less.
template <bool WIDE>
struct Fragment;

template <>
struct Fragment<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) {
    v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

template <>
struct Fragment<true> {
  f16x8 v[4];
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int a = s < 2 ? lo[2 * s] : hi[2 * s - 4], b = s < 2 ? lo[2 * s + 1] : hi[2 * s - 3];
      const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
      const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
      const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
      const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
      v[s] = f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
  }
};

__device__ __forceinline__ f32x4 mfma_block(const Fragment<false>& a, const Fragment<false>& b) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mfma_block(const Fragment<true>& a, const Fragment<true>& b) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[s], b.v[s], d, 0, 0, 0);
  return d;
}

// 16 bytes `c` of row `r` of a staged tile: rows of 128 bytes, their 16-byte
// parts permuted by the row so that 8 rows at one c cover all banks.
__device__ __forceinline__ int lds_at(int r, int c) { return r * kBlock + ((c ^ (r & 7)) << 4); }

template <bool WIDE>
__device__ __forceinline__ Fragment<WIDE> fragment(const uint8_t* tile, int row, int quad) {
  Fragment<WIDE> f;
  f.set(*reinterpret_cast<const i32x4*>(tile + lds_at(row, quad)),
        *reinterpret_cast<const i32x4*>(tile + lds_at(row, quad + 4)));
  return f;
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
// Streaming forms, for groups of few rows: the weights are read once, from
// memory to registers, and bound the time.  A wave takes 16 n of one group
// through K; the fragments of several blocks of 128 are in flight at once
// (2 KiB each).  With the memory as the bound, 16-bit products cost nothing
// and keep 32-bit sums.  No load stands behind a branch (rows and blocks past
// the end are clamped to the last ones and not used): a load that may or may
// not have been issued makes every wait behind it wait for all of them.
constexpr int kStreamThreads = 256;
constexpr int kStream16N = 64;               // n of a workgroup: 16 of each wave
constexpr int kStreamN = 32;                 // n of a workgroup, of each wave

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

// 16 rows: both operands go straight to registers.
constexpr int kAhead16 = 8;

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
        Fragment<true> fw, fx;
        fw.set(rw[p][0], rw[p][1]);
        fx.set(k < a.K ? rx[p][0] : zero, k + 64 < a.K ? rx[p][1] : zero);
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

// Up to 96 rows of one group against 32 n: the workgroup's four waves take
// every fourth block of K each, all operands straight from memory (the rows,
// read by every workgroup of the group, from the caches), and add their sums
// in LDS at the end, in order.  Without a barrier in the loop the waves run
// free; a tile's next rows are loaded as soon as its last ones are used.
constexpr int kStreamSplit = kStreamThreads / 64;          // waves that share a tile's K

// The loop for NT tiles of 16 rows (all of them present).
template <int NT>
__device__ __forceinline__ void stream_tiles(const MatmulArgs& a, const Tile& t, int n0, int wave, f32x4* sums) {
  constexpr int kAheadW = 2;                 // blocks of the weights in flight
  const int lane = threadIdx.x & 63, quad = lane >> 4, col = lane & 15;
  f32x4 acc[NT][2];
#pragma unroll
  for (int o = 0; o < NT; ++o) acc[o][0] = acc[o][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint8_t* w[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) w[u] = a.w + ((int64_t)t.g * a.N + min(n0 + u * 16 + col, a.N - 1)) * a.K;
  i32x4 rw[kAheadW][2][2], rx[NT][2];
  float sx[NT];
  auto block = [&](int b) { return min(b * kStreamSplit + wave, a.KB - 1); };
  auto load_w = [&](int slot, int b) {
#pragma unroll
    for (int u = 0; u < 2; ++u) load_parts(w[u], block(b), quad, a.K, rw[slot][u][0], rw[slot][u][1]);
  };
  int32_t from[NT];
#pragma unroll
  for (int o = 0; o < NT; ++o) from[o] = o * 16 + col < t.rows ? source_row(a, t.row + o * 16 + col) : -1;
  ScaleRow ws(a.w_scale + ((int64_t)t.g * a.NB + n0 / kBlock) * a.KB, a.KB);
  load_w(0, 0);
  auto load_x = [&](int o, int b) {
    const int64_t row = max(from[o], 0);
    load_parts(a.q + row * a.K, block(b), quad, a.K, rx[o][0], rx[o][1]);
    sx[o] = a.scale[row * a.KB + block(b)];
  };
#pragma unroll
  for (int o = 0; o < NT; ++o) load_x(o, 0);
#pragma unroll
  for (int p = 1; p < kAheadW; ++p) load_w(p, p);
  const int steps = (a.KB + kStreamSplit - 1) / kStreamSplit;
  for (int b0 = 0; b0 < steps; b0 += kAheadW) {
    ws.load_next((b0 + kAheadW) * kStreamSplit);
#pragma unroll
    for (int p = 0; p < kAheadW; ++p) {
      const int b = b0 + p, kb = b * kStreamSplit + wave;
      const i32x4 zero = {0, 0, 0, 0};
      const bool lo = kb * kBlock + quad * 16 < a.K, hi = kb * kBlock + quad * 16 + 64 < a.K;
      const bool in = kb < a.KB;             // past the end: not added
      const float wk = ws.get(p * kStreamSplit + wave);
      Fragment<true> fw[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) fw[u].set(rw[p][u][0], rw[p][u][1]);
#pragma unroll
      for (int o = 0; o < NT; ++o) {
        Fragment<true> fx;
        fx.set(lo ? rx[o][0] : zero, hi ? rx[o][1] : zero);
        const float sc = sx[o] * wk;
        load_x(o, b + 1);
        f32x4 d[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int u = 0; u < 2; ++u) d[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fw[u].v[c], fx.v[c], d[u], 0, 0, 0);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[o][u][j] = in ? acc[o][u][j] + d[u][j] * sc : acc[o][u][j];
      }
      load_w(p, b + kAheadW);                // behind the rows' loads: loads return in order
    }
    ws.advance();
  }
#pragma unroll
  for (int o = 0; o < NT; ++o)
#pragma unroll
    for (int u = 0; u < 2; ++u) sums[(o * 2 + u) * 64 + lane] = from[o] >= 0 ? acc[o][u] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

__global__ __launch_bounds__(kStreamThreads, 2) void expert_stream_kernel(MatmulArgs a, int32_t n_tiles, int32_t rows) {
  extern __shared__ __attribute__((aligned(16))) f32x4 sums[];   // [wave][rows / 16][2][64]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)(blockIdx.x % n_tiles) * kStreamN;
  const Tile t = find_tile(a.offsets, a.G, a.R, rows, (int32_t)(blockIdx.x / n_tiles), true);
  if (t.g < 0) return;
  const bool some = t.g < a.G && a.X > 0;
  const int tiles = (t.rows + 15) >> 4, each = rows * 8;
  if (some) {
    // a loop of its own for every number of tiles: no load behind a branch
    f32x4* mine = sums + wave * each;
    switch (tiles) {
      case 1: stream_tiles<1>(a, t, n0, wave, mine); break;
      case 2: stream_tiles<2>(a, t, n0, wave, mine); break;
      case 3: stream_tiles<3>(a, t, n0, wave, mine); break;
      case 4: stream_tiles<4>(a, t, n0, wave, mine); break;
      case 5: stream_tiles<5>(a, t, n0, wave, mine); break;
      default: stream_tiles<6>(a, t, n0, wave, mine); break;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tiles * 128; i += kStreamThreads) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (some) {
#pragma unroll
      for (int k = 0; k < kStreamSplit; ++k) v += sums[k * each + i];
    }
    const int r = (i >> 7) * 16 + (i & 15), n = n0 + (i >> 6 & 1) * 16 + (i >> 4 & 3) * 4;
    if (r < t.rows && n < a.N) store4(a.y, a.dtype, (int64_t)(t.row + r) * a.N + n, a.N - n, a.N % 4 == 0, v);
  }
}

// ---------------------------------------------------------------- tiles
template <bool WIDE>
__global__ __launch_bounds__(kMmThreads) void expert_matmul_kernel(MatmulArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t wt[kTile * kBlock];
  __shared__ __attribute__((aligned(16))) uint8_t xt[kTile * kBlock];
  __shared__ int32_t src[kTile];
  const int nb = (int)(blockIdx.x % a.NB);
  const Tile t = find_tile(a.offsets, a.G, a.R, kTile, (int32_t)(blockIdx.x / a.NB), true);
  if (t.g < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int quad = lane >> 4, col = lane & 15;
  const int wi = (wave & 1) * 64, wo = (wave >> 1) * 64;
  if (tid < kTile) {
    int32_t from = -1;
    if (tid < t.rows && t.g < a.G) {
      from = t.row + tid;
      if (a.rows != nullptr) {
        from = a.rows[from];
        from = from < 0 ? -1 : (int32_t)fastdiv_apply((uint32_t)from, a.fd_topk);
      }
      if (from >= a.X) from = -1;
    }
    src[tid] = from;
  }
  __syncthreads();
  f32x4 acc[4][4];
#pragma unroll
  for (int o = 0; o < 4; ++o)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[o][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (t.g < a.G) {
    const uint8_t* w = a.w + (int64_t)t.g * a.N * a.K;
    const float* ws = a.w_scale + ((int64_t)t.g * a.NB + nb) * a.KB;
    int32_t from[4];
#pragma unroll
    for (int o = 0; o < 4; ++o) from[o] = src[wo + o * 16 + col];
    for (int kb = 0; kb < a.KB; ++kb) {
      i32x4 rw[4], rx[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = (tid + p * kMmThreads) >> 3, c = tid & 7;
        const int64_t k = (int64_t)kb * kBlock + c * 16;
        const int n = nb * kTile + r;
        rw[p] = rx[p] = i32x4{0, 0, 0, 0};
        if (n < a.N && k < a.K) rw[p] = *reinterpret_cast<const i32x4*>(w + (int64_t)n * a.K + k);
        if (src[r] >= 0 && k < a.K) rx[p] = *reinterpret_cast<const i32x4*>(a.q + (int64_t)src[r] * a.K + k);
      }
      float sc[4];
#pragma unroll
      for (int o = 0; o < 4; ++o) sc[o] = from[o] >= 0 ? ws[kb] * a.scale[(int64_t)from[o] * a.KB + kb] : 0.0f;
      __syncthreads();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = (tid + p * kMmThreads) >> 3, c = tid & 7;
        *reinterpret_cast<i32x4*>(wt + lds_at(r, c)) = rw[p];
        *reinterpret_cast<i32x4*>(xt + lds_at(r, c)) = rx[p];
      }
      __syncthreads();
      Fragment<WIDE> fi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fi[i] = fragment<WIDE>(wt, wi + i * 16 + col, quad);
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const Fragment<WIDE> fo = fragment<WIDE>(xt, wo + o * 16 + col, quad);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 d = mfma_block(fi[i], fo);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[o][i][j] += d[j] * sc[o];
        }
      }
    }
  }
  const bool vec = a.N % 4 == 0;
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const int ro = wo + o * 16 + col;
    if (ro >= t.rows) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = nb * kTile + wi + i * 16 + quad * 4;
      store4(a.y, a.dtype, (int64_t)(t.row + ro) * a.N + n, a.N - n, vec, acc[o][i]);
    }
  }
}

template <bool WIDE>
__global__ __launch_bounds__(kMmThreads) void expert_wgrad_kernel(WgradArgs a, int32_t ni, int32_t no) {
  __shared__ __attribute__((aligned(16))) uint8_t it[kTile * kBlock];
  __shared__ __attribute__((aligned(16))) uint8_t ot[kTile * kBlock];
  const int g = (int)(blockIdx.x / (ni * no));
  const int bo = (int)(blockIdx.x / ni % no), bi = (int)(blockIdx.x % ni);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int quad = lane >> 4, col = lane & 15;
  const int wi = (wave & 1) * 64, wo = (wave >> 1) * 64;
  // the group's blocks of 128 rows
  int64_t b0 = 0, b1 = 0;
  for (int h = 0; h <= g; ++h) {
    const int32_t lo = clamp_row(a.offsets[h], a.R), hi = clamp_row(a.offsets[h + 1], a.R);
    b0 = b1;
    b1 += hi > lo ? ((int64_t)hi - lo + kBlock - 1) / kBlock : 0;
  }
  if (b1 > a.Rp / kBlock) b1 = a.Rp / kBlock;
  f32x4 acc[4][4];
#pragma unroll
  for (int o = 0; o < 4; ++o)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[o][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t b = b0; b < b1; ++b) {
    i32x4 ri[4], ro[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = (tid + p * kMmThreads) >> 3, c = tid & 7;
      const int64_t i = (int64_t)bi * kTile + r, o = (int64_t)bo * kTile + r;
      ri[p] = ro[p] = i32x4{0, 0, 0, 0};
      if (i < a.K) ri[p] = *reinterpret_cast<const i32x4*>(a.x + i * a.Rp + b * kBlock + c * 16);
      if (o < a.N) ro[p] = *reinterpret_cast<const i32x4*>(a.dy + o * a.Rp + b * kBlock + c * 16);
    }
    float so[4];
    f32x4 si[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t o = (int64_t)bo * kTile + wo + t * 16 + col;
      so[t] = o < a.N ? a.dy_scale[b * a.N + o] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = (int64_t)bi * kTile + wi + t * 16 + quad * 4 + j;
        si[t][j] = i < a.K ? a.x_scale[b * a.K + i] : 0.0f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = (tid + p * kMmThreads) >> 3, c = tid & 7;
      *reinterpret_cast<i32x4*>(it + lds_at(r, c)) = ri[p];
      *reinterpret_cast<i32x4*>(ot + lds_at(r, c)) = ro[p];
    }
    __syncthreads();
    Fragment<WIDE> fi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) fi[i] = fragment<WIDE>(it, wi + i * 16 + col, quad);
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      const Fragment<WIDE> fo = fragment<WIDE>(ot, wo + o * 16 + col, quad);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 d = mfma_block(fi[i], fo);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[o][i][j] += d[j] * (so[o] * si[i][j]);
      }
    }
  }
  const bool vec = a.K % 4 == 0;
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const int64_t n = (int64_t)bo * kTile + wo + o * 16 + col;
    if (n >= a.N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = (int64_t)bi * kTile + wi + i * 16 + quad * 4;
      const int64_t left = a.K - k;
      store4(a.dw, a.dtype, ((int64_t)g * a.N + n) * a.K + k, left < 4 ? (int)left : 4, vec, acc[o][i]);
    }
  }
}

// The form of a product: rows to a tile and n to a workgroup.
enum MatmulForm { kStream16, kStream, kTiles };

struct MatmulPlan {
  MatmulForm form;
  int rows, n;
};

MatmulPlan plan_matmul(int64_t R, int32_t G) {
  const int64_t average = ceil_div(R, G);
  if (average <= 8) return {kStream16, 16, kStream16N};
  // room for groups half as large again as the average, so that few need a second tile
  if (average <= 64) return {kStream, average <= 42 ? 64 : 96, kStreamN};
  return {kTiles, kTile, kTile};
}

}  // namespace

int64_t matmul_tiles(int64_t R, int64_t N, int32_t G) {
  const MatmulPlan p = plan_matmul(R, G);
  // every group adds at most one tile that is not full, and a tile has a row
  return (std::min(R, R / p.rows + G) + 2) * ceil_div(N, p.n);
}

int64_t wgrad_tiles(int64_t N, int64_t K, int32_t G) { return G * ceil_div(N, kTile) * ceil_div(K, kTile); }

hipError_t launch_expert_matmul(const MatmulArgs& args, hipStream_t stream) {
  if (args.R == 0) return hipSuccess;
  MatmulArgs a = args;
  a.large = matrix_bound(a.R, a.N, a.K, (double)a.R * a.K + (double)a.G * a.N * a.K + 2.0 * a.R * a.N);
  const MatmulPlan p = plan_matmul(a.R, a.G);
  const dim3 grid((unsigned)matmul_tiles(a.R, a.N, a.G));
  const int32_t n_tiles = (int32_t)ceil_div(a.N, p.n);
  switch (p.form) {
    case kStream16:
      expert_stream16_kernel<<<grid, dim3(kStreamThreads), 0, stream>>>(a, n_tiles);
      break;
    case kStream:
      expert_stream_kernel<<<grid, dim3(kStreamThreads), (size_t)kStreamSplit * p.rows * 8 * 16, stream>>>(a, n_tiles, p.rows);
      break;
    case kTiles:
      if (a.dtype == kF32 || !a.large) expert_matmul_kernel<true><<<grid, dim3(kMmThreads), 0, stream>>>(a);
      else expert_matmul_kernel<false><<<grid, dim3(kMmThreads), 0, stream>>>(a);
      break;
  }
  return hipGetLastError();
}

hipError_t launch_expert_wgrad(const WgradArgs& a, hipStream_t stream) {
  const int32_t ni = (int32_t)ceil_div(a.K, kTile), no = (int32_t)ceil_div(a.N, kTile);
  const dim3 grid((unsigned)wgrad_tiles(a.N, a.K, a.G));
  const bool large = matrix_bound(a.N, a.K, a.R, (double)a.R * (a.N + a.K) + 2.0 * a.G * a.N * a.K);
  if (a.dtype == kF32 || !large) expert_wgrad_kernel<true><<<grid, dim3(kMmThreads), 0, stream>>>(a, ni, no);
  else expert_wgrad_kernel<false><<<grid, dim3(kMmThreads), 0, stream>>>(a, ni, no);
  return hipGetLastError();
}

}  // namespace eplb
