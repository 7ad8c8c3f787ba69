// Blocks of 128 in 8-bit floating point: along rows (activations), down the
// rows of a group (operands of a weight gradient), 128 x 128 (weights).
//
// All three read 2 or 4 bytes and write 1 per element.  Elements stay in
// registers between the block's maximum and the rounding.
#include "experts_device.h"

namespace eplb {

namespace {

constexpr int kQThreads = 256;

// Eight elements from i on, in 32 bits; those at `left` and behind are 0.
template <bool VEC>
__device__ __forceinline__ void load8(const void* p, int32_t dtype, int64_t i, int64_t left, float (&v)[8]) {
  if (VEC && left >= 8) {
    if (dtype == kF32) {
      const f32x4* f = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
      const f32x4 a = f[0], b = f[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
      const i32x4 h = *reinterpret_cast<const i32x4*>(static_cast<const u16*>(p) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = (uint32_t)h[j];
        v[2 * j] = dtype == kBf16 ? bf16_to_float((u16)w) : f16_to_float((u16)w);
        v[2 * j + 1] = dtype == kBf16 ? bf16_to_float((u16)(w >> 16)) : f16_to_float((u16)(w >> 16));
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? load_as_float(p, dtype, i + j) : 0.0f;
}

// How a thread loads eight elements of a block of rows: one by one, or as 16 or
// 32 bytes of a type known at compile time.  Then all rows' loads are in flight
// at once: nothing stands between them, rows and columns past the end read the
// first ones and are zeroed afterwards.
constexpr int kScalar = -1;                  // else EPLB_DTYPE_*

template <int M>
struct Raw8 {
  i32x4 v[M == kF32 ? 2 : 1];
};

template <int M>
__device__ __forceinline__ Raw8<M> fetch8(const void* p, int64_t i) {
  Raw8<M> r;
  const i32x4* from = reinterpret_cast<const i32x4*>(static_cast<const uint8_t*>(p) + i * (M == kF32 ? 4 : 2));
  r.v[0] = from[0];
  if constexpr (M == kF32) r.v[1] = from[1];
  return r;
}

template <int M>
__device__ __forceinline__ void unpack8(const Raw8<M>& r, bool in, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (M == kF32) {
      v[j] = in ? __int_as_float(r.v[0][j]) : 0.0f;
      v[4 + j] = in ? __int_as_float(r.v[1][j]) : 0.0f;
    } else {
      const uint32_t w = in ? (uint32_t)r.v[0][j] : 0;
      v[2 * j] = M == kBf16 ? bf16_to_float((u16)w) : f16_to_float((u16)w);
      v[2 * j + 1] = M == kBf16 ? bf16_to_float((u16)(w >> 16)) : f16_to_float((u16)(w >> 16));
    }
  }
}

// Calls f with the way to load.
template <typename F>
hipError_t by_load(bool vec, int32_t dtype, F f) {
  if (!vec) return f(std::integral_constant<int, kScalar>());
  if (dtype == kF32) return f(std::integral_constant<int, kF32>());
  if (dtype == kBf16) return f(std::integral_constant<int, kBf16>());
  return f(std::integral_constant<int, kF16>());
}

// Largest magnitude; a NaN or an infinity among the values gives infinity.
template <int N>
__device__ __forceinline__ float magnitude(const float (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(v[j]) <= 3.4028235e38f ? fabsf(v[j]) : INFINITY);
  return m;
}

// The scale of a block and the factor of its elements; a block that is not
// finite gets the scale NaN and the factor 0.
__device__ __forceinline__ float scale_of(float amax, float& factor) {
  if (amax == INFINITY) {
    factor = 0.0f;
    return NAN;
  }
  return block_scale(amax, factor);
}

// v * factor; 0 where the factor is (0 times an infinity or a NaN is not).
__device__ __forceinline__ float scaled(float v, float factor) { return factor == 0.0f ? 0.0f : v * factor; }

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* p, int64_t i, int64_t left, uint32_t a, uint32_t b) {
  if (VEC && left >= 8) {
    *reinterpret_cast<uint2*>(p + i) = make_uint2(a, b);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) p[i + j] = (uint8_t)((j < 4 ? a : b) >> (8 * (j & 3)));
}

// A block is 16 lanes of 8 elements, 16 bytes of a 16-bit type a lane; a
// workgroup takes 16 blocks.  8192 x 4096 bfloat16: 25 us (102 MB, 4.1 TB/s, two
// thirds of a copy's rate): the vector units are busy for 90 % of it.
template <bool VEC>
__global__ __launch_bounds__(kQThreads) void quantize_rows_kernel(const void* __restrict__ x, int32_t dtype, int64_t ld,
                                                                  int64_t R, int64_t C, int64_t nb,
                                                                  uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int part = threadIdx.x & 15;
  const int64_t blocks = R * nb, step = (int64_t)gridDim.x * (kQThreads / 16);
  for (int64_t b = (int64_t)blockIdx.x * (kQThreads / 16) + threadIdx.x / 16; b < blocks; b += step) {
    const int64_t r = b / nb, c = (b - r * nb) * kBlock + part * 8;
    float v[8];
    load8<VEC>(x, dtype, r * ld + c, C - c, v);
    float m = magnitude(v);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 16));
    float f;
    const float sc = scale_of(m, f);
    if (part == 0) scale[b] = sc;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = scaled(v[j], f);
    store8<VEC>(q, r * C + c, C - c, pack_f8(v[0], v[1], v[2], v[3]), pack_f8(v[4], v[5], v[6], v[7]));
  }
}

// One block of 128 rows and 128 columns per workgroup: a thread holds 8 rows
// of 8 columns (16 bytes a load), whose 8-bit values are 8 consecutive bytes of
// 8 rows of the output; they pass through LDS so that a store covers a whole
// 128-byte run.  The gathers of `rows` are whole 256-byte runs of a 16-bit
// type.  16384 rows of 4096 bfloat16 columns, each source row read twice: 58 us
// (201 MB, 3.5 TB/s; 80 us with each row's load behind a choice of its type);
// 2048 columns: 34 us.  LDS bounds it, busy for 86 % of the time, three quarters
// of that with bank conflicts (the turned block's stores).
template <int M>
__global__ __launch_bounds__(kQThreads) void quantize_columns_kernel(const void* __restrict__ x, int32_t dtype,
                                                                     int64_t ld, int64_t X, int64_t C,
                                                                     const int32_t* __restrict__ rows, int32_t R,
                                                                     FastDiv fd_k, const int32_t* __restrict__ offsets,
                                                                     int32_t G, int64_t Rp, uint8_t* __restrict__ q,
                                                                     float* __restrict__ scale, int32_t col_tiles) {
  __shared__ float part[16][kBlock + 4];
  __shared__ __attribute__((aligned(16))) uint8_t turned[kBlock][kBlock + 16];
  __shared__ int32_t src[kBlock];
  const int32_t b = (int32_t)(blockIdx.x / col_tiles);
  const Tile t = find_tile(offsets, G, R, kBlock, b, false);
  if (t.g < 0) return;
  if (threadIdx.x < kBlock) {
    int32_t from = -1;
    if ((int)threadIdx.x < t.rows) {
      from = t.row + threadIdx.x;
      if (rows != nullptr) {
        from = rows[from];
        from = from < 0 ? -1 : (int32_t)fastdiv_apply((uint32_t)from, fd_k);
      }
      if (from >= X) from = -1;
    }
    src[threadIdx.x] = from;
  }
  __syncthreads();
  const int cx = threadIdx.x & 15, band = threadIdx.x >> 4;
  const int64_t c0 = (int64_t)(blockIdx.x % col_tiles) * kBlock, c = c0 + cx * 8;
  float v[8][8];
  if constexpr (M == kScalar) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t from = src[band * 8 + i];
      load8<false>(x, dtype, (int64_t)(from < 0 ? 0 : from) * ld + c, from < 0 ? 0 : C - c, v[i]);
    }
  } else {                                   // X > 0, C % 8 == 0
    const bool in = c < C;
    int32_t from[8];
    Raw8<M> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) from[i] = src[band * 8 + i];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = fetch8<M>(x, (int64_t)(from[i] < 0 ? 0 : from[i]) * ld + (in ? c : 0));
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack8<M>(raw[i], in && from[i] >= 0, v[i]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i][j]) <= 3.4028235e38f ? fabsf(v[i][j]) : INFINITY);
    part[band][cx * 8 + j] = m;
  }
  __syncthreads();
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, part[i][cx * 8 + j]);
    const float sc = scale_of(m, f[j]);
    if (band == 0 && c + j < C) scale[(int64_t)b * C + c + j] = sc;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i][j] = scaled(v[i][j], f[j]);
    *reinterpret_cast<uint2*>(&turned[cx * 8 + j][band * 8]) =
        make_uint2(pack_f8(v[0][j], v[1][j], v[2][j], v[3][j]), pack_f8(v[4][j], v[5][j], v[6][j], v[7][j]));
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int i = threadIdx.x + p * kQThreads, r = i >> 3, at = (i & 7) * 16;
    if (c0 + r < C)
      *reinterpret_cast<uint4*>(q + (c0 + r) * Rp + (int64_t)b * kBlock + at) = *reinterpret_cast<const uint4*>(&turned[r][at]);
  }
}

// One 128 x 128 block per workgroup: a thread holds 8 rows of 8 columns, so
// that it has 8 consecutive bytes of both layouts.  9 x 2048 x 4096 bfloat16
// with both outputs: 60 us (302 MB, 5.1 TB/s, 0.8 of a copy's rate).
template <int M>
__global__ __launch_bounds__(kQThreads) void quantize_weights_kernel(const void* __restrict__ w, int32_t dtype, int64_t N,
                                                                     int64_t K, int32_t nn, int32_t nk,
                                                                     uint8_t* __restrict__ q, float* __restrict__ scale,
                                                                     uint8_t* __restrict__ qt,
                                                                     float* __restrict__ scale_t) {
  __shared__ float wave_max[kQThreads / 64];
  const int64_t per = (int64_t)nn * nk;
  const int64_t g = blockIdx.x / per;
  const int32_t bn = (int32_t)(blockIdx.x % per / nk), bk = (int32_t)(blockIdx.x % nk);
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int64_t n0 = (int64_t)bn * kBlock + ry * 8, k0 = (int64_t)bk * kBlock + cx * 8;
  constexpr bool VEC = M != kScalar;
  float v[8][8];
  float m = 0.0f;
  if constexpr (M == kScalar) {
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<false>(w, dtype, (g * N + n0 + i) * K + k0, n0 + i < N ? K - k0 : 0, v[i]);
  } else {                                   // K % 8 == 0
    Raw8<M> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = fetch8<M>(w, (g * N + (n0 + i < N ? n0 + i : 0)) * K + (k0 < K ? k0 : 0));
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack8<M>(raw[i], n0 + i < N && k0 < K, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, magnitude(v[i]));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQThreads / 64; ++i) m = fmaxf(m, wave_max[i]);
  float f;
  const float sc = scale_of(m, f);
  if (threadIdx.x == 0) {
    scale[(g * nn + bn) * nk + bk] = sc;
    if (qt != nullptr) scale_t[(g * nk + bk) * nn + bn] = sc;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = scaled(v[i][j], f);
    if (n0 + i < N)
      store8<VEC>(q, (g * N + n0 + i) * K + k0, K - k0, pack_f8(v[i][0], v[i][1], v[i][2], v[i][3]),
                  pack_f8(v[i][4], v[i][5], v[i][6], v[i][7]));
  }
  if (qt == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (k0 + j < K) {
      const uint32_t a = pack_f8(v[0][j], v[1][j], v[2][j], v[3][j]), b = pack_f8(v[4][j], v[5][j], v[6][j], v[7][j]);
      if (N % 8 == 0) store8<VEC>(qt, (g * K + k0 + j) * N + n0, N - n0, a, b);
      else store8<false>(qt, (g * K + k0 + j) * N + n0, N - n0, a, b);
    }
}

bool aligned(const void* p, int64_t n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

}  // namespace

hipError_t launch_quantize_rows(const void* x, int32_t dtype, int64_t ld, int64_t R, int64_t C, uint8_t* q,
                                float* scale, hipStream_t stream) {
  if (R == 0) return hipSuccess;
  const int64_t nb = ceil_div(C, kBlock);
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(R * nb, kQThreads / 16), 1 << 16);
  const bool vec = aligned(x, 16) && ld * dtype_size(dtype) % 16 == 0 && C % 8 == 0 && aligned(q, 8);
  if (vec) quantize_rows_kernel<true><<<dim3(grid), dim3(kQThreads), 0, stream>>>(x, dtype, ld, R, C, nb, q, scale);
  else quantize_rows_kernel<false><<<dim3(grid), dim3(kQThreads), 0, stream>>>(x, dtype, ld, R, C, nb, q, scale);
  return hipGetLastError();
}

hipError_t launch_quantize_columns(const void* x, int32_t dtype, int64_t ld, int64_t X, int64_t C,
                                   const int32_t* rows, int64_t R, int32_t K, const int32_t* offsets, int32_t G,
                                   int64_t Rp, uint8_t* q, float* scale, hipStream_t stream) {
  if (Rp == 0) return hipSuccess;
  const int64_t col_tiles = ceil_div(C, kBlock);
  const dim3 grid((unsigned)(Rp / kBlock * col_tiles));
  const FastDiv fd = fastdiv_make((uint32_t)K);
  const bool vec = X > 0 && aligned(x, 16) && ld * dtype_size(dtype) % 16 == 0 && C % 8 == 0;
  return by_load(vec, dtype, [&](auto mode) {
    quantize_columns_kernel<decltype(mode)::value><<<grid, dim3(kQThreads), 0, stream>>>(
        x, dtype, ld, X, C, rows, (int32_t)R, fd, offsets, G, Rp, q, scale, (int32_t)col_tiles);
    return hipGetLastError();
  });
}

hipError_t launch_quantize_weights(const void* w, int32_t dtype, int32_t G, int64_t N, int64_t K, uint8_t* q,
                                   float* scale, uint8_t* qt, float* scale_t, hipStream_t stream) {
  const int64_t nn = ceil_div(N, kBlock), nk = ceil_div(K, kBlock);
  const dim3 grid((unsigned)(G * nn * nk));
  const bool vec = aligned(w, 16) && K % 8 == 0 && aligned(q, 8) && aligned(qt, 8);
  return by_load(vec, dtype, [&](auto mode) {
    quantize_weights_kernel<decltype(mode)::value><<<grid, dim3(kQThreads), 0, stream>>>(w, dtype, N, K, (int32_t)nn,
                                                                                         (int32_t)nk, q, scale, qt, scale_t);
    return hipGetLastError();
  });
}

}  // namespace eplb
