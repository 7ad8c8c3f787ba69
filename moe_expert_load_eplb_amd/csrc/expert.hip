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

}  // namespace

int64_t matmul_tiles(int64_t R, int64_t N, int32_t G) { return (R / kTile + G + 2) * ceil_div(N, kTile); }

int64_t wgrad_tiles(int64_t N, int64_t K, int32_t G) { return G * ceil_div(N, kTile) * ceil_div(K, kTile); }

hipError_t launch_expert_matmul(const MatmulArgs& a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  const dim3 grid((unsigned)matmul_tiles(a.R, a.N, a.G));
  if (a.dtype == kF32) expert_matmul_kernel<true><<<grid, dim3(kMmThreads), 0, stream>>>(a);
  else expert_matmul_kernel<false><<<grid, dim3(kMmThreads), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_expert_wgrad(const WgradArgs& a, hipStream_t stream) {
  const int32_t ni = (int32_t)ceil_div(a.K, kTile), no = (int32_t)ceil_div(a.N, kTile);
  const dim3 grid((unsigned)wgrad_tiles(a.N, a.K, a.G));
  if (a.dtype == kF32) expert_wgrad_kernel<true><<<grid, dim3(kMmThreads), 0, stream>>>(a, ni, no);
  else expert_wgrad_kernel<false><<<grid, dim3(kMmThreads), 0, stream>>>(a, ni, no);
  return hipGetLastError();
}

}  // namespace eplb
