// The experts' rows joined to tokens, and the gradients of that.
//
// Each row is read once and each output written once; nothing is computed that
// the memory would not have time for.  A workgroup takes whole tokens, each with
// the lanes that its width needs, eight elements to a lane; a choice's rows are
// loaded eight at a time before the first is used.
#include "layer_internal.h"

namespace eplb {

namespace {

constexpr int kThreads = 256;
constexpr int kEach = 8;                   // elements of a lane

typedef u16 u16x8 __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x8 __attribute__((ext_vector_type(8), aligned(4)));

// Eight elements from `at` on (rows of any width: aligned to an element), or the `n` that there are.
template <int DTYPE>
__device__ __forceinline__ void load8(const void* p, int64_t at, int n, float (&v)[kEach]) {
  if (n >= kEach) {
    if (DTYPE == kF32) {
      const f32x8 x = *reinterpret_cast<const f32x8*>(static_cast<const float*>(p) + at);
#pragma unroll
      for (int j = 0; j < kEach; ++j) v[j] = x[j];
    } else {
      const u16x8 x = *reinterpret_cast<const u16x8*>(static_cast<const u16*>(p) + at);
#pragma unroll
      for (int j = 0; j < kEach; ++j) v[j] = DTYPE == kBf16 ? bf16_to_float(x[j]) : f16_to_float(x[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) v[j] = j < n ? load_as_float(p, DTYPE, at + j) : 0.0f;
}

__device__ __forceinline__ void load8(const void* p, int32_t dtype, int64_t at, int n, float (&v)[kEach]) {
  if (dtype == kF32) load8<kF32>(p, at, n, v);
  else if (dtype == kBf16) load8<kBf16>(p, at, n, v);
  else load8<kF16>(p, at, n, v);
}

__device__ __forceinline__ void store8(void* p, int32_t dtype, int64_t at, int n, const float (&v)[kEach]) {
  if (n >= kEach) {
    if (dtype == kF32) {
      f32x8 x;
#pragma unroll
      for (int j = 0; j < kEach; ++j) x[j] = v[j];
      *reinterpret_cast<f32x8*>(static_cast<float*>(p) + at) = x;
    } else {
      u16x8 x;
#pragma unroll
      for (int j = 0; j < kEach; ++j) x[j] = dtype == kBf16 ? float_to_bf16(v[j]) : float_to_f16(v[j]);
      *reinterpret_cast<u16x8*>(static_cast<u16*>(p) + at) = x;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (j < n) store_float(p, dtype, at + j, v[j]);
}

// Lanes of a token: a power of two, a workgroup at most.
int lanes_for(int64_t C) {
  int n = 1;
  while (n < kThreads && (int64_t)n * kEach < C) n *= 2;
  return n;
}

// WHOLE: a workgroup to a token (what a token's lanes have in common is then held once for a wave).
template <int DTYPE, bool WHOLE>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a, int32_t lanes) {
  const int each = WHOLE ? 1 : kThreads / lanes;
  const int mine = WHOLE ? 0 : threadIdx.x / lanes;
  const int64_t c = (int64_t)blockIdx.y * kThreads * kEach + (WHOLE ? threadIdx.x : threadIdx.x % lanes) * kEach;
  const int n = (int)min((int64_t)kEach, a.C - c);
  if (n <= 0) return;
  for (int64_t t = (int64_t)blockIdx.x * each + mine; t < a.T; t += (int64_t)gridDim.x * each) {
    float sum[kEach] = {};
    for (int k0 = 0; k0 < a.K; k0 += 8) {
      float v[8][kEach], w[8];
      int32_t p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = t * a.K + min(k0 + j, a.K - 1);
        p[j] = a.place[i];
        w[j] = a.weights == nullptr ? 1.0f : a.weights[i];
        if (k0 + j >= a.K || p[j] >= a.R) p[j] = -1;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p[j] >= 0) load8<DTYPE>(a.y, p[j] * a.C + c, n, v[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (p[j] >= 0) {
#pragma unroll
          for (int e = 0; e < kEach; ++e) sum[e] = fmaf(w[j], v[j][e], sum[e]);
        }
    }
    store8(a.out, a.out_dtype, t * a.C + c, n, sum);
  }
}

// A token's lanes go over its width together; the choices' sums of products
// are added up over the lanes at the end, in a fixed order.
template <int DTYPE, bool WHOLE>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(CombineBackwardArgs a, int32_t lanes) {
  __shared__ float part[8][kThreads / 64];
  const int each = WHOLE ? 1 : kThreads / lanes;
  const int mine = WHOLE ? 0 : threadIdx.x / lanes, lane = WHOLE ? threadIdx.x : threadIdx.x % lanes;
  const int64_t rows = a.T * a.K;
  for (int64_t t0 = (int64_t)blockIdx.x * each; t0 < a.T; t0 += (int64_t)gridDim.x * each) {
    const int64_t t = t0 + mine;
    const bool some = t < a.T;
    for (int k0 = 0; k0 < a.K; k0 += 8) {
      float w[8], dot[8] = {};
      int32_t p[8];
      bool write[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = (some ? t : 0) * a.K + min(k0 + j, a.K - 1);
        p[j] = a.place[i];
        w[j] = a.weights == nullptr ? 1.0f : a.weights[i];
        if (!some || k0 + j >= a.K || p[j] >= rows) p[j] = -1;
        write[j] = p[j] >= 0 && a.order[p[j]] == i;
      }
      if (some)
        for (int64_t c = (int64_t)lane * kEach; c < a.C; c += (int64_t)lanes * kEach) {
          const int n = (int)min((int64_t)kEach, a.C - c);
          float d[kEach], y[8][kEach];
          load8(a.d_out, a.dtype, t * a.C + c, n, d);
          if (a.d_weights != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (p[j] >= 0) load8<DTYPE>(a.y, p[j] * a.C + c, n, y[j]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (write[j]) {
              float g[kEach];
#pragma unroll
              for (int e = 0; e < kEach; ++e) g[e] = w[j] * d[e];
              store8(a.d_y, DTYPE, p[j] * a.C + c, n, g);
            }
            if (a.d_weights != nullptr && p[j] >= 0) {
#pragma unroll
              for (int e = 0; e < kEach; ++e) dot[j] = fmaf(d[e], y[j][e], dot[j]);
            }
          }
        }
      if (a.d_weights == nullptr) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        for (int s = min(lanes, 64) / 2; s > 0; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
      if (lanes > 64) {
        __syncthreads();                   // the sums before these have been read
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) part[j][threadIdx.x >> 6] = dot[j];
        }
        __syncthreads();
        const int waves = lanes / 64, first = mine * waves;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dot[j] = 0.0f;
          for (int s = 0; s < waves; ++s) dot[j] += part[j][first + s];
        }
      }
      if (some && lane == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (k0 + j < a.K) a.d_weights[t * a.K + k0 + j] = dot[j];
      }
    }
    // rows that no choice is the only one of: zeros
    if (some)
      for (int k = 0; k < a.K; ++k) {
        const int64_t r = t * a.K + k;
        const int32_t i = a.order[r];
        if (i >= 0 && i < rows && a.place[i] == r) continue;
        for (int64_t c = (int64_t)lane * kEach; c < a.C; c += (int64_t)lanes * kEach) {
          const float zero[kEach] = {};
          store8(a.d_y, DTYPE, r * a.C + c, (int)min((int64_t)kEach, a.C - c), zero);
        }
      }
  }
}

// Workgroups along the tokens: what is past them is taken in turns.
unsigned groups_for(int64_t T, int lanes) {
  return (unsigned)std::min(ceil_div(T, kThreads / lanes), int64_t(1) << 22);
}

template <int DTYPE>
void launch(const CombineArgs& a, hipStream_t stream) {
  const int lanes = lanes_for(a.C);
  const dim3 grid(groups_for(a.T, lanes), (unsigned)ceil_div(a.C, kThreads * kEach));
  if (lanes == kThreads) combine_kernel<DTYPE, true><<<grid, kThreads, 0, stream>>>(a, lanes);
  else combine_kernel<DTYPE, false><<<grid, kThreads, 0, stream>>>(a, lanes);
}

template <int DTYPE>
void launch_backward(const CombineBackwardArgs& a, hipStream_t stream) {
  const int lanes = lanes_for(a.C);
  const dim3 grid(groups_for(a.T, lanes));
  if (lanes == kThreads) combine_backward_kernel<DTYPE, true><<<grid, kThreads, 0, stream>>>(a, lanes);
  else combine_backward_kernel<DTYPE, false><<<grid, kThreads, 0, stream>>>(a, lanes);
}

}  // namespace

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t stream) {
  if (a.dtype == kF32) launch<kF32>(a, stream);
  else if (a.dtype == kBf16) launch<kBf16>(a, stream);
  else launch<kF16>(a, stream);
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const CombineBackwardArgs& a, hipStream_t stream) {
  if (a.y_dtype == kF32) launch_backward<kF32>(a, stream);
  else if (a.y_dtype == kBf16) launch_backward<kBf16>(a, stream);
  else launch_backward<kF16>(a, stream);
  return hipGetLastError();
}

}  // namespace eplb
