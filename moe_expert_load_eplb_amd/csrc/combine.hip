// The experts' rows joined to tokens, and the gradients of that.
//
// Each row is read once and each output written once; nothing is computed that
// the memory would not have time for.  A token is one wave's, or a workgroup's where
// its row is wide, so that what its choices name is in scalar registers.  All of a
// lane's rows, eight choices of eight elements, are asked for before the first is
// used, with no branch among them: a row has a descriptor of its own, of no bytes
// where the choice has none, and what lies past it is zeros, or not written.
//
// Measured, random places: 16384 tokens of 8 rows of 2048 bfloat16: 102 us, 5.9
// TB/s; their gradients 232 us, 4.9 TB/s (with a branch to each row: 150 and 443),
// 167 us without that of the weights, which alone reads y.
#include "layer_internal.h"

namespace eplb {

namespace {

constexpr int kWidest = 512;               // lanes of a token at most
constexpr int kAlone = 4;                  // waves of a workgroup where each has a token
constexpr int kEach = 8;                   // elements of a lane
constexpr int kOnce = 2;                   // loads and stores: not to be kept in the caches (119 us without, 102 with)

// A row's descriptor, the same for the wave.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* p, int64_t row, int64_t bytes, bool some) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(static_cast<const uint8_t*>(p)) + (some ? row * bytes : 0),
                                           0, some ? (int)bytes : 0, 0x00020000);
}

constexpr int size_of(int dtype) { return dtype == kF32 ? 4 : 2; }

// A lane's eight elements of a row as they lie in memory, U of them next to each other and 64 U from one such unit to the
// next.  16 bytes across lines take the memory units several turns, and rows of a width that is no multiple of 8 start
// anywhere: units are 16 bytes where the width is such a multiple, else pairs, or single ones for odd widths.  (4097 tokens
// of 6 rows of 2050 half-precision values: 31 us in pairs, 52 in eights; their gradients 66 and 191.)  Narrow rows are taken
// in smaller units, too: more lanes have one.
template <int DTYPE, int U>
struct Eight {
  static constexpr int kBytes = U * size_of(DTYPE), kUnits = kEach / U;
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kUnits][kWords];

  // first: this lane's first element; left: the elements from the wave's first one on (what is past them is not asked for)
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int first, int left) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (kBytes > 2 && u > 0 && u * 64 * U >= left) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) w[u][j] = 0;
        continue;
      }
      const int at = (first + u * 64 * U) * size_of(DTYPE);
      if constexpr (kBytes == 2) {
        w[u][0] = __builtin_amdgcn_raw_buffer_load_b16(row, at, 0, kOnce);
      } else if constexpr (kBytes == 4) {
        w[u][0] = __builtin_amdgcn_raw_buffer_load_b32(row, at, 0, kOnce);
      } else if constexpr (kBytes == 8) {
        const auto x = __builtin_amdgcn_raw_buffer_load_b64(row, at, 0, kOnce);
        w[u][0] = x[0];
        w[u][1] = x[1];
      } else {
#pragma unroll
        for (int h = 0; h < kWords; h += 4) {
          const auto x = __builtin_amdgcn_raw_buffer_load_b128(row, at + h * 4, 0, kOnce);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[u][h + j] = x[j];
        }
      }
    }
  }
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t row, int first, int left) const {
    typedef uint32_t Two __attribute__((ext_vector_type(2)));
    typedef uint32_t Four __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (u > 0 && u * 64 * U >= left) break;
      const int at = (first + u * 64 * U) * size_of(DTYPE);
      if constexpr (kBytes == 2) __builtin_amdgcn_raw_buffer_store_b16((u16)w[u][0], row, at, 0, kOnce);
      else if constexpr (kBytes == 4) __builtin_amdgcn_raw_buffer_store_b32(w[u][0], row, at, 0, kOnce);
      else if constexpr (kBytes == 8) __builtin_amdgcn_raw_buffer_store_b64(Two{w[u][0], w[u][1]}, row, at, 0, kOnce);
      else
#pragma unroll
        for (int h = 0; h < kWords; h += 4)
          __builtin_amdgcn_raw_buffer_store_b128(Four{w[u][h], w[u][h + 1], w[u][h + 2], w[u][h + 3]}, row, at + h * 4, 0, kOnce);
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    const int u = i / U, e = i % U;
    if constexpr (DTYPE == kF32) {
      return __uint_as_float(w[u][e]);
    } else {
      const u16 h = (u16)(w[u][e / 2] >> e % 2 * 16);
      return DTYPE == kBf16 ? bf16_to_float(h) : f16_to_float(h);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[kEach]) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int u = i / U, e = i % U;
      if constexpr (DTYPE == kF32) {
        w[u][e] = __float_as_uint(v[i]);
      } else {
        const uint32_t h = DTYPE == kBf16 ? float_to_bf16(v[i]) : float_to_f16(v[i]);
        w[u][e / 2] = e % 2 == 0 ? h : w[u][e / 2] | h << 16;
      }
    }
  }
};

template <int DTYPE, int U>
__device__ __forceinline__ void store_eight(void* p, int64_t row, int64_t C, int first, int left, const float (&v)[kEach]) {
  Eight<DTYPE, U> x;
  x.set(v);
  x.store(row_of(p, row, C * size_of(DTYPE), true), first, left);
}

// A token's width over the waves of a workgroup: one, and kAlone tokens to a workgroup, or `waves`, in `slices` workgroups
// where it is past kWidest lanes.
struct Width {
  int waves, slices;
  int block() const { return 64 * (waves == 1 ? kAlone : waves); }
};

Width width_for(int64_t C) {
  const int64_t waves = ceil_div(C, 64 * kEach), slices = ceil_div(waves, kWidest / 64);
  return Width{(int)ceil_div(waves, slices), (int)slices};
}

// `K` choices of 8 / K tokens at once: a token of few choices alone asks for too little at a time (8192 tokens of 2 rows of
// 4096 32-bit values: 73 us by fours, 92 alone).
template <int DTYPE, int U, int K>
__global__ __launch_bounds__(kWidest) void combine_kernel(CombineArgs a, int32_t waves) {
  constexpr int kTokens = 8 / K;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int each = waves == 1 ? kAlone : 1;
  const int begin = ((int)blockIdx.y * waves + (waves == 1 ? 0 : wave)) * (64 * kEach), left = (int)a.C - begin;
  const int first = begin + (int)(threadIdx.x & 63) * U;
  for (int64_t t0 = ((int64_t)blockIdx.x * each + (waves == 1 ? wave : 0)) * kTokens; t0 < a.T;
       t0 += (int64_t)gridDim.x * each * kTokens) {
    float sum[kTokens][kEach] = {};
    for (int k0 = 0; k0 < a.K; k0 += K) {
      Eight<DTYPE, U> v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t t = min(t0 + j / K, a.T - 1), i = t * a.K + min(k0 + j % K, a.K - 1);
        const int32_t p = a.place[i];
        const bool some = k0 + j % K < a.K && p >= 0 && p < a.R;
        w[j] = !some ? 0.0f : a.weights == nullptr ? 1.0f : a.weights[i];
        if (k0 + j % K < a.K && t0 + j / K < a.T) v[j].load(row_of(a.y, p, a.C * size_of(DTYPE), some), first, left);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k0 + j % K < a.K && t0 + j / K < a.T) {
#pragma unroll
          for (int e = 0; e < kEach; ++e) sum[j / K][e] = fmaf(w[j], v[j][e], sum[j / K][e]);
        }
    }
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
      if (t0 + n >= a.T) break;
      if (a.out_dtype == kF32) store_eight<kF32, U>(a.out, t0 + n, a.C, first, left, sum[n]);
      else if (a.out_dtype == kBf16) store_eight<kBf16, U>(a.out, t0 + n, a.C, first, left, sum[n]);
      else store_eight<kF16, U>(a.out, t0 + n, a.C, first, left, sum[n]);
    }
  }
}

// A token's lanes go over its width together; the choices' sums of products
// are added up over the lanes at the end, in a fixed order.
template <int DTYPE, int U>
__global__ __launch_bounds__(kWidest) void combine_backward_kernel(CombineBackwardArgs a, int32_t waves) {
  __shared__ float part[8][kWidest / 64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int each = waves == 1 ? kAlone : 1;
  const int begin = (waves == 1 ? 0 : wave) * (64 * kEach);
  const int64_t rows = a.T * a.K, bytes = a.C * size_of(DTYPE);
  for (int64_t t = (int64_t)blockIdx.x * each + (waves == 1 ? wave : 0); t < a.T; t += (int64_t)gridDim.x * each) {
    // rows t K .. of d_y that no choice is the only one of get zeros: bit k
    bool lost = false;
    if (lane < a.K) {
      const int32_t i = a.order[t * a.K + lane];
      lost = i < 0 || i >= rows || a.place[i] != t * a.K + lane;
    }
    u64 none = __ballot(lost);
    for (int k0 = 0; k0 < a.K; k0 += 8) {
      float w[8], dot[8] = {};
      int32_t p[8];
      bool some[8], write[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = t * a.K + min(k0 + j, a.K - 1);
        p[j] = a.place[i];
        w[j] = a.weights == nullptr ? 1.0f : a.weights[i];
        some[j] = k0 + j < a.K && p[j] >= 0 && p[j] < rows;
        write[j] = some[j] && a.order[some[j] ? p[j] : 0] == i;
      }
      for (int64_t c = 0; c < a.C; c += waves * (64 * kEach)) {
        const int left = (int)a.C - (int)c - begin, at = (int)c + begin + lane * U;
        Eight<DTYPE, U> y[8];
        if (a.d_weights != nullptr) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k0 + j < a.K) y[j].load(row_of(a.y, p[j], bytes, some[j]), at, left);
        }
        float d[kEach];
        auto load_d = [&](auto type) {
          Eight<decltype(type)::value, U> v;
          v.load(row_of(a.d_out, t, a.C * size_of(decltype(type)::value), true), at, left);
#pragma unroll
          for (int e = 0; e < kEach; ++e) d[e] = v[e];
        };
        if (a.dtype == kF32) load_d(std::integral_constant<int, kF32>());
        else if (a.dtype == kBf16) load_d(std::integral_constant<int, kBf16>());
        else load_d(std::integral_constant<int, kF16>());
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (k0 + j >= a.K) break;
          Eight<DTYPE, U> x;
          float g[kEach];
#pragma unroll
          for (int e = 0; e < kEach; ++e) g[e] = w[j] * d[e];
          x.set(g);
          x.store(row_of(a.d_y, p[j], bytes, write[j]), at, left);
          if (a.d_weights != nullptr) {
            // a choice of no row: nothing, whatever d_out holds
#pragma unroll
            for (int e = 0; e < kEach; ++e) dot[j] = fmaf(some[j] ? d[e] : 0.0f, y[j][e], dot[j]);
          }
        }
      }
      if (a.d_weights == nullptr) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        for (int s = 32; s > 0; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
      if (waves == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (lane == j && k0 + j < a.K) a.d_weights[t * a.K + k0 + j] = dot[j];
        continue;
      }
      __syncthreads();                     // the sums before these have been read
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[j][wave] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < 8 && k0 + (int)threadIdx.x < a.K) {
        float sum = 0.0f;
        for (int s = 0; s < waves; ++s) sum += part[threadIdx.x][s];
        a.d_weights[t * a.K + k0 + threadIdx.x] = sum;
      }
    }
    for (; none != 0; none &= none - 1) {
      const int64_t r = t * a.K + __ffsll((unsigned long long)none) - 1;
      const float zero[kEach] = {};
      for (int64_t c = 0; c < a.C; c += waves * (64 * kEach))
        store_eight<DTYPE, U>(a.d_y, r, a.C, (int)c + begin + lane * U, (int)a.C - (int)c - begin, zero);
    }
  }
}

// Workgroups along the tokens: what is past them is taken in turns.
unsigned groups_for(int64_t T, int waves, int tokens) {
  return (unsigned)std::min(ceil_div(T, (waves == 1 ? kAlone : 1) * tokens), int64_t(1) << 22);
}

template <int DTYPE, int U, int K>
void launch_choices(const CombineArgs& a, hipStream_t stream) {
  const Width w = width_for(a.C);
  combine_kernel<DTYPE, U, K><<<dim3(groups_for(a.T, w.waves, 8 / K), w.slices), w.block(), 0, stream>>>(a, w.waves);
}

template <int DTYPE, int U>
void launch(const CombineArgs& a, hipStream_t stream) {
  // several tokens to a wave only where there are workgroups for the chip all the same (64 tokens of 2 rows of 4096: 7.7 us
  // by fours, 5.1 alone)
  const int waves = width_for(a.C).waves, few = a.K <= 2 ? 2 : a.K <= 4 ? 4 : 8;
  const int choices = groups_for(a.T, waves, 8 / few) >= 512 ? few : 8;
  if (choices == 2) launch_choices<DTYPE, U, 2>(a, stream);
  else if (choices == 4) launch_choices<DTYPE, U, 4>(a, stream);
  else launch_choices<DTYPE, U, 8>(a, stream);
}

template <int DTYPE, int U>
void launch(const CombineBackwardArgs& a, hipStream_t stream) {
  const Width w = width_for(a.C);
  combine_backward_kernel<DTYPE, U><<<groups_for(a.T, w.waves, 1), w.block(), 0, stream>>>(a, w.waves);
}

bool on_words(const void* p) { return (uintptr_t)p % 4 == 0; }
bool on_words(const CombineArgs& a) { return on_words(a.y) && on_words(a.out); }
bool on_words(const CombineBackwardArgs& a) { return on_words(a.d_out) && on_words(a.y) && on_words(a.d_y); }

// Units of more than two bytes need rows that start at a multiple of four.
template <int DTYPE, typename Args>
void launch_for(const Args& a, hipStream_t stream) {
  if (a.C % 2 != 0 || !on_words(a)) launch<DTYPE, 1>(a, stream);
  else if (a.C % 8 == 0 && a.C > 128) launch<DTYPE, 16 / size_of(DTYPE)>(a, stream);
  else launch<DTYPE, 2>(a, stream);
}

}  // namespace

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t stream) {
  if (a.dtype == kF32) launch_for<kF32>(a, stream);
  else if (a.dtype == kBf16) launch_for<kBf16>(a, stream);
  else launch_for<kF16>(a, stream);
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const CombineBackwardArgs& a, hipStream_t stream) {
  if (a.y_dtype == kF32) launch_for<kF32>(a, stream);
  else if (a.y_dtype == kBf16) launch_for<kBf16>(a, stream);
  else launch_for<kF16>(a, stream);
  return hipGetLastError();
}

}  // namespace eplb
