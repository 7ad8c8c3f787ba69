// The router: scores, the choice of K experts per token, the balance loss and
// the gradients of both.
//
// A row of E logits belongs to LPR lanes of one wave, VPL values each (expert
// j * LPR + lane), so every sum and maximum over the experts is a butterfly
// over LPR lanes and nothing of the row is read twice.
#include "experts_internal.h"

namespace eplb {

namespace {

constexpr int kGateThreads = 256;
constexpr int kLossRows = 64;                // rows of one workgroup of the loss

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, LPR);
  return v;
}

template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, LPR));
  return v;
}

// Each step is one correctly rounded 32-bit operation (and the library's
// exponential), so that a choice between near equal keys does not depend on
// how the expression is compiled.
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// A row's logits in 32 bits; experts past E hold minus infinity.
template <int LPR, int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int32_t dtype, int64_t at, int32_t E, int lane,
                                            float (&x)[VPL]) {
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * LPR + lane;
    x[j] = e < E ? load_as_float(logits, dtype, at + e) : -INFINITY;
  }
}

// Scores of a row.  Softmax: z = 1; sigmoid: z = sum of the scores + 1e-20,
// what a share of the balance loss divides by.
template <int LPR, int VPL>
__device__ __forceinline__ float scores(int32_t scoring, int32_t E, int lane, const float (&x)[VPL], float (&s)[VPL]) {
  if (scoring == kSigmoid) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      s[j] = j * LPR + lane < E ? sigmoid(x[j]) : 0.0f;
      z += s[j];
    }
    return row_sum<LPR>(z) + kScoreEps;
  }
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) m = fmaxf(m, x[j]);
  m = row_max<LPR>(m);
  if (m == -INFINITY) m = 0.0f;              // no expert is allowed: all scores are 0
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    s[j] = expf(x[j] - m);
    z += s[j];
  }
  z = row_sum<LPR>(z) + kScoreEps;
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[j] /= z;
  return 1.0f;
}

// Keys of the experts outside the top_groups best groups become minus
// infinity.  The row's keys pass through LDS so that lane g can scan group g.
template <int LPR, int VPL>
__device__ __forceinline__ void limit_groups(const GateArgs& a, int lane, float* row, float (&key)[VPL]) {
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * LPR + lane;
    if (e < a.E) row[e] = key[j];
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int size = a.E / a.G;
  u64 keep = 0;
  // a group's score, by lane g of each run of LPR groups
  float score[(kMaxGroups + LPR - 1) / LPR];
#pragma unroll
  for (int c = 0; c < (kMaxGroups + LPR - 1) / LPR; ++c) {
    const int g = c * LPR + lane;
    float b1 = -INFINITY, b2 = -INFINITY;
    if (g < a.G)
      for (int i = 0; i < size; ++i) {
        const float v = row[g * size + i];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
    const float sum = a.group_top == 2 ? b1 + b2 : b1;
    score[c] = sum != sum ? -INFINITY : sum;
  }
#pragma unroll
  for (int c = 0; c < (kMaxGroups + LPR - 1) / LPR; ++c) {
    const int g = c * LPR + lane;
    int before = 0;
#pragma unroll
    for (int d = 0; d < (kMaxGroups + LPR - 1) / LPR; ++d) {
      const int n = min(LPR, a.G - d * LPR);
      for (int i = 0; i < n; ++i) {
        const float o = __shfl(score[d], i, LPR);
        before += o > score[c] || (o == score[c] && d * LPR + i < g);
      }
    }
    const u64 all = __ballot(g < a.G && before < a.top_groups);
    const int shift = (threadIdx.x & 63) / LPR * LPR;
    const u64 mine = LPR == 64 ? all : (all >> shift) & ((u64(1) << (LPR & 63)) - 1);
    keep |= mine << (c * LPR & 63);
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * LPR + lane;
    const int g = (int)fastdiv_apply((uint32_t)e, a.fd_group);
    if (e < a.E && !(keep >> g & 1)) key[j] = -INFINITY;
  }
}

// One row: the choice (or the given ids), its weights, and, for the loss, the
// row's shares and counts added to the lane's own sums.
template <int LPR, int VPL, bool LOSS>
__device__ __forceinline__ void gate_row(const GateArgs& a, int64_t t, bool real, int lane, float* row, int32_t* cnt,
                                         float (&psum)[VPL]) {
  float x[VPL], s[VPL];
  load_logits<LPR, VPL>(a.logits, a.dtype, t * a.ld, real ? a.E : 0, lane, x);
  const float z = scores<LPR, VPL>(a.scoring, a.E, lane, x, s);
  if (LOSS && real) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) psum[j] += s[j] / z;
  }
  if (LOSS && a.given) {
    if (real)
      for (int k = lane; k < a.K; k += LPR) {
        const int32_t e = a.ids[t * a.K + k];
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&cnt[e], 1);
      }
    return;
  }
  float key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * LPR + lane;
    float v = a.scoring == kSigmoid ? s[j] : x[j];
    if (a.bias != nullptr && e < a.E) v += a.bias[e];
    key[j] = e < a.E && real && v == v ? v : -INFINITY;
  }
  if (a.top_groups < a.G) limit_groups<LPR, VPL>(a, lane, row, key);
  float chosen[(kMaxK + LPR - 1) / LPR];
  int32_t expert[(kMaxK + LPR - 1) / LPR];
#pragma unroll
  for (int c = 0; c < (kMaxK + LPR - 1) / LPR; ++c) chosen[c] = 0.0f, expert[c] = -1;
  for (int k = 0; k < a.K; ++k) {
    float best = -INFINITY, bs = 0.0f;
    int be = 1 << 30;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > best) best = key[j], be = j * LPR + lane, bs = s[j];
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) {
      const float ob = __shfl_xor(best, m, LPR), os = __shfl_xor(bs, m, LPR);
      const int oe = __shfl_xor(be, m, LPR);
      if (ob > best || (ob == best && oe < be)) best = ob, be = oe, bs = os;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (j * LPR + lane == be) key[j] = -INFINITY;
#pragma unroll
    for (int c = 0; c < (kMaxK + LPR - 1) / LPR; ++c)
      if (c * LPR + lane == k && best > -INFINITY) chosen[c] = bs, expert[c] = be;
  }
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < (kMaxK + LPR - 1) / LPR; ++c) sum += chosen[c];
  sum = row_sum<LPR>(sum) + kScoreEps;
  if (t < a.T) {
#pragma unroll
    for (int c = 0; c < (kMaxK + LPR - 1) / LPR; ++c) {
      const int k = c * LPR + lane;
      if (k < a.K) {
        a.ids[t * a.K + k] = expert[c];
        a.weights[t * a.K + k] = a.normalize ? a.scale * chosen[c] / sum : a.scale * chosen[c];
        if (LOSS && expert[c] >= 0) atomicAdd(&cnt[expert[c]], 1);
      }
    }
  }
}

template <int LPR, int VPL>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a) {
  extern __shared__ float rows_lds[];        // [rows at once][E]
  constexpr int kRows = kGateThreads / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int64_t t = (int64_t)blockIdx.x * kRows + sub;
  float none[VPL];
  const bool real = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
  gate_row<LPR, VPL, false>(a, t, real, lane, rows_lds + sub * a.E, nullptr, none);
}

// Number of entries of seg[0 .. S] that are at most t, minus one: the segment
// that holds row t, -1 before the first one, S behind the last one.
__device__ __forceinline__ int64_t segment_of(const int32_t* seg, int64_t S, int64_t t) {
  int64_t lo = 0, hi = S + 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (seg[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

__device__ __forceinline__ int64_t piece_end(const int32_t* seg, int64_t S, int64_t s, int64_t row, int64_t row1) {
  const int64_t e = s >= S ? row1 : seg[s + 1];
  return e <= row ? row + 1 : e < row1 ? e : row1;
}

// Floats of one partial sum: E sums of shares, E counts, the rows counted.
__host__ __device__ inline int64_t part_stride(int32_t E) { return (2 * (int64_t)E + 1 + 3) / 4 * 4; }

// Workgroup c takes rows c * kLossRows on, piece by piece where a segment
// ends.  The piece of segment s goes to partial sum c + s: two pieces never
// share one, as each next piece has a larger c or a larger s.
template <int LPR, int VPL>
__global__ __launch_bounds__(kGateThreads) void gate_loss_kernel(GateArgs a) {
  extern __shared__ float lds[];             // [rows at once][E] keys, then shares; [E] counts
  constexpr int kRows = kGateThreads / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float* row = lds + sub * a.E;
  int32_t* cnt = reinterpret_cast<int32_t*>(lds + kRows * a.E);
  __shared__ int32_t kept;
  const int64_t row0 = (int64_t)blockIdx.x * kLossRows;
  const int64_t row1 = row0 + kLossRows < a.T ? row0 + kLossRows : a.T;
  for (int64_t r = row0; r < row1;) {
    const int64_t s = segment_of(a.seg, a.S, r);
    const int64_t end = piece_end(a.seg, a.S, s, r, row1);
    for (int e = threadIdx.x; e < a.E; e += kGateThreads) cnt[e] = 0;
    if (threadIdx.x == 0) kept = 0;
    __syncthreads();
    float psum[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) psum[j] = 0.0f;
    int mine = 0;
    for (int64_t t0 = r; t0 < end; t0 += kRows) {
      const int64_t t = t0 + sub;
      const bool real = t < end && (a.mask == nullptr || a.mask[t] != 0);
      gate_row<LPR, VPL, true>(a, t < end ? t : a.T, real, lane, row, cnt, psum);
      mine += real;
    }
    if (lane == 0 && mine > 0) atomicAdd(&kept, mine);
    __syncthreads();
    if (s >= 0 && s < a.S) {
      float* part = a.part + (blockIdx.x + s) * part_stride(a.E);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j * LPR + lane < a.E) row[j * LPR + lane] = psum[j];
      __syncthreads();
      for (int e = threadIdx.x; e < a.E; e += kGateThreads) {
        float v = 0.0f;
        for (int i = 0; i < kRows; ++i) v += lds[i * a.E + e];
        part[e] = v;
        reinterpret_cast<int32_t*>(part)[a.E + e] = cnt[e];
      }
      if (threadIdx.x == 0) reinterpret_cast<int32_t*>(part)[2 * a.E] = kept;
    }
    __syncthreads();
    r = end;
  }
}

// Segment s: its partial sums added in the order of the rows.
__global__ __launch_bounds__(1024) void gate_loss_reduce_kernel(GateArgs a) {
  __shared__ float sums[16];
  const int64_t s = blockIdx.x;
  int64_t lo = a.seg[s], hi = a.seg[s + 1];
  if (lo < 0) lo = 0;
  if (hi > a.T) hi = a.T;
  const int64_t c0 = lo / kLossRows, c1 = hi > lo ? (hi - 1) / kLossRows + 1 : c0;
  const int64_t stride = part_stride(a.E);
  int64_t n = 0;
  for (int64_t c = c0; c < c1; ++c) n += reinterpret_cast<const int32_t*>(a.part + (c + s) * stride)[2 * a.E];
  float term = 0.0f;
  for (int e = threadIdx.x; e < a.E; e += 1024) {
    float p = 0.0f;
    int64_t k = 0;
    for (int64_t c = c0; c < c1; ++c) {
      const float* part = a.part + (c + s) * stride;
      p += part[e];
      k += reinterpret_cast<const int32_t*>(part)[a.E + e];
    }
    const float prob = n > 0 ? p / (float)n : 0.0f;
    a.prob[s * a.E + e] = prob;
    a.counts[s * a.E + e] = (int32_t)k;
    if (n > 0) term += (float)k * (float)a.E / ((float)a.K * (float)n) * prob;
  }
  term = row_sum<64>(term);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.0f;
    for (int i = 0; i < 16; ++i) v += sums[i];
    a.loss[s] = a.alpha * v;
    a.tokens[s] = (int32_t)n;
  }
}

// d logits.  With g_e the gradient of a row's scores:
//   weights, normalised: w_k = c s_k / D, D = sum of the chosen s + 1e-20:
//     g += (c d_k - sum_m (c d_m) s_m / D) / D at the chosen experts
//   loss: share_e has the gradient a_e = alpha d_loss E counts_e / (K n^2):
//     sigmoid: g += (a_e - sum_i a_i share_i) / Z;   softmax: g += a_e
//   sigmoid: dx = g s (1 - s);   softmax: dx = s (g - sum_i g_i s_i)
template <int LPR, int VPL>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(GateBackwardArgs a, int32_t per_wave) {
  extern __shared__ float grads[];           // [rows at once][E], zero but for the row in work
  constexpr int kRows = kGateThreads / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float* grad = grads + sub * a.E;
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (j * LPR + lane < a.E) grad[j * LPR + lane] = 0.0f;
  int64_t in_seg = -2;
  float coef[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) coef[j] = 0.0f;
  for (int i = 0; i < per_wave; ++i) {
    const int64_t t = ((int64_t)blockIdx.x * per_wave + i) * kRows + sub;
    const bool inside = t < a.T;
    const bool real = inside && (a.mask == nullptr || a.mask[t] != 0);
    if (a.d_loss != nullptr && inside) {
      const int64_t sg = segment_of(a.seg, a.S, t);
      if (sg != in_seg) {
        in_seg = sg;
        const bool has = sg >= 0 && sg < a.S && a.tokens[sg] > 0;
        const float n = has ? (float)a.tokens[sg] : 1.0f;
        const float f = has ? a.alpha * a.d_loss[sg] * (float)a.E / ((float)a.K * n) / n : 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int e = j * LPR + lane;
          coef[j] = has && e < a.E ? f * (float)a.counts[sg * a.E + e] : 0.0f;
        }
      }
    }
    float x[VPL], s[VPL];
    load_logits<LPR, VPL>(a.logits, a.dtype, t * a.ld, real ? a.E : 0, lane, x);
    const float z = scores<LPR, VPL>(a.scoring, a.E, lane, x, s);
    if (a.d_weights != nullptr) {
      // the row's scores stand in LDS for a moment, for the chosen to be read
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j * LPR + lane < a.E) grad[j * LPR + lane] = s[j];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      constexpr int kC = (kMaxK + LPR - 1) / LPR;
      int32_t id[kC];
      float sk[kC], gk[kC], D = 0.0f, dot = 0.0f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int k = c * LPR + lane;
        id[c] = real && k < a.K ? a.ids[t * a.K + k] : -1;
        if ((uint32_t)id[c] >= (uint32_t)a.E) id[c] = -1;
        sk[c] = id[c] >= 0 ? grad[id[c]] : 0.0f;
        gk[c] = id[c] >= 0 ? a.scale * a.d_weights[t * a.K + k] : 0.0f;
        D += sk[c];
        dot += gk[c] * sk[c];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j * LPR + lane < a.E) grad[j * LPR + lane] = 0.0f;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (a.normalize) {
        D = row_sum<LPR>(D) + kScoreEps;
        dot = row_sum<LPR>(dot) / D;
#pragma unroll
        for (int c = 0; c < kC; ++c) gk[c] = id[c] >= 0 ? (gk[c] - dot) / D : 0.0f;
      }
      // an expert named twice gets the sum of both, taken in the order of k
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if (c * LPR >= a.K) break;
        float g = 0.0f;
#pragma unroll
        for (int d = 0; d < kC; ++d) {
          const int n = min(LPR, a.K - d * LPR);
          for (int m = 0; m < n; ++m) {
            const int om = __shfl(id[d], m, LPR);
            const float og = __shfl(gk[d], m, LPR);
            if (om == id[c]) g += og;
          }
        }
        if (id[c] >= 0) grad[id[c]] = g;
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    float g[VPL], dot = 0.0f;
    if (a.scoring == kSigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot += coef[j] * (s[j] / z);
      dot = row_sum<LPR>(dot);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * LPR + lane;
      g[j] = e < a.E ? grad[e] : 0.0f;
      g[j] += a.scoring == kSigmoid ? (coef[j] - dot) / z : coef[j];
    }
    if (a.scoring != kSigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot += g[j] * s[j];
      dot = row_sum<LPR>(dot);
    }
    if (inside) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int e = j * LPR + lane;
        if (e < a.E) {
          const float dx = a.scoring == kSigmoid ? g[j] * s[j] * (1.0f - s[j]) : s[j] * (g[j] - dot);
          store_float(a.d_logits, a.dtype, t * a.E + e, real ? dx : 0.0f);
        }
      }
    }
  }
}

// Calls f with the number of values per lane that covers E experts on 64 lanes.
template <typename F>
hipError_t by_width(int32_t E, F f) {
  if (E <= 64) return f(std::integral_constant<int, 1>());
  if (E <= 128) return f(std::integral_constant<int, 2>());
  if (E <= 256) return f(std::integral_constant<int, 4>());
  if (E <= 512) return f(std::integral_constant<int, 8>());
  if (E <= 1024) return f(std::integral_constant<int, 16>());
  if (E <= 2048) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 64>());
}

}  // namespace

int64_t gate_loss_part_bytes(int64_t T, int32_t E, int64_t S) {
  return (ceil_div(T, kLossRows) + S) * part_stride(E) * 4;
}

hipError_t launch_gate(const GateArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  return by_width(a.E, [&](auto vpl) {
    constexpr int LPR = 64, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
    const size_t lds = a.top_groups < a.G ? (size_t)kRows * a.E * 4 : 0;
    gate_kernel<LPR, VPL><<<dim3((unsigned)ceil_div(a.T, kRows)), dim3(kGateThreads), lds, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_gate_loss(const GateArgs& a, hipStream_t stream) {
  if (a.T > 0) {
    const hipError_t err = by_width(a.E, [&](auto vpl) {
      constexpr int LPR = 64, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
      const size_t lds = (size_t)(kRows + 1) * a.E * 4;
      gate_loss_kernel<LPR, VPL><<<dim3((unsigned)ceil_div(a.T, kLossRows)), dim3(kGateThreads), lds, stream>>>(a);
      return hipGetLastError();
    });
    if (err != hipSuccess) return err;
  }
  gate_loss_reduce_kernel<<<dim3((unsigned)a.S), dim3(1024), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBackwardArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  return by_width(a.E, [&](auto vpl) {
    constexpr int LPR = 64, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
    const size_t lds = (size_t)kRows * a.E * 4;
    // a few rows per wave where there are many, so that a segment's counts are read once for them
    const int32_t per_wave = (int32_t)std::min<int64_t>(8, std::max<int64_t>(1, a.T / (kRows * 1024)));
    gate_backward_kernel<LPR, VPL><<<dim3((unsigned)ceil_div(a.T, (int64_t)kRows * per_wave)), dim3(kGateThreads), lds,
                                     stream>>>(a, per_wave);
    return hipGetLastError();
  });
}

}  // namespace eplb
