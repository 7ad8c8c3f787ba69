// The router: scores, the choice of K experts per token, the balance loss and
// the gradients of both.
//
// A row of E logits belongs to LPR lanes of one wave, VPL values each: four
// consecutive experts per lane and turn, so that a row's loads are 16 (or 8)
// bytes a lane and its sums and maxima over the experts are butterflies over
// LPR lanes.  16 lanes to a row for many rows (four rows share the cost of
// every butterfly), 64 for few (shorter chains).
//
// What bounds the choice is arithmetic, not memory: an exponential and a
// division per logit (about 20 instructions), and the selection.  For the K
// largest of a row: every lane's own largest key goes to LDS; the K-th
// largest of those bounds the K-th largest key from below, so that only a
// few more than K keys (11 of 256 for K = 8) can be among the K largest.
// They are compacted into LDS and ranked by counting.
#include "experts_internal.h"

namespace eplb {

namespace {

constexpr int kGateThreads = 256;
constexpr int kLossRows = 32;                // rows of one workgroup of the loss
constexpr int kV = 4;                        // consecutive experts of a lane
constexpr int64_t kManyRows = 2048;          // rows from which 16 lanes take one

// LDS between lanes of one wave: its own operations stay in order, the
// compiler has to keep them so.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), kCtrl, 0xF, 0xF, true));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Reduction over the LPR lanes of a row, every lane gets the result: within
// 16 lanes by moves (neighbours, pairs, quads, halves), then over the rows of
// 16.
template <int LPR, typename Op>
__device__ __forceinline__ float row_reduce(float v, Op op) {
  v = op(v, dpp<0xB1>(v));                   // quad_perm [1, 0, 3, 2]
  v = op(v, dpp<0x4E>(v));                   // quad_perm [2, 3, 0, 1]
  v = op(v, dpp<0x141>(v));                  // row_half_mirror
  v = op(v, dpp<0x140>(v));                  // row_mirror
  if (LPR == 64) v = op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
  return v;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return row_reduce<LPR>(v, [](float a, float b) { return a + b; });
}

template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  return row_reduce<LPR>(v, [](float a, float b) { return fmaxf(a, b); });
}

// 1 / d correctly rounded, for d >= 1: the hardware's approximation, one
// Newton step, and Markstein's correction by the remainder, which rounds
// correctly where no intermediate is denormal.  Half the instructions of the
// general division, and the same bits.
__device__ __forceinline__ float reciprocal(float d) {
  if (d > 0x1p100f) return 1.0f / d;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(fmaf(-d, r, 1.0f), r, r);
  return fmaf(fmaf(-d, r, 1.0f), r, r);
}

// Each step is one correctly rounded 32-bit operation (and the library's
// exponential), so that a choice between near equal keys does not depend on
// how the expression is compiled.
__device__ __forceinline__ float sigmoid(float x) { return reciprocal(1.0f + expf(-x)); }

// Expert of value j of a lane.
template <int LPR>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return (j / kV * LPR + lane) * kV + j % kV;
}

// A row's logits in 32 bits; experts past E hold minus infinity.
template <int LPR, int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int32_t dtype, bool vec, int64_t at, int32_t E,
                                            int lane, float (&x)[VPL]) {
#pragma unroll
  for (int j = 0; j < VPL; j += kV) {
    const int e = expert_of<LPR>(j, lane);
    if (vec && e + kV <= E) {
      if (dtype == kF32) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(static_cast<const float*>(logits) + at + e);
#pragma unroll
        for (int i = 0; i < kV; ++i) x[j + i] = f[i];
      } else {
        const uint2 h = *reinterpret_cast<const uint2*>(static_cast<const u16*>(logits) + at + e);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const u16 v = (u16)((i < 2 ? h.x : h.y) >> (16 * (i & 1)));
          x[j + i] = dtype == kBf16 ? bf16_to_float(v) : f16_to_float(v);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) x[j + i] = e + i < E ? load_as_float(logits, dtype, at + e + i) : -INFINITY;
    }
  }
}

// Scores of a row.  Returns what a share of the balance loss is multiplied
// with (softmax: 1; sigmoid: 1 / (sum of the scores + 1e-20)); softmax also
// leaves the row's maximum and 1 / (its sum + 1e-20), sigmoid the sum.
template <int LPR, int VPL>
__device__ __forceinline__ float scores(int32_t scoring, int32_t E, int lane, const float (&x)[VPL], float (&s)[VPL],
                                        float& m, float& z) {
  if (scoring == kSigmoid) {
    z = 0.0f;
    m = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      s[j] = expert_of<LPR>(j, lane) < E ? sigmoid(x[j]) : 0.0f;
      z += s[j];
    }
    z = row_sum<LPR>(z) + kScoreEps;
    return 1.0f / z;
  }
  m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) m = fmaxf(m, x[j]);
  m = row_max<LPR>(m);
  if (m == -INFINITY) m = 0.0f;              // no expert is allowed: all scores are 0
  z = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    s[j] = expf(x[j] - m);
    z += s[j];
  }
  z = 1.0f / (row_sum<LPR>(z) + kScoreEps);
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[j] *= z;
  return 1.0f;
}

// LDS of one row: its keys for the group scores, the lanes' largest keys and
// the candidates of the choice.  The keys share their place with the rest.
constexpr int row_lds_words(int LPR) { return LPR * 2 + LPR * 2 * 3; }

// Keys of the experts outside the top_groups best groups become minus
// infinity.  The row's keys pass through LDS so that lane g can scan group g;
// the scans start at different places, as the groups' starts may share a bank.
template <int LPR, int VPL>
__device__ __forceinline__ void limit_groups(const GateArgs& a, int lane, float* row, float (&key)[VPL]) {
  constexpr int kC = kMaxGroups / LPR;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = expert_of<LPR>(j, lane);
    if (e < a.E) row[e] = key[j];
  }
  wave_sync();
  const int size = a.E / a.G;
  u64 keep = 0;
  float score[kC];                           // of group c * LPR + lane
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    score[c] = -INFINITY;
    if (c * LPR >= a.G) continue;
    const int g = c * LPR + lane;
    float b1 = -INFINITY, b2 = -INFINITY;
    if (g < a.G) {
      int i = g % size;
      for (int n = 0; n < size; ++n) {
        const float v = row[g * size + i];
        i = i + 1 < size ? i + 1 : 0;
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
    }
    const float sum = a.group_top == 2 ? b1 + b2 : b1;
    score[c] = sum != sum ? -INFINITY : sum;
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    if (c * LPR >= a.G) continue;
    const int g = c * LPR + lane;
    int before = 0;
#pragma unroll
    for (int d = 0; d < kC; ++d) {
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
    const int e = expert_of<LPR>(j, lane);
    const int g = (int)fastdiv_apply((uint32_t)e, a.fd_group);
    if (e < a.E && !(keep >> g & 1)) key[j] = -INFINITY;
  }
  wave_sync();                               // the keys' place is used again
}

// The choice of a row: the K largest keys above minus infinity, ties to the
// lowest expert.  Calls put(rank, expert, score, in) for this lane's share of
// the ranks; in: whether the rank has an expert.  The lanes that call put
// cover every rank below K once.
template <int LPR, int VPL, typename Put>
__device__ __forceinline__ void choose(int32_t K, int lane, float* row, float (&key)[VPL], const float (&s)[VPL],
                                       Put put) {
  constexpr int kCap = 2 * LPR;
  u64* cand = reinterpret_cast<u64*>(row);   // [kCap] ordered key above the complement of the expert
  float* cand_s = row + 2 * kCap;            // [kCap] scores
  u64* top = reinterpret_cast<u64*>(row + 3 * kCap);   // [LPR] the lanes' largest
  if (K <= LPR) {
    // floats as integers of the same order; -0 counts as 0
    auto ordered = [](float v, int e) {
      const uint32_t b = __float_as_uint(v + 0.0f);
      const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
      return (u64)o << 32 | (uint32_t)~e;
    };
    float best = -INFINITY;
    int be = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > best) best = key[j], be = expert_of<LPR>(j, lane);
    const u64 mine = ordered(best, be);
    top[lane] = mine;
    wave_sync();
    int before = 0;
#pragma unroll
    for (int i = 0; i < LPR; ++i) before += top[i] > mine;
    // lane maxima differ unless both are minus infinity; then the bound is that
    const u64 at_rank = __ballot(before == K - 1 && best > -INFINITY);
    const int shift = (threadIdx.x & 63) / LPR * LPR;
    const u64 in_row = LPR == 64 ? at_rank : (at_rank >> shift) & ((u64(1) << (LPR & 63)) - 1);
    const int src = in_row != 0 ? __ffsll((unsigned long long)in_row) - 1 : 0;
    const float bound = in_row != 0 ? __shfl(best, src, LPR) : -INFINITY;
    const int bound_e = __shfl(be, src, LPR);
    int n = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      n += key[j] > bound || (key[j] == bound && bound > -INFINITY && expert_of<LPR>(j, lane) <= bound_e);
    int incl = n;
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) {
      const int v = __shfl_up(incl, d, LPR);
      if (lane >= d) incl += v;
    }
    const int total = __shfl(incl, LPR - 1, LPR);
    if (!__any(total > kCap)) {
      int at = incl - n;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int e = expert_of<LPR>(j, lane);
        if (key[j] > bound || (key[j] == bound && bound > -INFINITY && e <= bound_e)) {
          cand[at] = ordered(key[j], e);
          cand_s[at] = s[j];
          ++at;
        }
      }
      wave_sync();
      int most = total;
#pragma unroll
      for (int d = LPR; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (c * LPR >= most) break;
        const int i = c * LPR + lane;
        const u64 own = i < total ? cand[i] : 0;
        int rank = 0;
        for (int o = 0; o < most; ++o) rank += o < total && cand[o] > own;
        if (i < total && rank < K) put(rank, (int)~(uint32_t)own, cand_s[i], true);
      }
      if (lane >= total && lane < K) put(lane, -1, 0.0f, false);
      wave_sync();
      return;
    }
    wave_sync();
  }
  // one by one: more choices than lanes, or more candidates than places (many
  // equal keys, or fewer lanes than K with any key at all)
  for (int k = 0; k < K; ++k) {
    float best = -INFINITY, bs = 0.0f;
    int be = 1 << 30;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > best) best = key[j], be = expert_of<LPR>(j, lane), bs = s[j];
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) {
      const float ob = __shfl_xor(best, m, LPR), os = __shfl_xor(bs, m, LPR);
      const int oe = __shfl_xor(be, m, LPR);
      if (ob > best || (ob == best && oe < be)) best = ob, be = oe, bs = os;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (expert_of<LPR>(j, lane) == be) key[j] = -INFINITY;
    if (lane == k % LPR) put(k, best > -INFINITY ? be : -1, bs, best > -INFINITY);
  }
}

// One row: the choice (or the given ids), its weights, and, for the loss, the
// row's shares and counts added to the lane's own sums.
template <int LPR, int VPL, bool LOSS>
__device__ __forceinline__ void gate_row(const GateArgs& a, int64_t t, bool real, int lane, float* row, int32_t* cnt,
                                         float (&psum)[VPL]) {
  float x[VPL], s[VPL], m, z;
  load_logits<LPR, VPL>(a.logits, a.dtype, a.vec, t * a.ld, real ? a.E : 0, lane, x);
  const float rz = scores<LPR, VPL>(a.scoring, a.E, lane, x, s, m, z);
  if (LOSS && real) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) psum[j] += s[j] * rz;
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
    const int e = expert_of<LPR>(j, lane);
    float v = a.scoring == kSigmoid ? s[j] : x[j];
    if (a.bias != nullptr && e < a.E) v += a.bias[e];
    key[j] = e < a.E && real && x[j] > -INFINITY && v == v ? v : -INFINITY;
  }
  if (a.top_groups < a.G) limit_groups<LPR, VPL>(a, lane, row, key);
  // a lane holds at most two ranks (K <= LPR)
  float chosen = 0.0f, kept[2] = {0.0f, 0.0f};
  int at[2] = {-1, -1};
  const int64_t out = t * a.K;
  const bool inside = t < a.T;
  choose<LPR, VPL>(a.K, lane, row, key, s, [&](int k, int e, float v, bool in) {
    if (!inside) return;
    a.ids[out + k] = e;
    if (LOSS && in) atomicAdd(&cnt[e], 1);
    chosen += v;
    if (at[0] < 0) at[0] = k, kept[0] = v;
    else at[1] = k, kept[1] = v;
  });
  const float sum = a.normalize ? row_sum<LPR>(chosen) + kScoreEps : 1.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (at[i] >= 0) a.weights[out + at[i]] = a.normalize ? a.scale * kept[i] / sum : a.scale * kept[i];
}

template <int LPR, int VPL>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a, int32_t row_words) {
  extern __shared__ float lds[];             // [rows at once][row_words]
  constexpr int kRows = kGateThreads / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int64_t t = (int64_t)blockIdx.x * kRows + sub;
  float none[VPL];
  const bool real = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
  gate_row<LPR, VPL, false>(a, t, real, lane, lds + sub * row_words, nullptr, none);
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
__global__ __launch_bounds__(kGateThreads) void gate_loss_kernel(GateArgs a, int32_t row_words) {
  extern __shared__ float lds[];             // [rows at once][row_words]: the choice's, then shares; [E] counts
  constexpr int kRows = kGateThreads / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float* row = lds + sub * row_words;
  int32_t* cnt = reinterpret_cast<int32_t*>(lds + kRows * row_words);
  __shared__ int32_t kept;
  // the reduction's tickets (behind the partial sums) start at zero
  for (int64_t s = (int64_t)blockIdx.x * kGateThreads + threadIdx.x; s < a.S; s += (int64_t)gridDim.x * kGateThreads)
    a.ticket[s] = 0;
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
      for (int j = 0; j < VPL; ++j) {
        const int e = expert_of<LPR>(j, lane);
        if (e < a.E) row[e] = psum[j];
      }
      __syncthreads();
      for (int e = threadIdx.x; e < a.E; e += kGateThreads) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) v += lds[i * row_words + e];
        part[e] = v;
        reinterpret_cast<int32_t*>(part)[a.E + e] = cnt[e];
      }
      if (threadIdx.x == 0) reinterpret_cast<int32_t*>(part)[2 * a.E] = kept;
    }
    __syncthreads();
    r = end;
  }
}

constexpr int kReduceThreads = 1024;
constexpr int kReduceParts = kReduceThreads / 64;    // partial sums read at once, 64 experts of each

// 64 experts of segment s: wave w adds the partial sums w, w + 16, ... in
// order, then the 16 sums are added in order.  The last workgroup of a segment
// (by a ticket) adds the loss's terms, in the order of the experts.
__global__ __launch_bounds__(kReduceThreads) void gate_loss_reduce_kernel(GateArgs a, int32_t parts) {
  __shared__ float sums[kReduceParts][64];
  __shared__ int32_t counts[kReduceParts][64];
  __shared__ int32_t rows[kReduceParts];
  const int64_t s = blockIdx.x / parts;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (int)(blockIdx.x % parts) * 64 + lane;
  int64_t lo = a.seg[s], hi = a.seg[s + 1];
  if (lo < 0) lo = 0;
  if (hi > a.T) hi = a.T;
  const int64_t c0 = lo / kLossRows, c1 = hi > lo ? (hi - 1) / kLossRows + 1 : c0;
  const int64_t stride = part_stride(a.E);
  float p = 0.0f;
  int32_t k = 0, n = 0;
#pragma unroll 4
  for (int64_t c = c0 + wave; c < c1; c += kReduceParts) {
    const float* part = a.part + (c + s) * stride;
    if (e < a.E) {
      p += part[e];
      k += reinterpret_cast<const int32_t*>(part)[a.E + e];
    }
    n += reinterpret_cast<const int32_t*>(part)[2 * a.E];
  }
  sums[wave][lane] = p;
  counts[wave][lane] = k;
  if (lane == 0) rows[wave] = n;
  __syncthreads();
  if (wave == 0) {
    p = 0.0f;
    k = n = 0;
#pragma unroll
    for (int w = 0; w < kReduceParts; ++w) p += sums[w][lane], k += counts[w][lane], n += rows[w];
    const float prob = n > 0 ? p / (float)n : 0.0f;
    float term = 0.0f;
    if (e < a.E) {
      a.prob[s * a.E + e] = prob;
      a.counts[s * a.E + e] = k;
      if (n > 0) term = (float)k * (float)a.E / ((float)a.K * (float)n) * prob;
    }
    term = row_sum<64>(term);
    if (lane == 0) {
      a.terms[s * parts + blockIdx.x % parts] = term;
      if (blockIdx.x % parts == 0) a.tokens[s] = n;
      __threadfence();
      if (atomicAdd(&a.ticket[s], 1) == parts - 1) {
        __threadfence();
        float v = 0.0f;
        for (int i = 0; i < parts; ++i) v += __hip_atomic_load(&a.terms[s * parts + i], __ATOMIC_RELAXED,
                                                               __HIP_MEMORY_SCOPE_AGENT);
        a.loss[s] = a.alpha * v;
      }
    }
  }
}

// d logits.  With g_e the gradient of a row's scores:
//   weights, normalised: w_k = c s_k / D, D = sum of the chosen s + 1e-20:
//     g += (c d_k - sum_m (c d_m) s_m / D) / D at the chosen experts
//   loss: share_e has the gradient a_e = alpha d_loss E counts_e / (K n^2):
//     sigmoid: g += (a_e - sum_i a_i share_i) / Z;   softmax: g += a_e
//   sigmoid: dx = g s (1 - s);   softmax: dx = s (g - sum_i g_i s_i)
// One read of the logits and one write of their gradients; the scores are
// computed again rather than kept by the forward pass (as many bytes as the
// logits, written and read).
template <int LPR, int VPL>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(GateBackwardArgs a, int32_t per_group) {
  extern __shared__ float grads[];           // [rows at once][E rounded up to 4], zero but for the row in work
  constexpr int kRows = kGateThreads / LPR;
  constexpr int kC = LPR == 64 ? 1 : kMaxK / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float* grad = grads + sub * ((a.E + 3) / 4 * 4 + 4);
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (expert_of<LPR>(j, lane) < a.E) grad[expert_of<LPR>(j, lane)] = 0.0f;
  int64_t seg_end = -1;                      // where the coefficients in registers stop to hold
  float coef[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) coef[j] = 0.0f;
  for (int i = 0; i < per_group; ++i) {
    const int64_t t = ((int64_t)blockIdx.x * per_group + i) * kRows + sub;
    const bool inside = t < a.T;
    const bool real = inside && (a.mask == nullptr || a.mask[t] != 0);
    float x[VPL], s[VPL], m, z;
    load_logits<LPR, VPL>(a.logits, a.dtype, a.vec, t * a.ld, real ? a.E : 0, lane, x);
    int32_t id[kC];
    float gk[kC], xk[kC];
    if (a.d_weights != nullptr) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int k = c * LPR + lane;
        id[c] = real && k < a.K ? a.ids[t * a.K + k] : -1;
        if ((uint32_t)id[c] >= (uint32_t)a.E) id[c] = -1;
        gk[c] = id[c] >= 0 ? a.scale * a.d_weights[t * a.K + k] : 0.0f;
        xk[c] = id[c] >= 0 ? load_as_float(a.logits, a.dtype, t * a.ld + id[c]) : -INFINITY;
      }
    }
    if (a.d_loss != nullptr && inside && t >= seg_end) {
      const int64_t sg = segment_of(a.seg, a.S, t);
      seg_end = piece_end(a.seg, a.S, sg, t, a.T);
      const bool has = sg >= 0 && sg < a.S && a.tokens[sg] > 0;
      const float n = has ? (float)a.tokens[sg] : 1.0f;
      const float f = has ? a.alpha * a.d_loss[sg] * (float)a.E / ((float)a.K * n) / n : 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int e = expert_of<LPR>(j, lane);
        coef[j] = has && e < a.E ? f * (float)a.counts[sg * a.E + e] : 0.0f;
      }
    }
    const float rz = scores<LPR, VPL>(a.scoring, a.E, lane, x, s, m, z);
    if (a.d_weights != nullptr) {
      float sk[kC], D = 0.0f, dot = 0.0f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if (c * LPR >= a.K) break;
        sk[c] = id[c] < 0 ? 0.0f : a.scoring == kSigmoid ? sigmoid(xk[c]) : expf(xk[c] - m) * z;
        D += sk[c];
        dot += gk[c] * sk[c];
      }
      if (a.normalize) {
        const float rd = 1.0f / (row_sum<LPR>(D) + kScoreEps);
        dot = row_sum<LPR>(dot) * rd;
#pragma unroll
        for (int c = 0; c < kC; ++c) gk[c] = id[c] >= 0 ? (gk[c] - dot) * rd : 0.0f;
      }
      // an expert named twice gets the sum of both, taken in the order of k
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if (c * LPR >= a.K) break;
        float g = 0.0f;
#pragma unroll
        for (int d = 0; d < kC; ++d) {
          const int n = min(LPR, a.K - d * LPR);
          for (int q = 0; q < n; ++q) {
            const int om = __shfl(id[d], q, LPR);
            const float og = __shfl(gk[d], q, LPR);
            if (om == id[c]) g += og;
          }
        }
        if (id[c] >= 0) grad[id[c]] = g;
      }
      wave_sync();
    }
    float g[VPL], dot = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = expert_of<LPR>(j, lane);
      g[j] = e < a.E ? grad[e] : 0.0f;
    }
    if (a.d_weights != nullptr) {            // the place of the chosen is zero again for the next row
      wave_sync();
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (c * LPR < a.K && id[c] >= 0) grad[id[c]] = 0.0f;
      wave_sync();
    }
    if (a.scoring == kSigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) dot += coef[j] * s[j];
      dot = row_sum<LPR>(dot) * rz;
#pragma unroll
      for (int j = 0; j < VPL; ++j) g[j] = (g[j] + (coef[j] - dot) * rz) * s[j] * (1.0f - s[j]);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        g[j] += coef[j];
        dot += g[j] * s[j];
      }
      dot = row_sum<LPR>(dot);
#pragma unroll
      for (int j = 0; j < VPL; ++j) g[j] = s[j] * (g[j] - dot);
    }
    if (!inside) continue;
#pragma unroll
    for (int j = 0; j < VPL; j += kV) {
      const int e = expert_of<LPR>(j, lane);
      if (!real) g[j] = g[j + 1] = g[j + 2] = g[j + 3] = 0.0f;
      if (a.vec_out && e + kV <= a.E) {
        if (a.dtype == kF32) {
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.d_logits) + t * a.E + e) = f32x4{g[j], g[j + 1], g[j + 2], g[j + 3]};
        } else {
          uint2 w;
          if (a.dtype == kBf16) {
            w.x = float_to_bf16(g[j]) | (uint32_t)float_to_bf16(g[j + 1]) << 16;
            w.y = float_to_bf16(g[j + 2]) | (uint32_t)float_to_bf16(g[j + 3]) << 16;
          } else {
            w.x = float_to_f16(g[j]) | (uint32_t)float_to_f16(g[j + 1]) << 16;
            w.y = float_to_f16(g[j + 2]) | (uint32_t)float_to_f16(g[j + 3]) << 16;
          }
          *reinterpret_cast<uint2*>(static_cast<u16*>(a.d_logits) + t * a.E + e) = w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (e + i < a.E) store_float(a.d_logits, a.dtype, t * a.E + e + i, g[j + i]);
      }
    }
  }
}

// Calls f with the lanes per row and the values per lane that cover E experts:
// 16 lanes for E <= 512 and K <= 16 where there are rows enough to fill the
// chip with four to a wave, else 64.
template <typename F>
hipError_t by_width(int64_t T, int32_t E, int32_t K, F f) {
  typedef std::integral_constant<int, 16> L16;
  typedef std::integral_constant<int, 64> L64;
  if (E <= 512 && K <= 16 && T >= kManyRows) {
    if (E <= 64) return f(L16(), std::integral_constant<int, 4>());
    if (E <= 128) return f(L16(), std::integral_constant<int, 8>());
    if (E <= 256) return f(L16(), std::integral_constant<int, 16>());
    return f(L16(), std::integral_constant<int, 32>());
  }
  if (E <= 256) return f(L64(), std::integral_constant<int, 4>());
  if (E <= 512) return f(L64(), std::integral_constant<int, 8>());
  if (E <= 1024) return f(L64(), std::integral_constant<int, 16>());
  if (E <= 2048) return f(L64(), std::integral_constant<int, 32>());
  return f(L64(), std::integral_constant<int, 64>());
}

// LDS words of a row in the choice; rows start 8 banks apart.
int32_t choice_words(int lpr, int32_t E, bool groups) {
  const int32_t n = std::max(row_lds_words(lpr), groups ? E : 0);
  return (n + 31) / 32 * 32 + 8;
}

int64_t loss_parts(int32_t E) { return ceil_div(E, 64); }

bool aligned4(const void* p, int32_t dtype, int64_t ld) {
  return ((uintptr_t)p & (uintptr_t)(4 * dtype_size(dtype) - 1)) == 0 && ld % 4 == 0;
}

}  // namespace

int64_t gate_loss_part_bytes(int64_t T, int32_t E, int64_t S) {
  return ((ceil_div(T, kLossRows) + S) * part_stride(E) + S * (loss_parts(E) + 1)) * 4;
}

hipError_t launch_gate(const GateArgs& args, hipStream_t stream) {
  if (args.T == 0) return hipSuccess;
  GateArgs a = args;
  a.vec = aligned4(a.logits, a.dtype, a.ld);
  return by_width(a.T, a.E, a.K, [&](auto lpr, auto vpl) {
    constexpr int LPR = decltype(lpr)::value, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
    const int32_t words = choice_words(LPR, a.E, a.top_groups < a.G);
    gate_kernel<LPR, VPL><<<dim3((unsigned)ceil_div(a.T, kRows)), dim3(kGateThreads), (size_t)kRows * words * 4, stream>>>(
        a, words);
    return hipGetLastError();
  });
}

hipError_t launch_gate_loss(const GateArgs& args, hipStream_t stream) {
  GateArgs a = args;
  a.vec = aligned4(a.logits, a.dtype, a.ld);
  const int64_t parts = loss_parts(a.E);
  a.terms = a.part + (ceil_div(a.T, kLossRows) + a.S) * part_stride(a.E);
  a.ticket = reinterpret_cast<int32_t*>(a.terms + a.S * parts);
  const hipError_t err = by_width(a.T, a.E, a.K, [&](auto lpr, auto vpl) {
    constexpr int LPR = decltype(lpr)::value, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
    const int32_t words = choice_words(LPR, a.E, true);      // the shares' sums pass through the same place
    const unsigned grid = (unsigned)std::max<int64_t>(1, ceil_div(a.T, kLossRows));
    gate_loss_kernel<LPR, VPL><<<dim3(grid), dim3(kGateThreads), ((size_t)kRows * words + a.E) * 4, stream>>>(a, words);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  gate_loss_reduce_kernel<<<dim3((unsigned)(a.S * parts)), dim3(kReduceThreads), 0, stream>>>(a, (int32_t)parts);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBackwardArgs& args, hipStream_t stream) {
  if (args.T == 0) return hipSuccess;
  GateBackwardArgs a = args;
  a.vec = aligned4(a.logits, a.dtype, a.ld);
  a.vec_out = aligned4(a.d_logits, a.dtype, a.E);
  return by_width(a.T, a.E, a.K, [&](auto lpr, auto vpl) {
    constexpr int LPR = decltype(lpr)::value, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
    const size_t lds = (size_t)kRows * ((a.E + 3) / 4 * 4 + 4) * 4;
    // a few rows per lane group where there are many, so that a segment's counts are read once for them
    const int32_t per_group = (int32_t)std::min<int64_t>(8, std::max<int64_t>(1, a.T / (kRows * 512)));
    gate_backward_kernel<LPR, VPL><<<dim3((unsigned)ceil_div(a.T, (int64_t)kRows * per_group)), dim3(kGateThreads),
                                     lds, stream>>>(a, per_group);
    return hipGetLastError();
  });
}

}  // namespace eplb
