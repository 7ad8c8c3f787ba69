// The router: scores, the choice of K experts per token, the balance loss and
// the gradients of both.
//
// A row of E logits belongs to LPR lanes of one wave, VPL values each: four
// consecutive experts per lane and turn, so that a row's loads are 16 (or 8)
// bytes a lane and its sums and maxima over the experts are butterflies over
// LPR lanes.  16 lanes to a row for many rows (four rows share the cost of
// every butterfly), 64 for few (shorter chains).
//
// What bounds the choice is arithmetic, not memory: 76 vector instructions per
// logit (the vector units are busy for 79 % of the kernel's time), of which an
// exponential and a division are about 20 and the group limit and the selection
// the rest, so all of it is free of branches that differ between lanes.  For the K largest of a row:
// the largest keys of 16 parts of it go to LDS; the K-th largest of those
// bounds the K-th largest key from below, so that only a few more than K keys
// (11 of 256 for K = 8) can be among the K largest.  They are compacted into
// LDS and ranked by counting.
//
// Measured, 16384 tokens, 256 experts in 8 groups (4 taken), 8 chosen,
// sigmoid: the choice 14.9 us from bfloat16 logits (9.5 MB: 0.63 TB/s); with
// the loss 24.3 + 7.3 us from 32-bit ones, the gradient 17.0 us (34 MB: 2.0
// TB/s; vector units busy for 39 %, its two waves to a SIMD wait for 62 % of their
// time).  One token: 3.4 us, the chain of its butterflies.
#include "experts_internal.h"

namespace eplb {

namespace {

constexpr int kGateThreads = 256;
constexpr int kLossThreads = 512;
constexpr int kLossBlocks = 512;             // workgroups of the loss, at most
constexpr int kV = 4;                        // consecutive experts of a lane
constexpr int kParts = 16;                   // parts of a row whose maxima bound the choice

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

template <int kCtrl, int kRowMask>
__device__ __forceinline__ int dpp_or_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, kRowMask, 0xF, false);
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

// Sum over the row's lanes up to and with this one.
template <int LPR>
__device__ __forceinline__ int row_scan(int v) {
  v += dpp_or_zero<0x111, 0xF>(v);           // row_shr 1, 2, 4, 8
  v += dpp_or_zero<0x112, 0xF>(v);
  v += dpp_or_zero<0x114, 0xF>(v);
  v += dpp_or_zero<0x118, 0xF>(v);
  if (LPR == 64) {
    v += dpp_or_zero<0x142, 0xA>(v);         // row_bcast 15 into rows 1 and 3
    v += dpp_or_zero<0x143, 0xC>(v);         // row_bcast 31 into rows 2 and 3
  }
  return v;
}

// The value of the row's last lane.
template <int LPR>
__device__ __forceinline__ int row_last(int v) {
  if (LPR == 64) return __builtin_amdgcn_readlane(v, 63);
  return __builtin_amdgcn_mov_dpp(v, 0x15F, 0xF, 0xF, true);   // row_newbcast 15
}

// 1 / d correctly rounded, for 1 <= d <= 2^126: the hardware's approximation,
// one Newton step, and Markstein's correction by the remainder, which rounds
// correctly where no intermediate is denormal (compared with the division for
// every 32-bit d of that range).  Half the instructions of the general division,
// and the same bits.
__device__ __forceinline__ float reciprocal(float d) {
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(fmaf(-d, r, 1.0f), r, r);
  return fmaf(fmaf(-d, r, 1.0f), r, r);
}

// Each step is one correctly rounded 32-bit operation (and the library's
// exponential), so that a choice between near equal keys does not depend on
// how the expression is compiled.
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Expert of value j of a lane.
template <int LPR>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return (j / kV * LPR + lane) * kV + j % kV;
}

// A row's logits in 32 bits; experts past E hold minus infinity.  `on`:
// whether the row is read at all.  vec: E and the rows' addresses are
// multiples of four logits.
template <int LPR, int VPL>
__device__ __forceinline__ void load_logits(const void* logits, int32_t dtype, bool vec, int64_t at, int32_t E, bool on,
                                            int lane, float (&x)[VPL]) {
  if (!on) at = 0;                           // row 0 is always there
  const int end = on ? E : 0;
  if (vec) {
    if (dtype == kF32) {
      const float* p = static_cast<const float*>(logits) + at;
#pragma unroll
      for (int j = 0; j < VPL; j += kV) {
        const f32x4 f = *reinterpret_cast<const f32x4*>(p + min(expert_of<LPR>(j, lane), E - kV));
#pragma unroll
        for (int k = 0; k < kV; ++k) x[j + k] = f[k];
      }
    } else {
      const u16* p = static_cast<const u16*>(logits) + at;
      uint2 h[VPL / kV];
#pragma unroll
      for (int j = 0; j < VPL; j += kV)
        h[j / kV] = *reinterpret_cast<const uint2*>(p + min(expert_of<LPR>(j, lane), E - kV));
      if (dtype == kBf16) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const uint32_t w = j % kV < 2 ? h[j / kV].x : h[j / kV].y;
          x[j] = __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
        }
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) x[j] = f16_to_float((u16)((j % kV < 2 ? h[j / kV].x : h[j / kV].y) >> (16 * (j & 1))));
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = expert_of<LPR>(j / kV * kV, lane) < end ? x[j] : -INFINITY;
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = load_as_float(logits, dtype, at + min(expert_of<LPR>(j, lane), E - 1));
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = expert_of<LPR>(j, lane) < end ? x[j] : -INFINITY;
  }
}

// Scores of a row.  Returns what a share of the balance loss is multiplied
// with (softmax: 1; sigmoid: 1 / (sum of the scores + 1e-20)); softmax also
// leaves the row's maximum and 1 / (its sum + 1e-20).
template <int LPR, int VPL>
__device__ __forceinline__ float scores(int32_t scoring, const float (&x)[VPL], float (&s)[VPL], float& m, float& z) {
  if (scoring == kSigmoid) {
    m = z = 0.0f;
    bool far = false;                        // some logit is below -87
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const float d = 1.0f + expf(-x[j]);
      const float r = reciprocal(d);
      s[j] = x[j] == -INFINITY ? 0.0f : r;
      far |= (d > 0x1p126f) & (x[j] > -INFINITY);
    }
    if (__any(far)) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) s[j] = sigmoid(x[j]);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) z += s[j];
    return 1.0f / (row_sum<LPR>(z) + kScoreEps);
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

// The two largest of both pairs, each in order.
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}

template <int kCtrl>
__device__ __forceinline__ void merge2_dpp(float& a1, float& a2) {
  const float b1 = dpp<kCtrl>(a1), b2 = dpp<kCtrl>(a2);
  merge2(a1, a2, b1, b2);
}

constexpr int kGroupWords = kMaxGroups + 4;  // LDS words of the groups' scores

// Keys of the experts outside the top_groups best groups become minus
// infinity.  The groups' scores meet in LDS; lane g then ranks group g.
template <int LPR, int VPL>
__device__ __forceinline__ void limit_groups(const GateArgs& a, int lane, float* row, float (&key)[VPL]) {
  constexpr int kC = kMaxGroups / LPR;
  const int size = a.E / a.G;
  const int lanes = size / kV;               // lanes of a group, where it has whole ones
  const bool whole = size % kV == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
  auto score = [&](float b1, float b2) {
    const float v = a.group_top == 2 ? b1 + b2 : b1;
    return v == v ? v : -INFINITY;           // +infinity and -infinity met
  };
  if (lane < 4) row[a.G + lane] = -INFINITY; // the scores are read by fours
  if (whole) {
    // a group is `lanes` neighbouring lanes in one turn of the row
#pragma unroll
    for (int j = 0; j < VPL; j += kV) {
      float b1 = fmaxf(key[j], key[j + 1]), b2 = fminf(key[j], key[j + 1]);
      merge2(b1, b2, fmaxf(key[j + 2], key[j + 3]), fminf(key[j + 2], key[j + 3]));
      if (lanes > 1) merge2_dpp<0xB1>(b1, b2);
      if (lanes > 2) merge2_dpp<0x4E>(b1, b2);
      if (lanes > 4) merge2_dpp<0x141>(b1, b2);
      if (lanes > 8) merge2_dpp<0x140>(b1, b2);
      const int e = expert_of<LPR>(j, lane);
      if (e < a.E) row[fastdiv_apply((uint32_t)e, a.fd_group)] = score(b1, b2);
    }
  } else {
    // group g by lane g, through LDS; the scans start at different places, as
    // the groups' starts may share a bank
    float* keys = row + kGroupWords;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = expert_of<LPR>(j, lane);
      if (e < a.E) keys[e] = key[j];
    }
    wave_sync();
    for (int g = lane; g < a.G; g += LPR) {
      float b1 = -INFINITY, b2 = -INFINITY;
      const int first = g % size;
#pragma unroll 4
      for (int n = 0; n < size; ++n) {
        const int i = first + n;
        merge2(b1, b2, keys[g * size + (i < size ? i : i - size)], -INFINITY);
      }
      row[g] = score(b1, b2);
    }
  }
  wave_sync();
  u64 keep = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    if (c * LPR >= a.G) break;
    const int g = c * LPR + lane;
    const float own = row[min(g, a.G)];
    int before = 0;
    for (int i = 0; i < a.G; i += 4) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(row + i);
#pragma unroll
      for (int u = 0; u < 4; ++u) before += (int)(o[u] > own) | ((int)(o[u] == own) & (int)(i + u < g));
    }
    const u64 all = __ballot(g < a.G && before < a.top_groups);
    const int shift = (threadIdx.x & 63) / LPR * LPR;
    const u64 mine = LPR == 64 ? all : (all >> shift) & ((u64(1) << (LPR & 63)) - 1);
    keep |= mine << (c * LPR & 63);
  }
  if (whole) {
#pragma unroll
    for (int j = 0; j < VPL; j += kV) {
      const uint32_t g = fastdiv_apply((uint32_t)expert_of<LPR>(j, lane), a.fd_group);
      const bool in = keep >> (g & 63) & 1;  // experts past E hold minus infinity already
#pragma unroll
      for (int k = 0; k < kV; ++k) key[j + k] = in ? key[j + k] : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const uint32_t g = fastdiv_apply((uint32_t)expert_of<LPR>(j, lane), a.fd_group);
      key[j] = keep >> (g & 63) & 1 ? key[j] : -INFINITY;
    }
  }
  wave_sync();                               // the place is used again
}

// LDS words of the choice of one row (kCap candidates, a place for what is
// none, their scores, the parts' maxima).
constexpr int choose_cap(int LPR) { return LPR == 16 ? 48 : 64; }
constexpr int choose_lds_words(int LPR) { return choose_cap(LPR) * 3 + 4 + kParts; }

// The choice of a row: the K largest keys above minus infinity, ties to the
// lowest expert.  Calls put(slot, rank, expert, score, in) for this lane's
// share of the ranks, at most one per slot (below kSlots); in: whether the rank has an
// expert.  The row's lanes cover every rank below K once.
template <int LPR, int VPL, typename Put>
__device__ __forceinline__ void choose(int32_t K, int lane, float* row, float (&key)[VPL], const float (&s)[VPL],
                                       Put put) {
  constexpr int kCap = choose_cap(LPR), kSlots = kCap / LPR;
  u64* cand = reinterpret_cast<u64*>(row);   // [kCap + 1] ordered key above the complement of the expert
  float* cand_s = row + 2 * kCap + 2;        // [kCap + 1] scores
  float* top = row + 3 * kCap + 4;           // [kParts]
  if (K <= kParts) {
    float best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = fmaxf(best, key[j]);
    if (LPR == 64) {                         // lanes l, l + 16, l + 32 and l + 48 make a part
      best = fmaxf(best, __shfl_xor(best, 16));
      best = fmaxf(best, __shfl_xor(best, 32));
    }
    top[lane % kParts] = best;
#pragma unroll
    for (int i = 0; i < kCap; i += LPR) cand[i + lane] = 0;
    wave_sync();
    int above = 0;                           // parts whose maximum is as large
#pragma unroll
    for (int i = 0; i < kParts; ++i) above += top[i] >= best;
    const float bound = fmaxf(row_max<LPR>(above >= K ? best : -INFINITY), -3.4028235e38f);
    int n = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) n += key[j] >= bound;
    const int incl = row_scan<LPR>(n);
    const int total = row_last<LPR>(incl);
    if (!__any(total > kCap)) {
      int at = incl - n;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        // floats as integers of the same order; -0 counts as 0
        const uint32_t b = __float_as_uint(key[j] + 0.0f);
        const uint32_t o = b ^ (uint32_t)((int32_t)b >> 31 | (int32_t)0x80000000);
        const bool in = key[j] >= bound;
        const int to = in ? at : kCap;
        cand[to] = (u64)o << 32 | (uint32_t)~expert_of<LPR>(j, lane);
        cand_s[to] = s[j];
        at += in;
      }
      wave_sync();
      int most = total;
      if (LPR == 16)
        most = max(max(__builtin_amdgcn_readlane(total, 0), __builtin_amdgcn_readlane(total, 16)),
                   max(__builtin_amdgcn_readlane(total, 32), __builtin_amdgcn_readlane(total, 48)));
      most = __builtin_amdgcn_readfirstlane(most);
#pragma unroll
      for (int c = 0; c < kSlots; ++c) {
        const int i = c * LPR + lane;
        if (c * LPR >= most) break;
        const u64 own = cand[i];
        int rank = 0;
        for (int o = 0; o < most; o += 4) {  // kCap is a multiple of 4, unused places are 0
#pragma unroll
          for (int u = 0; u < 4; ++u) rank += cand[o + u] > own;
        }
        if (i < total && rank < K) put(c, rank, (int)~(uint32_t)own, cand_s[i], true);
      }
      if (lane >= total && lane < K) put(kSlots - 1, lane, -1, 0.0f, false);
      wave_sync();
      return;
    }
    wave_sync();
  }
  // one by one: more choices than parts, or more candidates than places (many
  // equal keys, or fewer parts than K with any key at all)
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
    if (lane == k % LPR) put(0, k, best > -INFINITY ? be : -1, bs, best > -INFINITY);
  }
}

// One row: the choice (or the given ids), its weights, and, for the loss, the
// row's shares and counts added to the lane's own sums.
template <int LPR, int VPL, bool LOSS>
__device__ __forceinline__ void gate_row(const GateArgs& a, int64_t t, bool real, int lane, float* row, int32_t* cnt,
                                         float (&psum)[VPL]) {
  float x[VPL], s[VPL], m, z;
  load_logits<LPR, VPL>(a.logits, a.dtype, a.vec, t * a.ld, a.E, real, lane, x);
  float key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) key[j] = 0.0f;
  if (a.bias != nullptr) {
    if (a.vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += kV) {
        const f32x4 b = *reinterpret_cast<const f32x4*>(a.bias + min(expert_of<LPR>(j, lane), a.E - kV));
#pragma unroll
        for (int k = 0; k < kV; ++k) key[j + k] = b[k];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = a.bias[min(expert_of<LPR>(j, lane), a.E - 1)];
    }
  }
  const float rz = scores<LPR, VPL>(a.scoring, x, s, m, z);
  if (LOSS) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) psum[j] += real ? s[j] * rz : 0.0f;
    if (a.given) {
      if (real)
        for (int k = lane; k < a.K; k += LPR) {
          const int32_t e = a.ids[t * a.K + k];
          if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&cnt[e], 1);
        }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const float v = (a.scoring == kSigmoid ? s[j] : x[j]) + key[j];
    key[j] = ((x[j] > -INFINITY) & (v == v)) ? v : -INFINITY;
  }
  if (a.top_groups < a.G) limit_groups<LPR, VPL>(a, lane, row, key);
  constexpr int kSlots = choose_cap(LPR) / LPR;
  float kept[kSlots], chosen = 0.0f;
  int at[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) kept[i] = 0.0f, at[i] = -1;
  const int64_t out = t * a.K;
  const bool inside = t < a.T;
  choose<LPR, VPL>(a.K, lane, row, key, s, [&](int slot, int k, int e, float v, bool in) {
    if (inside) a.ids[out + k] = e;
    if (LOSS && in && inside) atomicAdd(&cnt[e], 1);
    at[slot] = inside ? k : -1;
    kept[slot] = v;
  });
#pragma unroll
  for (int i = 0; i < kSlots; ++i) chosen += kept[i];
  const float sum = a.normalize ? row_sum<LPR>(chosen) + kScoreEps : 1.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (at[i] >= 0) a.weights[out + at[i]] = a.normalize ? a.scale * kept[i] / sum : a.scale * kept[i];
}

template <int LPR, int VPL>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a, int32_t row_words) {
  extern __shared__ __attribute__((aligned(16))) float lds[];     // [rows at once][row_words]
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

// Whether 16 lanes take a row (else 64): four rows then share every butterfly
// and every step of the selection, but a lane holds four times the experts, so
// the rows have to fill the chip with a quarter of the waves.  Kernel times of
// the choice, 16 lanes and 64, 8 of E (6 of 64): E = 64, 2048 rows: 3.4 and 3.8
// us; E = 128, 2048: 4.2 and 3.9, 4096: 4.3 and 4.7; E = 256, 4096: 5.7 and
// 4.7, 8192: 6.5 and 6.9, 16384: 9.1 and 11.1.  With the loss the same turn
// (E = 256, 4096 rows: 14.6 and 17.0, 2048: 14.4 and 12.4).  Past 256 experts
// 16 lanes gain nothing (E = 512, K = 16, 16384 rows: 40.9 and 38.2).
__host__ __device__ inline bool narrow_rows(int64_t T, int32_t E) { return E <= 256 && T >= 32 * (int64_t)E; }

// Rows of one workgroup of the loss: one row to a lane group where there are
// few, else as many as make kLossBlocks workgroups (and partial sums).
int32_t loss_chunk(int64_t T, int32_t E) {
  const int64_t least = kLossThreads / (narrow_rows(T, E) ? 16 : 64);
  return (int32_t)std::max<int64_t>(least, ceil_div(ceil_div(T, kLossBlocks), least) * least);
}

// Workgroup c takes rows c * chunk on, piece by piece where a segment ends.
// The piece of segment s goes to partial sum c + s: two pieces never share one,
// as each next piece has a larger c or a larger s.
template <int LPR, int VPL>
__global__ __launch_bounds__(kLossThreads) void gate_loss_kernel(GateArgs a, int32_t row_words, int32_t chunk) {
  // [rows at once][row_words]: the choice's, then shares; [E] counts
  extern __shared__ __attribute__((aligned(16))) float lds[];
  constexpr int kRows = kLossThreads / LPR;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float* row = lds + sub * row_words;
  int32_t* cnt = reinterpret_cast<int32_t*>(lds + kRows * row_words);
  __shared__ int32_t kept;
  // the reduction's tickets (behind the partial sums) start at zero
  for (int64_t s = (int64_t)blockIdx.x * kLossThreads + threadIdx.x; s < a.S; s += (int64_t)gridDim.x * kLossThreads)
    a.ticket[s] = 0;
  const int64_t row0 = (int64_t)blockIdx.x * chunk;
  const int64_t row1 = row0 + chunk < a.T ? row0 + chunk : a.T;
  for (int64_t r = row0; r < row1;) {
    const int64_t s = segment_of(a.seg, a.S, r);
    const int64_t end = piece_end(a.seg, a.S, s, r, row1);
    for (int e = threadIdx.x; e < a.E; e += kLossThreads) cnt[e] = 0;
    if (threadIdx.x == 0) kept = 0;
    __syncthreads();
    float psum[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) psum[j] = 0.0f;
    int mine = 0;
    for (int64_t t0 = r; t0 < end; t0 += kRows) {
      const int64_t t = t0 + sub;
      const bool real = t < end && (a.mask == nullptr || a.mask[t] != 0);
      // the lane's number is not the same to the compiler in every turn: what
      // it would keep for all of them (addresses, comparisons, the bias) takes
      // more registers than there are
      int turn_lane = lane;
      asm volatile("" : "+v"(turn_lane));
      gate_row<LPR, VPL, true>(a, t < end ? t : a.T, real, turn_lane, row, cnt, psum);
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
      for (int e = threadIdx.x; e < a.E; e += kLossThreads) {
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
__global__ __launch_bounds__(kReduceThreads) void gate_loss_reduce_kernel(GateArgs a, int32_t parts, int32_t chunk) {
  __shared__ float sums[kReduceParts][64];
  __shared__ int32_t counts[kReduceParts][64];
  __shared__ int32_t rows[kReduceParts];
  const int64_t s = blockIdx.x / parts;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (int)(blockIdx.x % parts) * 64 + lane;
  int64_t lo = a.seg[s], hi = a.seg[s + 1];
  if (lo < 0) lo = 0;
  if (hi > a.T) hi = a.T;
  const int32_t c0 = (int32_t)(lo / chunk), c1 = hi > lo ? (int32_t)((hi - 1) / chunk) + 1 : c0;
  const int64_t stride = part_stride(a.E);
  const int at = e < a.E ? e : a.E - 1;
  float p = 0.0f;
  int32_t k = 0, n = 0;
  for (int32_t c = c0 + wave; c < c1; c += 8 * kReduceParts) {
    float vp[8];
    int32_t vk[8], vn[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {            // all loads in flight at once; past the end the last one again
      const int32_t cc = c + u * kReduceParts;
      const float* part = a.part + (min(cc, c1 - 1) + s) * stride;
      vp[u] = part[at];
      vk[u] = reinterpret_cast<const int32_t*>(part)[a.E + at];
      vn[u] = reinterpret_cast<const int32_t*>(part)[2 * a.E];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = c + u * kReduceParts < c1;
      p += in ? vp[u] : 0.0f;
      k += in ? vk[u] : 0;
      n += in ? vn[u] : 0;
    }
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
  // [rows at once][E rounded up to 4], zero but for the row in work
  extern __shared__ __attribute__((aligned(16))) float grads[];
  constexpr int kRows = kGateThreads / LPR;
  constexpr int kC = 1;                      // K <= LPR
  const int first_lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float* grad = grads + sub * ((a.E + 3) / 4 * 4 + 4);
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (expert_of<LPR>(j, first_lane) < a.E) grad[expert_of<LPR>(j, first_lane)] = 0.0f;
  int64_t seg_end = -1;                      // where the coefficients in registers stop to hold
  float coef[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) coef[j] = 0.0f;
  for (int i = 0; i < per_group; ++i) {
    int lane = first_lane;                   // as in the loss: nothing is kept from turn to turn
    asm volatile("" : "+v"(lane));
    const int64_t t = ((int64_t)blockIdx.x * per_group + i) * kRows + sub;
    const bool inside = t < a.T;
    const bool real = inside && (a.mask == nullptr || a.mask[t] != 0);
    float x[VPL], s[VPL], m, z;
    load_logits<LPR, VPL>(a.logits, a.dtype, a.vec, t * a.ld, a.E, real, lane, x);
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
    const float rz = scores<LPR, VPL>(a.scoring, x, s, m, z);
    if (a.d_weights != nullptr) {
      float sk[kC], D = 0.0f, dot = 0.0f;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
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
      // the chosen experts' gradients through LDS; an expert named twice (its
      // place then holds another lane's mark) gets the sum in the order of k
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (id[c] >= 0) grad[id[c]] = __int_as_float(c * LPR + lane);
      wave_sync();
      bool twice = false;
#pragma unroll
      for (int c = 0; c < kC; ++c) twice |= id[c] >= 0 && __float_as_int(grad[id[c] < 0 ? 0 : id[c]]) != c * LPR + lane;
      wave_sync();
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (id[c] >= 0) grad[id[c]] = gk[c];
      wave_sync();
      if (__any(twice)) {
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (id[c] >= 0) grad[id[c]] = 0.0f;
        wave_sync();
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll 1
          for (int k = 0; k < LPR; ++k) {
            if (lane == k && id[c] >= 0) grad[id[c]] += gk[c];
            wave_sync();
          }
      }
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
        if (id[c] >= 0) grad[id[c]] = 0.0f;
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
// 16 lanes for many rows (narrow_rows) and K <= 16, else 64.
template <typename F>
hipError_t by_width(int64_t T, int32_t E, int32_t K, F f) {
  typedef std::integral_constant<int, 16> L16;
  typedef std::integral_constant<int, 64> L64;
  if (narrow_rows(T, E) && K <= 16) {
    if (E <= 64) return f(L16(), std::integral_constant<int, 4>());
    if (E <= 128) return f(L16(), std::integral_constant<int, 8>());
    return f(L16(), std::integral_constant<int, 16>());
  }
  if (E <= 256) return f(L64(), std::integral_constant<int, 4>());
  if (E <= 512) return f(L64(), std::integral_constant<int, 8>());
  if (E <= 1024) return f(L64(), std::integral_constant<int, 16>());
  if (E <= 2048) return f(L64(), std::integral_constant<int, 32>());
  return f(L64(), std::integral_constant<int, 64>());
}

// LDS words of a row in the choice: its group scores and keys, or its
// candidates; rows start 8 banks apart.
int32_t choice_words(int lpr, int32_t E, bool groups) {
  const int32_t n = std::max(choose_lds_words(lpr), groups ? kGroupWords + E : 0);
  return (n + 31) / 32 * 32 + 8;
}

int64_t loss_parts(int32_t E) { return ceil_div(E, 64); }

bool aligned4(const void* p, int32_t dtype, int64_t ld, int32_t E) {
  return ((uintptr_t)p & (uintptr_t)(4 * dtype_size(dtype) - 1)) == 0 && ld % 4 == 0 && E % 4 == 0;
}

}  // namespace

int64_t gate_loss_part_bytes(int64_t T, int32_t E, int64_t S) {
  return ((ceil_div(T, loss_chunk(T, E)) + S) * part_stride(E) + S * (loss_parts(E) + 1)) * 4;
}

hipError_t launch_gate(const GateArgs& args, hipStream_t stream) {
  if (args.T == 0) return hipSuccess;
  GateArgs a = args;
  a.vec = aligned4(a.logits, a.dtype, a.ld, a.E) && aligned4(a.bias, kF32, a.E, a.E);
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
  a.vec = aligned4(a.logits, a.dtype, a.ld, a.E) && aligned4(a.bias, kF32, a.E, a.E);
  const int64_t parts = loss_parts(a.E);
  a.terms = a.part + (ceil_div(a.T, loss_chunk(a.T, a.E)) + a.S) * part_stride(a.E);
  a.ticket = reinterpret_cast<int32_t*>(a.terms + a.S * parts);
  const hipError_t err = by_width(a.T, a.E, a.K, [&](auto lpr, auto vpl) {
    constexpr int LPR = decltype(lpr)::value, VPL = decltype(vpl)::value, kRows = kLossThreads / LPR;
    const int32_t words = choice_words(LPR, a.E, true);      // the shares' sums pass through the same place
    const unsigned grid = (unsigned)std::max<int64_t>(1, ceil_div(a.T, loss_chunk(a.T, a.E)));
    gate_loss_kernel<LPR, VPL><<<dim3(grid), dim3(kLossThreads), ((size_t)kRows * words + a.E) * 4, stream>>>(
        a, words, loss_chunk(a.T, a.E));
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  gate_loss_reduce_kernel<<<dim3((unsigned)(a.S * parts)), dim3(kReduceThreads), 0, stream>>>(a, (int32_t)parts,
                                                                                              loss_chunk(a.T, a.E));
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBackwardArgs& args, hipStream_t stream) {
  if (args.T == 0) return hipSuccess;
  GateBackwardArgs a = args;
  a.vec = aligned4(a.logits, a.dtype, a.ld, a.E);
  a.vec_out = aligned4(a.d_logits, a.dtype, a.E, a.E);
  return by_width(a.T, a.E, a.K, [&](auto lpr, auto vpl) {
    constexpr int LPR = decltype(lpr)::value, VPL = decltype(vpl)::value, kRows = kGateThreads / LPR;
    const size_t lds = (size_t)kRows * ((a.E + 3) / 4 * 4 + 4) * 4;
    // A few rows per lane group where there are many, so that a segment's counts are read once for them.  1, 2, 4 and 8
    // rows: 16384 x 256 (here 2) 15.8, 15.1, 20.7 and 35.1 us; 4096 x 256 (1) 9.0, 9.0, 10.4, 16.8; 262144 x 256 bfloat16
    // (8) 165, 129, 116, 113; in between the rule is past the best: 65536 x 256 bfloat16 (8) 46.2, 37.2, 36.4, 43.0; 16384
    // x 512 (8) 27.1, 23.8, 22.6, 27.8.
    const int32_t per_group = (int32_t)std::min<int64_t>(8, std::max<int64_t>(1, a.T / (kRows * 512)));
    gate_backward_kernel<LPR, VPL><<<dim3((unsigned)ceil_div(a.T, (int64_t)kRows * per_group)), dim3(kGateThreads),
                                     lds, stream>>>(a, per_group);
    return hipGetLastError();
  });
}

}  // namespace eplb
