// Rows grouped by slot: a stable counting sort of the physical ids of every
// layer.
//
// The ids of a layer fall into segments of equal length, one workgroup each.
// The first launch counts every segment; in the second a workgroup adds up
// the counts of the segments before it (and of all, for the slots' starts),
// ranks its own ids in order and writes both directions of the permutation.
// A layer of one segment needs the second launch only.
//
// Bound by latency: of the launches, of the chain of 64-id steps in a wave
// (ballots, one LDS round trip each), and of the sums over segments.  512 ids,
// 320 slots: 4.5 us; 131,072 ids, 288 slots: 3.4 + 11.3 us (1.6 MB, whose copy
// would take 0.3; the waves wait for two thirds of the second launch).
#include "experts_internal.h"

namespace eplb {

namespace {

constexpr int kGroupSeg = 2048;              // ids of a segment: at most this many, or a multiple of it for long layers
constexpr int kGroupStep = 512;              // 64 ids of each of 8 waves
constexpr int kGroupMaxSegs = 256;           // segments of a layer

struct GroupSplit {
  int64_t n, seg, segs;
  int32_t waves;
};

// A workgroup ranks its ids 64 per wave at a time, so short segments shorten
// that chain and long ones the sums over the segments before.  Up to 2048 ids
// one segment, spread over all waves (58 layers x 1024 ids: 5.9 us, 7.3 with
// segments of 2048, 7.8 with two segments of 512).  Few layers of somewhat
// more: 16 segments (8192 ids: 7.7 us with segments of 512, 10.9 with 2048).
// Else 2048 (131,072 ids: 13.6 us, 14.3 with 1024, 17.0 with 4096; 58 layers x
// 65,536 ids: 29.9 us, 41.0 with 1024, 32.6 with 4096).
GroupSplit plan_group(int64_t L, int64_t n, int32_t P) {
  GroupSplit s;
  s.n = n;
  if (n <= kGroupSeg) s.seg = ceil_div(n, kGroupStep) * kGroupStep;
  else if (L <= 16 && n <= 16 * kGroupSeg) s.seg = ceil_div(ceil_div(n, 16), kGroupStep) * kGroupStep;
  else s.seg = ceil_div(ceil_div(n, kGroupMaxSegs), kGroupSeg) * kGroupSeg;
  if (s.seg < kGroupStep) s.seg = kGroupStep;
  s.segs = ceil_div(n, s.seg);
  if (s.segs < 1) s.segs = 1;
  s.waves = P < 4096 ? 8 : 2;                // one set of counters per wave, at most 144 KiB of LDS in all
  return s;
}

__device__ __forceinline__ int32_t slot_of(int32_t id, int32_t first, int32_t P) {
  const int64_t g = (int64_t)id - first;
  return g >= 0 && g < P ? (int32_t)g : P;
}

__global__ __launch_bounds__(512) void group_count_kernel(const int32_t* __restrict__ ids, GroupSplit sp,
                                                          int32_t first, int32_t P, int32_t* __restrict__ ws) {
  extern __shared__ int32_t cnt[];           // [P + 1]
  const int64_t l = blockIdx.x / sp.segs, s = blockIdx.x % sp.segs;
  for (int p = threadIdx.x; p <= P; p += blockDim.x) cnt[p] = 0;
  __syncthreads();
  const int64_t i0 = s * sp.seg, i1 = i0 + sp.seg < sp.n ? i0 + sp.seg : sp.n;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x)
    atomicAdd(&cnt[slot_of(ids[l * sp.n + i], first, P)], 1);
  __syncthreads();
  int32_t* out = ws + blockIdx.x * (int64_t)(P + 1);
  for (int p = threadIdx.x; p <= P; p += blockDim.x) out[p] = cnt[p];
}

__global__ __launch_bounds__(512) void group_place_kernel(const int32_t* __restrict__ ids, GroupSplit sp,
                                                          int32_t first, int32_t P, int32_t bits,
                                                          const int32_t* __restrict__ ws,
                                                          int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                          int32_t* __restrict__ place) {
  extern __shared__ int32_t lds[];           // [waves][P + 1] counters, [P + 1] starts
  __shared__ int32_t wave_sum[8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = sp.waves, NT = waves * 64;
  const int C = P + 1;
  int32_t* mine = lds + wave * C;
  int32_t* start = lds + waves * C;
  const int64_t l = blockIdx.x / sp.segs, s = blockIdx.x % sp.segs;
  const int64_t i0 = s * sp.seg, i1 = i0 + sp.seg < sp.n ? i0 + sp.seg : sp.n;
  const int64_t part = sp.seg / waves;       // a multiple of 64
  const int64_t w0 = i0 + wave * part, w1 = w0 + part < i1 ? w0 + part : i1;
  const int32_t* in = ids + l * sp.n;
  for (int p = threadIdx.x; p < waves * C; p += NT) lds[p] = 0;
  __syncthreads();
  for (int64_t i = w0 + lane; i < w1; i += 64) atomicAdd(&mine[slot_of(in[i], first, P)], 1);
  __syncthreads();

  // slots p0 .. p0 + per - 1 of this thread: totals, and what stands before this segment
  const int per = (C + NT - 1) / NT;
  const int p0 = threadIdx.x * per, p1 = p0 + per < C ? p0 + per : C;
  int32_t sum = 0;
  for (int p = p0; p < p1; ++p) {
    int32_t total = 0, before = 0;
    if (sp.segs == 1) {
      for (int w = 0; w < waves; ++w) total += lds[w * C + p];
    } else {
      // 16 loads in flight; past the last segment its count again, not added
      const int32_t* col = ws + l * sp.segs * C + p;
      const int segs = (int)sp.segs, here = (int)s;
      for (int j0 = 0; j0 < segs; j0 += 16) {
        int32_t c[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) c[j] = col[(int64_t)min(j0 + j, segs - 1) * C];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          total += j0 + j < segs ? c[j] : 0;
          before += j0 + j < here ? c[j] : 0;
        }
      }
    }
    start[p] = sum;
    sum += total;
    // the waves' counters become what stands before each of them, this slot's start left out
    for (int w = 0; w < waves; ++w) {
      const int32_t c = lds[w * C + p];
      lds[w * C + p] = before;
      before += c;
    }
  }
  int32_t incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int32_t base = incl - sum;
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
  for (int p = p0; p < p1; ++p) {
    const int32_t at = base + start[p];
    if (s == 0) offsets[l * C + p] = at;     // start of the ids of no slot = end of the last slot
    for (int w = 0; w < waves; ++w) lds[w * C + p] += at;
  }
  __syncthreads();

  // 64 ids at a time, in order: lanes with the same slot find each other by
  // one ballot per bit of the slot number
  for (int64_t i = w0; i < w1; i += 64) {
    const bool in_range = i + lane < w1;
    const int32_t g = in_range ? slot_of(in[i + lane], first, P) : 0;
    u64 same = __ballot(in_range);
    for (int b = 0; b < bits; ++b) {
      const u64 set = __ballot(g >> b & 1);
      same &= g >> b & 1 ? set : ~set;
    }
    if (in_range) {
      const int32_t to = mine[g] + __popcll(same & ((u64(1) << lane) - 1));
      order[l * sp.n + to] = (int32_t)(i + lane);
      place[l * sp.n + i + lane] = to;
    }
    __builtin_amdgcn_wave_barrier();
    if (in_range && (same >> lane) == 1) mine[g] += __popcll(same);   // the last of them
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

}  // namespace

bool group_rows_fits(int64_t L, int64_t n, int32_t P) { return L * plan_group(L, n, P).segs <= kMaxLayers; }

int64_t group_rows_bytes(int64_t L, int64_t n, int32_t P) {
  const GroupSplit sp = plan_group(L, n, P);
  return sp.segs == 1 ? 0 : L * sp.segs * (int64_t)(P + 1) * 4;
}

hipError_t launch_group_rows(const int32_t* ids, int64_t L, int64_t n, int32_t first, int32_t P, int32_t* ws,
                             int32_t* offsets, int32_t* order, int32_t* place, hipStream_t stream) {
  if (L == 0) return hipSuccess;
  const GroupSplit sp = plan_group(L, n, P);
  const dim3 grid((unsigned)(L * sp.segs));
  if (sp.segs > 1) {
    group_count_kernel<<<grid, dim3(512), (size_t)(P + 1) * 4, stream>>>(ids, sp, first, P, ws);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  int32_t bits = 0;
  while ((1 << bits) <= P) ++bits;
  const size_t lds = (size_t)(sp.waves + 1) * (P + 1) * 4;
  group_place_kernel<<<grid, dim3(sp.waves * 64), lds, stream>>>(ids, sp, first, P, bits, ws, offsets, order, place);
  return hipGetLastError();
}

}  // namespace eplb
