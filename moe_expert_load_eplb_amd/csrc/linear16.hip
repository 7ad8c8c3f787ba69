// The experts' products in 16 bits and the gradient of their weights.
#include "tile16.h"

namespace eplb {

namespace {

// The loads of a weight gradient's tile: both operands lie across, and their rows of memory are those of one grouping.
// What rows names is held from one block to the next as it is read.
template <typename Inner, typename Outer>
struct WgradLoads {
  static constexpr int kRows = Inner::kLoads, kLoads = 2 * kRows;
  static_assert(Inner::kEach == Outer::kEach, "a lane loads the same rows of both");
  const Inner& in;
  const Outer& out;
  const int32_t* rows;                     // of the group's first row on, or NULL
  FastDiv topk;
  int X, first;                            // rows of x, the group's first row
  uint32_t at;
  int K, wave;
  int32_t named[kRows];

  __device__ __forceinline__ void fetch(int blk) {
#pragma unroll
    for (int p = 0; p < kRows; ++p) {
      const uint32_t k = in.k_of(p, blk);
      named[p] = rows == nullptr || k >= (uint32_t)K ? 0 : rows[k];
    }
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int p = 0; p < kRows; ++p) asm volatile("" : "+v"(named[p]));
  }
  __device__ __forceinline__ void issue(int i, int blk, uint32_t slot) const {
    const int p = i >> 1;
    const uint32_t k = in.k_of(p, blk);
    const int32_t row = (int32_t)(first + k);
    int32_t from = rows == nullptr ? row : named[p] < 0 ? -1 : (int32_t)fastdiv_apply((uint32_t)named[p], topk);
    if (k >= (uint32_t)K || from >= X) from = -1;
    if (i & 1) in.load_row(p, from, wave, at + slot);
    else out.load_row(p, from < 0 ? -1 : row, wave, at + slot + Inner::kBytes);   // a row of nothing counts for nothing
  }
};

template <Mode MODE, int WI, int WO, int IT, int OT>
__global__ __launch_bounds__(WI* WO * 64) void wgrad16_kernel(Wgrad16Args a, int32_t ni, int32_t no) {
  typedef Across<WI * IT * 32, WI * WO, IT, true> Inner;
  typedef Across<WO * OT * 32, WI * WO, OT, false> Outer;
  typedef Tile16<MODE, WI, WO, IT, OT, Inner, Outer> Tile_;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t id = die_order(blockIdx.x, gridDim.x);
  const int32_t g = id / (ni * no);
  int32_t row, column;
  band_order(id - g * (ni * no), no, ni, row, column);
  const int i0 = column * Tile_::kInner, o0 = row * Tile_::kOuter;
  const Span span = group_span(a.offsets, g, a.G, a.R);
  const int K = span.hi > span.lo ? span.hi - span.lo : 0;
  f32x16 acc[OT][IT];
  if (K > 0) {
    Inner in;
    Outer out;
    in.init(lane, wave, Tile_::inner_first(wave), static_cast<const uint8_t*>(a.x) + i0 * 2, a.ld * 2, a.C - i0);
    out.init(lane, wave, Tile_::outer_first(wave), static_cast<const uint8_t*>(a.dy) + o0 * 2, a.dy_ld * 2, a.N - o0);
    WgradLoads<Inner, Outer> loads{in, out, a.rows == nullptr ? nullptr : a.rows + span.lo, a.fd_topk, (int)a.X, span.lo,
                                   lds_address(lds), K, wave};
    Tile_::run(in, out, loads, K, lds, acc);
  }
  Tile_::store(acc, a.dw, a.dw_dtype, a.C, a.C - i0,
               [&](int r) -> int64_t { return o0 + r < a.N ? ((int64_t)g * a.N + o0 + r) * a.C + i0 : -1; },
               [&](int) { return K > 0; });
}

// Tiles of 256 x 256 (four waves of 128 x 128) and of 128 x 128 (four of 64 x 64).
constexpr int kWI = 2, kWO = 2;
constexpr int kLarge = 256, kSmall = 128;

int64_t tile_rows(int64_t R, int32_t G, int tile) {
  // every group adds at most one tile that is not full, and a tile has a row
  return std::min(R, R / tile + G) + 2;
}

bool large_linear(int64_t R, int64_t width, int32_t G) {
  return R >= 128 * (int64_t)G && (R / kLarge + G / 2) * ceil_div(width, kLarge) >= 128;
}

bool large_wgrad(int64_t N, int64_t C, int32_t G) { return G * ceil_div(N, kLarge) * ceil_div(C, kLarge) >= 128; }

template <Mode MODE, int T, Weights FORM>
hipError_t launch(const Linear16Args& a, hipStream_t stream) {
  typedef LinearTile<MODE, kWI, kWO, T, T, FORM> Tile_;
  const int64_t width = FORM == kWeightsTransposed ? a.C : a.N, columns = ceil_div(width, Tile_::kInner);
  linear_tile_kernel<MODE, kWI, kWO, T, T, FORM>
      <<<dim3((unsigned)(tile_rows(a.R, a.G, Tile_::kOuter) * columns)), dim3(Tile_::kThreads), Tile_::kLdsBytes,
         stream>>>(a, (int32_t)columns);
  return hipGetLastError();
}

template <Mode MODE, Weights FORM>
hipError_t launch_form(const Linear16Args& a, hipStream_t stream) {
  return large_linear(a.R, FORM == kWeightsTransposed ? a.C : a.N, a.G) ? launch<MODE, 4, FORM>(a, stream)
                                                                        : launch<MODE, 2, FORM>(a, stream);
}

template <Mode MODE, int T>
hipError_t launch_wgrad(const Wgrad16Args& a, hipStream_t stream) {
  constexpr int kTile = 64 * T;
  const int64_t ni = ceil_div(a.C, kTile), no = ceil_div(a.N, kTile);
  wgrad16_kernel<MODE, kWI, kWO, T, T><<<dim3((unsigned)(a.G * ni * no)), dim3(256), 2 * 2 * kTile * 128, stream>>>(
      a, (int32_t)ni, (int32_t)no);
  return hipGetLastError();
}

template <Mode MODE>
hipError_t launch_wgrad_form(const Wgrad16Args& a, hipStream_t stream) {
  return large_wgrad(a.N, a.C, a.G) ? launch_wgrad<MODE, 4>(a, stream) : launch_wgrad<MODE, 2>(a, stream);
}

}  // namespace

int64_t linear16_blocks(int64_t R, int64_t outputs, int64_t, int32_t G, bool) {
  const int tile = large_linear(R, outputs, G) ? kLarge : kSmall;
  return tile_rows(R, G, tile) * ceil_div(outputs, tile);
}

int64_t wgrad16_blocks(int64_t, int64_t N, int64_t C, int32_t G) {
  const int tile = large_wgrad(N, C, G) ? kLarge : kSmall;
  return (int64_t)G * ceil_div(N, tile) * ceil_div(C, tile);
}

hipError_t launch_linear16(const Linear16Args& a, bool transpose, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  if (a.dtype == kF16)
    return transpose ? launch_form<kBothF16, kWeightsTransposed>(a, stream) : launch_form<kBothF16, kWeights>(a, stream);
  return transpose ? launch_form<kBothBf16, kWeightsTransposed>(a, stream) : launch_form<kBothBf16, kWeights>(a, stream);
}

hipError_t launch_wgrad16(const Wgrad16Args& a, hipStream_t stream) {
  return a.dtype == kF16 ? launch_wgrad_form<kBothF16>(a, stream) : launch_wgrad_form<kBothBf16>(a, stream);
}

}  // namespace eplb
