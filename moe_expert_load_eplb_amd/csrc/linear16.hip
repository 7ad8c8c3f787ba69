// The experts' products in 16 bits and the gradient of their weights.
#include "tile16.h"

namespace eplb {

namespace {

template <Mode MODE, int WI, int WO, int IT, int OT>
__global__ __launch_bounds__(WI* WO * 64) void wgrad16_kernel(Wgrad16Args a, int32_t ni, int32_t no) {
  typedef Across<WI * IT * 32, WI * WO, IT, true, true> Inner;
  typedef Across<WO * OT * 32, WI * WO, OT, false, true> Outer;
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
    in.gather(a.rows, span.lo, (int)a.X, a.fd_topk, K, false);
    out.init(lane, wave, Tile_::outer_first(wave), static_cast<const uint8_t*>(a.dy) + o0 * 2, a.dy_ld * 2, a.N - o0);
    out.gather(a.rows, span.lo, (int)a.X, a.fd_topk, K, true);
    Tile_::run(in, out, K, lds, acc, [&](int b) {
      in.fetch(b, K);
      out.fetch(b, K);
    });
  }
  Tile_::store(acc, a.dw, a.dw_dtype, a.C, a.C - i0,
               [&](int r) -> int64_t { return o0 + r < a.N ? ((int64_t)g * a.N + o0 + r) * a.C + i0 : -1; },
               [&](int) { return K > 0; });
}

constexpr int kWI = 2, kWO = 2, kIT = 2, kOT = 2;
constexpr int kTile = 128;

template <Mode MODE, Weights FORM>
hipError_t launch(const Linear16Args& a, hipStream_t stream) {
  typedef LinearTile<MODE, kWI, kWO, kIT, kOT, FORM> Tile_;
  const bool transpose = FORM == kWeightsTransposed;
  const int64_t width = transpose ? a.C : a.N;
  linear_tile_kernel<MODE, kWI, kWO, kIT, kOT, FORM>
      <<<dim3((unsigned)linear16_blocks(a.R, width, transpose ? a.N : a.C, a.G, transpose)), dim3(Tile_::kThreads),
         Tile_::kLdsBytes, stream>>>(a, (int32_t)ceil_div(width, kTile));
  return hipGetLastError();
}

template <Mode MODE>
hipError_t launch_wgrad(const Wgrad16Args& a, hipStream_t stream) {
  constexpr int kLds = 2 * 2 * kTile * 128;
  wgrad16_kernel<MODE, kWI, kWO, kIT, kOT><<<dim3((unsigned)wgrad16_blocks(a.R, a.N, a.C, a.G)), dim3(256), kLds, stream>>>(
      a, (int32_t)ceil_div(a.C, kTile), (int32_t)ceil_div(a.N, kTile));
  return hipGetLastError();
}

}  // namespace

int64_t linear16_blocks(int64_t R, int64_t outputs, int64_t, int32_t G, bool) {
  // every group adds at most one tile that is not full, and a tile has a row
  return (std::min(R, R / kTile + G) + 2) * ceil_div(outputs, kTile);
}

int64_t wgrad16_blocks(int64_t, int64_t N, int64_t C, int32_t G) {
  return (int64_t)G * ceil_div(N, kTile) * ceil_div(C, kTile);
}

hipError_t launch_linear16(const Linear16Args& a, bool transpose, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  if (a.dtype == kF16)
    return transpose ? launch<kBothF16, kWeightsTransposed>(a, stream) : launch<kBothF16, kWeights>(a, stream);
  return transpose ? launch<kBothBf16, kWeightsTransposed>(a, stream) : launch<kBothBf16, kWeights>(a, stream);
}

hipError_t launch_wgrad16(const Wgrad16Args& a, hipStream_t stream) {
  return a.dtype == kF16 ? launch_wgrad<kBothF16>(a, stream) : launch_wgrad<kBothBf16>(a, stream);
}

}  // namespace eplb
