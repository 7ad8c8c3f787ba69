// The experts' products with 4-bit weights.
//
// What a code and its scale stand for has two significant bits, so it is a
// bfloat16 number exactly: codes become bfloat16 operands of the matrix
// instruction, one conversion instruction for two of them, and no scale is left
// to apply to sums.  Half-precision rows are taken as two bfloat16 values each.
#include "tile16.h"

namespace eplb {

namespace {

constexpr int kWI = 2, kWO = 2, kIT = 2, kOT = 2;
constexpr int kTile = 128;

template <Mode MODE>
hipError_t launch(const Linear16Args& a, hipStream_t stream) {
  typedef LinearTile<MODE, kWI, kWO, kIT, kOT, kWeights4> Tile_;
  linear_tile_kernel<MODE, kWI, kWO, kIT, kOT, kWeights4>
      <<<dim3((unsigned)linear4_blocks(a.R, a.N, a.C, a.G)), dim3(Tile_::kThreads), Tile_::kLdsBytes, stream>>>(
          a, (int32_t)ceil_div(a.N, kTile));
  return hipGetLastError();
}

}  // namespace

int64_t linear4_blocks(int64_t R, int64_t N, int64_t, int32_t G) {
  // every group adds at most one tile that is not full, and a tile has a row
  return (std::min(R, R / kTile + G) + 2) * ceil_div(N, kTile);
}

hipError_t launch_linear4(const Linear16Args& a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  return a.dtype == kF16 ? launch<kSplit>(a, stream) : launch<kBothBf16>(a, stream);
}

}  // namespace eplb
