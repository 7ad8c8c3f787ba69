// The experts' products with 4-bit weights.
//
// What a code and its scale stand for has two significant bits, so it is a
// bfloat16 number exactly: codes become bfloat16 operands of the matrix
// instruction, one conversion instruction for two of them, and no scale is left
// to apply to sums.  Half-precision rows are taken as two bfloat16 values each.
#include "tile16.h"

namespace eplb {

namespace {

constexpr int kTile = 128;

template <Mode MODE, bool FAR>
hipError_t launch(const Linear16Args& a, hipStream_t stream) {
  linear_small_kernel<MODE, kWeights4, FAR>
      <<<dim3((unsigned)linear4_blocks(a.R, a.N, a.C, a.G)), dim3(256), 2 * 2 * 128 * 128, stream>>>(
          a, (int32_t)ceil_div(a.N, kTile));
  return hipGetLastError();
}

template <Mode MODE>
hipError_t launch_form(const Linear16Args& a, hipStream_t stream) {
  return a.X * a.ld * 2 >= (int64_t)kOutside ? launch<MODE, true>(a, stream) : launch<MODE, false>(a, stream);
}

}  // namespace

int64_t linear4_blocks(int64_t R, int64_t N, int64_t, int32_t G) {
  // every group adds at most one tile that is not full, and a tile has a row
  return (std::min(R, R / kTile + G) + 2) * ceil_div(N, kTile);
}

hipError_t launch_linear4(const Linear16Args& a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  return a.dtype == kF16 ? launch_form<kSplit>(a, stream) : launch_form<kBothBf16>(a, stream);
}

}  // namespace eplb
