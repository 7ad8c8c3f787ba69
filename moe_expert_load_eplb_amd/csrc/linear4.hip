// The experts' products with 4-bit weights.
//
// What a code and its scale stand for has two significant bits, so it is a
// bfloat16 number exactly: against bfloat16 rows, codes become bfloat16 operands of
// the matrix instruction, one conversion instruction for two of them, and no scale
// is left to apply to sums.  Against half-precision rows, whose range a scale may
// leave, they become half-precision operands without it, and each instruction's sum
// over 32 of k, one scale's, is multiplied by it in 32 bits.
//
// Few rows are bound by the start and the end of a kernel and by the conversions
// (stream16.h), many by the matrix unit: 16384 rows on 9, 4096 x 4096, launches back
// to back: 438 us, 1.25 PFLOP/s, half-precision rows 778 (four multiply-adds for each
// matrix instruction, and weights converted for 128 rows at a time).
#include "stream16.h"

namespace eplb {

namespace {

template <Mode MODE>
hipError_t launch_form(const Linear16Args& a, hipStream_t stream) {
  if (stream_suits(a.R, a.G) && a.X * a.ld * 2 < (int64_t)kOutside) return launch_stream<MODE, true>(a, stream);
  return launch_tiles<MODE, kWeights4>(a, stream);
}

}  // namespace

int64_t linear4_blocks(int64_t R, int64_t N, int64_t, int32_t G) {
  const int64_t tiles = tile_blocks(R, N, G, true);
  return stream_suits(R, G) ? std::max(tiles, stream_blocks(R, N, G, true)) : tiles;
}

hipError_t launch_linear4(const Linear16Args& a, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  return a.dtype == kF16 ? launch_form<kScaled>(a, stream) : launch_form<kBothBf16>(a, stream);
}

}  // namespace eplb
