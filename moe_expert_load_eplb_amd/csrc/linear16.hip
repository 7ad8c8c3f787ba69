// The experts' products in 16 bits and the gradient of their weights.
//
// y[r] = x[src(r)] w[g]^T, its gradient of the rows dy[r] w[g] with the weights read
// as they lie, and of the weights dw[g] = sum over r of dy[r]^T x[src(r)], rows of x
// gathered by the loads.  Large ones are bound by the matrix unit at the clock that
// power leaves, and by the start and the end of a tile: 16384 rows on 9, 4096 x 4096,
// launches back to back: 498 us, 1.10 PFLOP/s; rows' gradient 512, into 32 bits 529;
// weights' 611, 0.90.
#include "stream16.h"

namespace eplb {

namespace {

// The loads of a weight gradient's tile: both operands lie across, and their rows of memory are those of one grouping.
// What `rows` names is the same for the lanes of a memory row, and read into scalar registers a block ahead.
// FAR: x spans 2^31 bytes or more.
template <bool ROWS, bool FAR, typename Inner, typename Outer, int W>
struct WgradLoads {
  static constexpr int kEach = Inner::kEach, kRows = Inner::kLoads, kLoads = 2 * kRows, kDirect = kLoads;
  static_assert(kEach == Outer::kEach, "a lane loads the same rows of both");
  typedef const __attribute__((address_space(4))) int32_t* Scalars;
  Inner in;
  Outer out;
  const int32_t* rows;                     // ROWS: of the group's first row on
  FastDiv topk;
  uint32_t X;                              // rows of x
  uint32_t at;
  int K, wave, sub;                        // sub: which of the kEach memory rows of a load this lane is in
  uint32_t column[Inner::kKinds];          // ROWS: where in a row of x this lane's parts lie
  int32_t next[kRows][kEach];
  uint32_t now[kRows][kEach];              // ROWS: offset (FAR: index) of the row of x, or outside
  i32x4 from_x, from_dy;

  __device__ __forceinline__ void fetch(int blk) {
    if (!ROWS) return;
#pragma unroll
    for (int p = 0; p < kRows; ++p)
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const uint32_t k = (uint32_t)blk * kTileK + (p * W + wave) * kEach + j;
        next[p][j] = ((Scalars)rows)[k < (uint32_t)K ? k : (uint32_t)K - 1];
      }
  }
  __device__ __forceinline__ void begin(int blk) {
    from_dy = out.describe_block(blk, K);
    if (!ROWS) {
      from_x = in.describe_block(blk, K);
      return;
    }
#pragma unroll
    for (int p = 0; p < kRows; ++p)
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const uint32_t k = (uint32_t)blk * kTileK + (p * W + wave) * kEach + j;
        const uint32_t row = fastdiv_apply((uint32_t)next[p][j], topk) | (uint32_t)(next[p][j] >> 31);
        now[p][j] = row < X && k < (uint32_t)K ? (FAR ? row : row * in.ld) : kOutside;
      }
  }
  // a row of nothing counts for nothing, whatever dy holds there
  __device__ __forceinline__ void issue(int i, uint32_t slot) const {
    const int p = i >> 1;
    const uint32_t to = at + slot + (i & 1 ? 0 : Inner::kBytes);
    if (!ROWS) {
      if (i & 1) in.load(p, from_x, wave, to);
      else out.load(p, from_dy, wave, to);
      return;
    }
    uint32_t row = now[p][0];
#pragma unroll
    for (int j = 1; j < kEach; ++j) {
      uint32_t other = now[p][j];
      asm("" : "+s"(other));               // not an index into memory
      row = sub == j ? other : row;
    }
    if (i & 1) {
      const uint32_t c = column[p % Inner::kKinds];
      if (!FAR) part_to_lds(from_x, row + c, 0, to + (p * W + wave) * 1024);
      else part_to_lds((row | c) & kOutside ? g_zero_part : in.base + (uint64_t)row * in.ld + c, to + (p * W + wave) * 1024);
    } else {
      part_to_lds(from_dy, out.offset[p % Outer::kKinds] | (row & kOutside), p * (kEach * W) * out.ld,
                  to + (p * W + wave) * 1024);
    }
  }
};

template <Mode MODE, bool ROWS, bool FAR, int WI, int WO, int IT, int OT>
__global__ __launch_bounds__(WI* WO * 64) void wgrad16_kernel(Wgrad16Args a, int32_t ni, int32_t no) {
  typedef Across<WI * IT * 32, WI * WO> Inner;
  typedef Across<WO * OT * 32, WI * WO> Outer;
  typedef AcrossFragments<WI * IT * 32> InnerFragments;
  typedef AcrossFragments<WO * OT * 32> OuterFragments;
  typedef Tile16<MODE, WI, WO, IT, OT, InnerFragments, OuterFragments> Tile_;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t id = die_order(blockIdx.x, gridDim.x);
  const int32_t g = id / (ni * no);
  int32_t row, column;
  band_order(id - g * (ni * no), no, ni, row, column);
  const int i0 = column * Tile_::kInner, o0 = row * Tile_::kOuter;
  const Span span = group_span(a.offsets, g, a.G, a.R);
  int K = span.hi > span.lo ? span.hi - span.lo : 0;
  if (!ROWS && K > a.X - span.lo) K = a.X > span.lo ? (int)(a.X - span.lo) : 0;    // rows that x does not have
  if (a.X == 0) K = 0;
  typename Tile_::Sum acc[Tile_::kO][Tile_::kI];
  if (K > 0) {
    WgradLoads<ROWS, FAR, Inner, Outer, WI * WO> loads;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + i0 * 2;
    loads.in.init(lane, wave, ROWS ? x : x + span.lo * a.ld * 2, a.ld * 2, a.C - i0);
    loads.out.init(lane, wave, static_cast<const uint8_t*>(a.dy) + (span.lo * a.dy_ld + o0) * 2, a.dy_ld * 2, a.N - o0);
    loads.rows = ROWS ? a.rows + span.lo : nullptr;
    loads.topk = a.fd_topk;
    loads.X = (uint32_t)a.X;
    loads.at = lds_address(lds);
    loads.K = K;
    loads.wave = wave;
    loads.sub = lane / Inner::kParts;
    if (ROWS) {
#pragma unroll
      for (int i = 0; i < Inner::kKinds; ++i) loads.column[i] = Inner::column(lane, wave, i, a.C - i0);
      loads.from_x = describe(x, (uint64_t)a.X * a.ld * 2);
    }
    InnerFragments in;
    OuterFragments out;
    in.init(lane, Tile_::inner_first(wave));
    out.init(lane, Tile_::outer_first(wave));
    Tile_::start(loads);
    Tile_::run(in, out, loads, K, lds, acc);
  }
  Tile_::store(acc, lds, a.dw, a.dw_dtype, a.C, a.C - i0,
               [&](int r) -> int64_t { return o0 + r < a.N ? ((int64_t)g * a.N + o0 + r) * a.C + i0 : -1; },
               [&](int) { return K > 0; });
}
// 128 tiles: 28.7 us in small ones, 23.0 in large ones (8 groups of 512 rows, 512 x 2048), 256: 50 and 24.8 (4 groups of 512
// rows, 2048 x 2048).
bool large_wgrad(int64_t N, int64_t C, int32_t G) { return G * ceil_div(N, 256) * ceil_div(C, 256) >= 128; }

template <Mode MODE, bool ROWS>
hipError_t launch_wgrad_form(const Wgrad16Args& a, hipStream_t stream) {
  const bool far = ROWS && a.X * a.ld * 2 >= (int64_t)kOutside;
  if (!far && large_wgrad(a.N, a.C, a.G)) {
    const int64_t ni = ceil_div(a.C, 256), no = ceil_div(a.N, 256);
    wgrad16_kernel<MODE, ROWS, false, 4, 2, 2, 4>
        <<<dim3((unsigned)(a.G * ni * no)), dim3(512), 2 * 2 * 256 * 128, stream>>>(a, (int32_t)ni, (int32_t)no);
  } else {
    const int64_t ni = ceil_div(a.C, 128), no = ceil_div(a.N, 128);
    const dim3 grid((unsigned)(a.G * ni * no));
    if (far) wgrad16_kernel<MODE, ROWS, ROWS, 2, 2, 2, 2><<<grid, dim3(256), 2 * 2 * 128 * 128, stream>>>(a, ni, no);
    else wgrad16_kernel<MODE, ROWS, false, 2, 2, 2, 2><<<grid, dim3(256), 2 * 2 * 128 * 128, stream>>>(a, ni, no);
  }
  return hipGetLastError();
}

}  // namespace

int64_t linear16_blocks(int64_t R, int64_t outputs, int64_t, int32_t G, bool transpose) {
  const int64_t tiles = tile_blocks(R, outputs, G, false);
  return !transpose && stream_suits(R, G) ? std::max(tiles, stream_blocks(R, outputs, G, false)) : tiles;
}

int64_t wgrad16_blocks(int64_t, int64_t N, int64_t C, int32_t G) {
  return (int64_t)G * ceil_div(N, 128) * ceil_div(C, 128);       // of the smaller tiles, which every size may get
}

namespace {

template <Mode MODE>
hipError_t launch_form(const Linear16Args& a, bool transpose, hipStream_t stream) {
  if (transpose) return launch_tiles<MODE, kWeightsTransposed>(a, stream);
  if (stream_suits(a.R, a.G) && a.X * a.ld * 2 < (int64_t)kOutside) return launch_stream<MODE, false>(a, stream);
  return launch_tiles<MODE, kWeights>(a, stream);
}

}  // namespace

hipError_t launch_linear16(const Linear16Args& a, bool transpose, hipStream_t stream) {
  if (a.R == 0) return hipSuccess;
  return a.dtype == kF16 ? launch_form<kBothF16>(a, transpose, stream) : launch_form<kBothBf16>(a, transpose, stream);
}

hipError_t launch_wgrad16(const Wgrad16Args& a, hipStream_t stream) {
  if (a.dtype == kF16)
    return a.rows != nullptr ? launch_wgrad_form<kBothF16, true>(a, stream) : launch_wgrad_form<kBothF16, false>(a, stream);
  return a.rows != nullptr ? launch_wgrad_form<kBothBf16, true>(a, stream) : launch_wgrad_form<kBothBf16, false>(a, stream);
}

}  // namespace eplb
