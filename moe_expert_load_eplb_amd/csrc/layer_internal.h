// Internal declarations of the experts' products in 16 bits and with 4-bit
// weights and of the joining of their rows (not part of the ABI).
#pragma once

#include "experts_internal.h"

namespace eplb {

constexpr int64_t kMaxWidth = int64_t(1) << 22;     // columns of an operand, and elements between its rows
constexpr int kScaleGroup = 32;                     // 4-bit elements that a scale covers
constexpr int64_t kMaxBlocks = (int64_t(1) << 23) - 1;   // workgroups of one launch (512 work-items each at most)

// y[r][i] = sum over j of x[src(r)][j] * W[g(r)][i][j], W being w or (transpose) its transposed view.
struct Linear16Args {
  const void* x;             // rows ld apart
  const void* w;             // [G][N][C] 16-bit
  const uint8_t* q;          // or [G][N][C / 2] 4-bit and [G][N][C / 32]
  const uint8_t* scale;
  const int32_t* offsets;
  const int32_t* rows;
  void* y;                   // [R][N], transpose: [R][C]
  int64_t ld, X;
  int32_t R, N, C, G, topk, dtype, y_dtype;
  FastDiv fd_topk;
};

struct Wgrad16Args {
  const void* dy;            // [R][N], rows dy_ld apart
  const void* x;             // [X][C], rows ld apart
  const int32_t* offsets;
  const int32_t* rows;
  void* dw;                  // [G][N][C]
  int64_t dy_ld, ld, X;
  int32_t R, N, C, G, topk, dtype, dw_dtype;
  FastDiv fd_topk;
};

int64_t linear16_blocks(int64_t R, int64_t outputs, int64_t K, int32_t G, bool transpose);
int64_t linear4_blocks(int64_t R, int64_t N, int64_t C, int32_t G);
int64_t wgrad16_blocks(int64_t R, int64_t N, int64_t C, int32_t G);
hipError_t launch_linear16(const Linear16Args& a, bool transpose, hipStream_t stream);
hipError_t launch_linear4(const Linear16Args& a, hipStream_t stream);
hipError_t launch_wgrad16(const Wgrad16Args& a, hipStream_t stream);

hipError_t launch_quantize_weights4(const void* w, int32_t dtype, int64_t groups, uint8_t* q, uint8_t* scale,
                                    hipStream_t stream);

struct CombineArgs {
  const void* y;             // [R][C]
  const int32_t* place;      // [T][K]
  const float* weights;      // [T][K] or NULL
  void* out;                 // [T][C]
  int64_t R, C, T;
  int32_t K, dtype, out_dtype;
};

struct CombineBackwardArgs {
  const void* d_out;         // [T][C]
  const void* y;             // [T K][C]
  const int32_t* place;
  const int32_t* order;
  const float* weights;
  void* d_y;                 // [T K][C]
  float* d_weights;          // [T][K]
  int64_t C, T;
  int32_t K, dtype, y_dtype;
};

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t stream);
hipError_t launch_combine_rows_backward(const CombineBackwardArgs& a, hipStream_t stream);

}  // namespace eplb
