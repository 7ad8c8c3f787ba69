// Internal declarations of the router, the grouping and the experts' products
// (not part of the ABI).
#pragma once

#include "eplb_internal.h"

namespace eplb {

constexpr int32_t kF32 = 0, kBf16 = 1, kF16 = 2;    // EPLB_DTYPE_*
constexpr int32_t kSigmoid = 0;                     // EPLB_SCORE_SIGMOID
constexpr float kScoreEps = 1e-20f;                 // added to a sum of scores before it divides
constexpr float kF8Max = 448.0f;                    // largest finite 8-bit value
constexpr float kAmaxMin = 0x1p-100f;               // least block maximum a scale is made from
constexpr int64_t kMaxTokens = int64_t(1) << 25;    // tokens of one router call (64 work-items each)
constexpr int kMaxK = 64;                           // choices of a token
constexpr int kMaxGroups = 64;                      // expert groups of the router
constexpr int64_t kMaxSegments = int64_t(1) << 20;  // segments of one balance loss
constexpr int64_t kMaxLossParts = int64_t(1) << 21; // runs of 64 experts over all segments (1024 work-items each)
constexpr int kBlock = 128;                         // elements a scale covers along an axis
constexpr int kMaxSlots = 8192;                     // slots of a grouping, groups of a product
constexpr int64_t kMaxDim = int64_t(1) << 24;       // columns of an operand
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPadded = int64_t(1) << 32;    // grouped rows, every group rounded up to 128

typedef unsigned short u16;
typedef float f32x4 __attribute__((ext_vector_type(4)));

inline int64_t dtype_size(int32_t dtype) { return dtype == kF32 ? 4 : 2; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ float bf16_to_float(u16 h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ float f16_to_float(u16 h) { return (float)__builtin_bit_cast(_Float16, h); }
__device__ __forceinline__ u16 float_to_bf16(float f) { return __builtin_bit_cast(u16, (__bf16)f); }
__device__ __forceinline__ u16 float_to_f16(float f) { return __builtin_bit_cast(u16, (_Float16)f); }

__device__ __forceinline__ float load_as_float(const void* p, int32_t dtype, int64_t i) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  const u16 h = static_cast<const u16*>(p)[i];
  return dtype == kBf16 ? bf16_to_float(h) : f16_to_float(h);
}

__device__ __forceinline__ void store_float(void* p, int32_t dtype, int64_t i, float v) {
  if (dtype == kF32) static_cast<float*>(p)[i] = v;
  else static_cast<u16*>(p)[i] = dtype == kBf16 ? float_to_bf16(v) : float_to_f16(v);
}

// ---------------------------------------------------------------- router
struct GateArgs {
  const void* logits;
  int64_t ld, T, S;
  int32_t dtype, E, K, scoring, G, top_groups, group_top, normalize;
  float scale, alpha;
  const float* bias;
  const uint8_t* mask;
  const int32_t* seg;
  int32_t given;             // ids are an input (no choice is made)
  int32_t* ids;
  float* weights;
  bool vec;                  // four logits can be loaded at once
  float* part;               // partial sums of the loss
  float* terms;              // the loss by runs of 64 experts
  int32_t* ticket;           // workgroups of a segment that are done
  float* loss;
  int32_t* counts;
  float* prob;
  int32_t* tokens;
  FastDiv fd_group;          // expert -> group
};

struct GateBackwardArgs {
  const void* logits;
  int64_t ld, T, S;
  int32_t dtype, E, K, scoring, normalize;
  float scale, alpha;
  const uint8_t* mask;
  const int32_t* ids;
  const float* d_weights;
  const int32_t* seg;
  const int32_t* counts;
  const int32_t* tokens;
  const float* d_loss;
  void* d_logits;
  bool vec, vec_out;         // four logits / gradients at once
};

int64_t gate_loss_part_bytes(int64_t T, int32_t E, int64_t S);
hipError_t launch_gate(const GateArgs& a, hipStream_t stream);
hipError_t launch_gate_loss(const GateArgs& a, hipStream_t stream);
hipError_t launch_gate_backward(const GateBackwardArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- grouping
bool group_rows_fits(int64_t L, int64_t n, int32_t P);     // segments within one launch
int64_t group_rows_bytes(int64_t L, int64_t n, int32_t P);
hipError_t launch_group_rows(const int32_t* ids, int64_t L, int64_t n, int32_t first, int32_t P, int32_t* ws,
                             int32_t* offsets, int32_t* order, int32_t* place, hipStream_t stream);

// ---------------------------------------------------------------- 8-bit blocks
hipError_t launch_quantize_rows(const void* x, int32_t dtype, int64_t ld, int64_t R, int64_t C, uint8_t* q,
                                float* scale, hipStream_t stream);
hipError_t launch_quantize_columns(const void* x, int32_t dtype, int64_t ld, int64_t X, int64_t C,
                                   const int32_t* rows, int64_t R, int32_t K, const int32_t* offsets, int32_t G,
                                   int64_t Rp, uint8_t* q, float* scale, hipStream_t stream);
hipError_t launch_quantize_weights(const void* w, int32_t dtype, int32_t G, int64_t N, int64_t K, uint8_t* q,
                                   float* scale, uint8_t* qt, float* scale_t, hipStream_t stream);

// ---------------------------------------------------------------- products
struct MatmulArgs {
  const uint8_t* q;          // [X][K]
  const float* scale;        // [X][KB]
  const uint8_t* w;          // [G][N][K]
  const float* w_scale;      // [G][NB][KB]
  const int32_t* offsets;
  const int32_t* rows;
  void* y;
  int64_t X;
  int32_t R, N, K, KB, NB, G, topk, dtype;
  FastDiv fd_topk;
};

struct WgradArgs {
  const uint8_t* dy;         // [N][Rp]
  const float* dy_scale;     // [Rp / 128][N]
  const uint8_t* x;          // [K][Rp]
  const float* x_scale;      // [Rp / 128][K]
  const int32_t* offsets;
  void* dw;
  int64_t Rp;
  int32_t R, N, K, G, dtype;
};

int64_t matmul_tiles(int64_t R, int64_t N, int64_t K, int32_t G);
int64_t wgrad_tiles(int64_t N, int64_t K, int32_t G);
hipError_t launch_expert_matmul(const MatmulArgs& a, hipStream_t stream);
hipError_t launch_expert_wgrad(const WgradArgs& a, hipStream_t stream);

}  // namespace eplb
