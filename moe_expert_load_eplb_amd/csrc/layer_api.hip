// C ABI of the experts' products in 16 bits and with 4-bit weights and of the
// joining of their rows: host-side validation, then launches.  Declarations and
// the meaning of every argument: include/eplb_layer.h.
#include "eplb_check.h"
#include "eplb_layer.h"
#include "layer_internal.h"

using namespace eplb;

namespace {

int32_t result(hipError_t err) { return err == hipSuccess ? EPLB_OK : EPLB_E_HIP; }

bool known_dtype(int32_t d) { return d == EPLB_DTYPE_F32 || d == EPLB_DTYPE_BF16 || d == EPLB_DTYPE_F16; }
bool short_dtype(int32_t d) { return d == EPLB_DTYPE_BF16 || d == EPLB_DTYPE_F16; }

bool aligned(const void* p, int64_t n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

// Bytes of rows of n elements, ld apart.
int64_t span(int64_t rows, int64_t ld, int64_t n, int64_t size) {
  return rows <= 0 ? 0 : bytes_of((rows - 1) * ld + n, size, 1);
}

// What the three products have in common: x of X rows of `width` elements.
int32_t check_product(int32_t dtype, int64_t ld, int64_t width, int64_t X, int32_t G, int64_t R, int32_t topk, int64_t N,
                      int64_t C, int32_t out_dtype) {
  if (!short_dtype(dtype) || !known_dtype(out_dtype) || X < 0 || G < 1 || R < 0 || topk < 1 || N < 1 || C < 1)
    return EPLB_E_ARG;
  if (ld < width || ld % 8 != 0 || width % 8 != 0) return EPLB_E_ARG;
  if (N > kMaxWidth || C > kMaxWidth || ld > kMaxWidth || R > kMaxRows || X > kMaxRows || G > kMaxSlots)
    return EPLB_E_LIMIT;
  return EPLB_OK;
}

}  // namespace

extern "C" {

int32_t eplb_expert_matmul16(const void* x, int32_t dtype, int64_t ld, int64_t X, const void* w,
                             const int32_t* offsets, int32_t G, const int32_t* rows, int64_t R, int32_t topk,
                             int64_t N, int64_t C, int32_t transpose, int32_t y_dtype, void* y, void* stream) {
  const int64_t in_width = transpose ? N : C, out_width = transpose ? C : N;
  int32_t rc = check_product(dtype, ld, in_width, X, G, R, topk, N, C, y_dtype);
  if (rc != EPLB_OK) return rc;
  if (C % 8 != 0) return EPLB_E_ARG;
  if (linear16_blocks(R, out_width, in_width, G, transpose != 0) > kMaxBlocks) return EPLB_E_LIMIT;
  if (R == 0) return EPLB_OK;
  if (w == nullptr || offsets == nullptr || y == nullptr || (X > 0 && x == nullptr)) return EPLB_E_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16)) return EPLB_E_ARG;
  const Range in[4] = {{x, span(X, ld, in_width, 2)}, {w, bytes_of(G * N, C, 2)}, {offsets, (G + 1) * (int64_t)4},
                       {rows, R * 4}};
  const Range out[1] = {{y, bytes_of(R, out_width, dtype_size(y_dtype))}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  Linear16Args a = {};
  a.x = x; a.w = w; a.offsets = offsets; a.rows = rows; a.y = y; a.ld = ld; a.X = X;
  a.R = (int32_t)R; a.N = (int32_t)N; a.C = (int32_t)C; a.G = G; a.topk = topk; a.dtype = dtype; a.y_dtype = y_dtype;
  a.fd_topk = fastdiv_make((uint32_t)topk);
  return result(launch_linear16(a, transpose != 0, (hipStream_t)stream));
}

int32_t eplb_expert_wgrad16(const void* dy, int32_t dtype, int64_t dy_ld, int64_t R, const void* x, int64_t ld,
                            int64_t X, const int32_t* offsets, int32_t G, const int32_t* rows, int32_t topk, int64_t N,
                            int64_t C, int32_t dw_dtype, void* dw, void* stream) {
  int32_t rc = check_product(dtype, ld, C, X, G, R, topk, N, C, dw_dtype);
  if (rc != EPLB_OK) return rc;
  if (dy_ld < N || dy_ld % 8 != 0 || N % 8 != 0) return EPLB_E_ARG;
  if (dy_ld > kMaxWidth || wgrad16_blocks(R, N, C, G) > kMaxBlocks) return EPLB_E_LIMIT;
  if (offsets == nullptr || dw == nullptr || (R > 0 && dy == nullptr) || (X > 0 && x == nullptr)) return EPLB_E_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16)) return EPLB_E_ARG;
  const Range in[4] = {{dy, span(R, dy_ld, N, 2)}, {x, span(X, ld, C, 2)}, {offsets, (G + 1) * (int64_t)4},
                       {rows, R * 4}};
  const Range out[1] = {{dw, bytes_of(G * N, C, dtype_size(dw_dtype))}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  Wgrad16Args a = {};
  a.dy = dy; a.x = x; a.offsets = offsets; a.rows = rows; a.dw = dw; a.dy_ld = dy_ld; a.ld = ld; a.X = X;
  a.R = (int32_t)R; a.N = (int32_t)N; a.C = (int32_t)C; a.G = G; a.topk = topk; a.dtype = dtype; a.dw_dtype = dw_dtype;
  a.fd_topk = fastdiv_make((uint32_t)topk);
  return result(launch_wgrad16(a, (hipStream_t)stream));
}

int32_t eplb_quantize_weights4(const void* w, int32_t dtype, int32_t G, int64_t N, int64_t C, uint8_t* q,
                               uint8_t* scale, void* stream) {
  if (!known_dtype(dtype) || G < 0 || N < 1 || C < 1 || C % kScaleGroup != 0) return EPLB_E_ARG;
  if (N > kMaxWidth || C > kMaxWidth || G > kMaxSlots) return EPLB_E_LIMIT;
  const int64_t groups = G * N * (C / kScaleGroup);
  if (groups > kMaxBlocks * 64) return EPLB_E_LIMIT;
  if (groups == 0) return EPLB_OK;
  if (!aligned(w, 16) || !aligned(q, 16)) return EPLB_E_ARG;
  const Range in[1] = {{w, bytes_of(groups, kScaleGroup, dtype_size(dtype))}};
  const Range out[2] = {{q, groups * 16}, {scale, groups}};
  const int32_t rc = check_buffers(in, out);
  if (rc != EPLB_OK) return rc;
  return result(launch_quantize_weights4(w, dtype, groups, q, scale, (hipStream_t)stream));
}

int32_t eplb_expert_matmul4(const void* x, int32_t dtype, int64_t ld, int64_t X, const uint8_t* q,
                            const uint8_t* scale, const int32_t* offsets, int32_t G, const int32_t* rows, int64_t R,
                            int32_t topk, int64_t N, int64_t C, int32_t y_dtype, void* y, void* stream) {
  int32_t rc = check_product(dtype, ld, C, X, G, R, topk, N, C, y_dtype);
  if (rc != EPLB_OK) return rc;
  if (C % kScaleGroup != 0) return EPLB_E_ARG;
  if (linear4_blocks(R, N, C, G) > kMaxBlocks) return EPLB_E_LIMIT;
  if (R == 0) return EPLB_OK;
  if (q == nullptr || scale == nullptr || offsets == nullptr || y == nullptr || (X > 0 && x == nullptr))
    return EPLB_E_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4) || !aligned(y, 16)) return EPLB_E_ARG;
  const int64_t blocks = G * N * (C / kScaleGroup);
  const Range in[5] = {{x, span(X, ld, C, 2)}, {q, bytes_of(blocks, 16, 1)}, {scale, blocks},
                       {offsets, (G + 1) * (int64_t)4}, {rows, R * 4}};
  const Range out[1] = {{y, bytes_of(R, N, dtype_size(y_dtype))}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  Linear16Args a = {};
  a.x = x; a.q = q; a.scale = scale; a.offsets = offsets; a.rows = rows; a.y = y; a.ld = ld; a.X = X;
  a.R = (int32_t)R; a.N = (int32_t)N; a.C = (int32_t)C; a.G = G; a.topk = topk; a.dtype = dtype; a.y_dtype = y_dtype;
  a.fd_topk = fastdiv_make((uint32_t)topk);
  return result(launch_linear4(a, (hipStream_t)stream));
}

int32_t eplb_combine_rows(const void* y, int32_t dtype, int64_t R, int64_t C, const int32_t* place,
                          const float* weights, int64_t T, int32_t K, int32_t out_dtype, void* out, void* stream) {
  if (!known_dtype(dtype) || !known_dtype(out_dtype) || R < 0 || C < 1 || T < 0 || K < 1) return EPLB_E_ARG;
  if (C > kMaxDim || K > kMaxK || R > kMaxRows || T > kMaxRows / K) return EPLB_E_LIMIT;
  if (T == 0) return EPLB_OK;
  if (place == nullptr || out == nullptr || (R > 0 && y == nullptr)) return EPLB_E_ARG;
  if (!aligned(y, dtype_size(dtype)) || !aligned(out, dtype_size(out_dtype)) || !aligned(place, 4) ||
      !aligned(weights, 4))
    return EPLB_E_ARG;
  const Range in[3] = {{y, bytes_of(R, C, dtype_size(dtype))}, {place, T * K * 4}, {weights, T * K * 4}};
  const Range outs[1] = {{out, bytes_of(T, C, dtype_size(out_dtype))}};
  const int32_t rc = check_disjoint(in, outs);
  if (rc != EPLB_OK) return rc;
  CombineArgs a = {};
  a.y = y; a.place = place; a.weights = weights; a.out = out; a.R = R; a.C = C; a.T = T; a.K = K; a.dtype = dtype;
  a.out_dtype = out_dtype;
  return result(launch_combine_rows(a, (hipStream_t)stream));
}

int32_t eplb_combine_rows_backward(const void* d_out, int32_t dtype, const void* y, int32_t y_dtype, int64_t C,
                                   const int32_t* place, const int32_t* order, const float* weights, int64_t T,
                                   int32_t K, void* d_y, float* d_weights, void* stream) {
  if (!known_dtype(dtype) || !known_dtype(y_dtype) || C < 1 || T < 0 || K < 1) return EPLB_E_ARG;
  if (C > kMaxDim || K > kMaxK || T > kMaxRows / K) return EPLB_E_LIMIT;
  if (T == 0) return EPLB_OK;
  if (d_out == nullptr || place == nullptr || order == nullptr || d_y == nullptr || (d_weights != nullptr && y == nullptr))
    return EPLB_E_ARG;
  if (!aligned(d_out, dtype_size(dtype)) || !aligned(y, dtype_size(y_dtype)) || !aligned(d_y, dtype_size(y_dtype)) ||
      !aligned(place, 4) || !aligned(order, 4) || !aligned(weights, 4) || !aligned(d_weights, 4))
    return EPLB_E_ARG;
  const int64_t rows = T * K, bytes = bytes_of(rows, C, dtype_size(y_dtype));
  const Range in[5] = {{d_out, bytes_of(T, C, dtype_size(dtype))}, {y, bytes}, {place, rows * 4}, {order, rows * 4},
                       {weights, rows * 4}};
  const Range out[2] = {{d_y, bytes}, {d_weights, rows * 4}};
  const int32_t rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  CombineBackwardArgs a = {};
  a.d_out = d_out; a.y = y; a.place = place; a.order = order; a.weights = weights; a.d_y = d_y; a.d_weights = d_weights;
  a.C = C; a.T = T; a.K = K; a.dtype = dtype; a.y_dtype = y_dtype;
  return result(launch_combine_rows_backward(a, (hipStream_t)stream));
}

}  // extern "C"
