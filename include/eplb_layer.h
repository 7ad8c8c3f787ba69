/*
 * eplb_layer.h -- C ABI of the rest of an MoE layer around the EPLB hot path
 * on AMD Instinct MI355X (gfx950), in the same library: the experts' products
 * in 16-bit floating point with both gradients, the same products with 4-bit
 * weights, and the experts' rows joined back to tokens, with its gradients.
 *
 * The conventions, return codes and ownership rules are those of eplb.h; the
 * types, the groupings (offsets, rows, place) and what is 8-bit are those of
 * eplb_experts.h.
 */
#ifndef EPLB_LAYER_H_
#define EPLB_LAYER_H_

#include "eplb_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * eplb_expert_matmul16 -- the experts' product in 16 bits: every grouped row
 * times the transposed weights of its expert,
 *   y[r][n] = sum over c of x[src(r)][c] * w[g][n][c]
 * or, with transpose, times the weights as they are (the gradient with respect
 * to the rows),
 *   y[r][c] = sum over n of x[src(r)][n] * w[g][n][c]
 * where g is the group of row r and src(r) = rows[r] / topk, or r without rows.
 * Sums are held in 32 bits and the result is rounded once.  Equal inputs give
 * equal bits.  Rows of no group, and rows whose src(r) is outside [0, X), get
 * zeros, whatever x holds.
 *
 *   x          [X][C] dtype      ([X][N] with transpose) EPLB_DTYPE_BF16 or
 *                                EPLB_DTYPE_F16, rows ld elements apart; ld a
 *                                multiple of 8, 16-byte aligned
 *   w          [G][N][C] dtype   contiguous, 16-byte aligned
 *   offsets    [G + 1] int32     eplb_group_rows': non-decreasing.  Values are
 *                                clamped to 0 .. R, a group that ends before it
 *                                starts is empty; offsets that decrease make
 *                                groups that share rows: nothing outside the
 *                                arrays is reached, but what such rows get is
 *                                not defined
 *   rows       [R] int32         or NULL
 *   N, C                         1 .. 2^22; C a multiple of 8, N too with
 *                                transpose
 *   y          [R][N] y_dtype    out ([R][C] with transpose): any of the three
 *                                types; 16-byte aligned
 *
 * Errors of the products: EPLB_E_ARG (a size outside its range or not a
 * multiple as above, ld below the row's elements, a pointer not aligned, an
 * unknown or unfit dtype, a NULL array, an output sharing a byte with an
 * input), EPLB_E_LIMIT (N, C or ld > 2^22, R or X > 2^31 - 1, G > 8192, or more
 * than 2^23 - 1 tiles of the output), EPLB_E_HIP.
 */
int32_t eplb_expert_matmul16(const void* x, int32_t dtype, int64_t ld, int64_t X, const void* w,
                             const int32_t* offsets, int32_t G, const int32_t* rows, int64_t R, int32_t topk,
                             int64_t N, int64_t C, int32_t transpose, int32_t y_dtype, void* y, void* stream);

/*
 * eplb_expert_wgrad16 -- the gradient of that product with respect to the
 * weights: for every group g
 *   dw[g][n][c] = sum over the group's rows r of dy[r][n] * x[src(r)][c]
 * Rows whose src(r) is outside [0, X) count for nothing.  Sums are held in 32
 * bits and taken in the order of the rows; a group without rows gets zeros.
 *
 *   dy         [R][N] dtype      rows dy_ld elements apart
 *   x          [X][C] dtype      rows ld elements apart
 *   N, C                         multiples of 8
 *   dw         [G][N][C] dw_dtype  out, 16-byte aligned
 * Strides and alignment as above.  Errors: those of the products.
 */
int32_t eplb_expert_wgrad16(const void* dy, int32_t dtype, int64_t dy_ld, int64_t R, const void* x, int64_t ld,
                            int64_t X, const int32_t* offsets, int32_t G, const int32_t* rows, int32_t topk, int64_t N,
                            int64_t C, int32_t dw_dtype, void* dw, void* stream);

/*
 * 4-bit floating point with a power of two for each 32 elements: values are
 * the format with 1 sign, 2 exponent and 1 mantissa bits (magnitudes 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 as codes 0 .. 7, the sign in the fourth bit), two to a byte,
 * the even element in the low half.  A scale byte s stands for 2^(s - 127), 255
 * for NaN.  (The public microscaling format with 4-bit elements.)
 *
 * eplb_quantize_weights4 -- weights in that format, blocks of 32 along a row:
 * with a the block's largest magnitude, s - 127 is the least integer e >= -100
 * with a <= 7 * 2^e, and a value is the nearest magnitude to |x| / 2^e, ties to
 * the even code, 6 above it.  A block that holds an infinity or a NaN gets s =
 * 255 and codes 0.
 *   w          [G][N][C] dtype   any of the three types, contiguous
 *   C                            a multiple of 32
 *   q          [G][N][C / 2]     out, 16-byte aligned
 *   scale      [G][N][C / 32]    out
 * Errors: EPLB_E_ARG (a size < 1, G < 0, C % 32, an unknown dtype, a NULL array, a
 * pointer not aligned, an output sharing a byte with an input or the other),
 * EPLB_E_LIMIT (N or C > 2^22, G > 8192, more than 2^29 - 64 blocks of 32),
 * EPLB_E_HIP.
 */
int32_t eplb_quantize_weights4(const void* w, int32_t dtype, int32_t G, int64_t N, int64_t C, uint8_t* q,
                               uint8_t* scale, void* stream);

/*
 * eplb_expert_matmul4 -- eplb_expert_matmul16 (not transposed) with weights in
 * that format: what a code and its scale stand for is multiplied exactly, as
 * long as it is 0 or its magnitude is at least 2^-126 (scales of 2 .. 254; what
 * is below may count as 0, and a value past the largest finite 32-bit number
 * may be an infinity).
 *   q          [G][N][C / 2]     16-byte aligned
 *   scale      [G][N][C / 32]    4-byte aligned
 *   C                            a multiple of 32
 * The rest as there.  Errors: those of the products.
 */
int32_t eplb_expert_matmul4(const void* x, int32_t dtype, int64_t ld, int64_t X, const uint8_t* q,
                            const uint8_t* scale, const int32_t* offsets, int32_t G, const int32_t* rows, int64_t R,
                            int32_t topk, int64_t N, int64_t C, int32_t y_dtype, void* y, void* stream);

/*
 * eplb_combine_rows -- the experts' rows joined to tokens:
 *   out[t][c] = sum over k of weights[t][k] * y[place[t][k]][c]
 * in the order of k, by 32-bit fused multiply-adds, rounded once.  A choice
 * whose place is outside [0, R) adds nothing.  Without weights they are 1.
 *
 *   y          [R][C] dtype      contiguous
 *   place      [T][K] int32      eplb_group_rows'
 *   weights    [T][K] float32    or NULL
 *   out        [T][C] out_dtype  out
 *
 * Errors of the two calls: EPLB_E_ARG (a size < 0, C or K < 1, an unknown dtype,
 * a NULL array, a pointer not aligned to its type, an output sharing a byte with
 * an input or another output), EPLB_E_LIMIT (C > 2^24, K > 64, T * K or R >
 * 2^31 - 1), EPLB_E_HIP.
 */
int32_t eplb_combine_rows(const void* y, int32_t dtype, int64_t R, int64_t C, const int32_t* place,
                          const float* weights, int64_t T, int32_t K, int32_t out_dtype, void* out, void* stream);

/*
 * eplb_combine_rows_backward -- the gradients of that call for a grouping:
 *   d_weights[t][k]     = sum over c of d_out[t][c] * y[place[t][k]][c]
 *   d_y[place[t][k]][c] = weights[t][k] * d_out[t][c]
 * place and order are eplb_group_rows' outputs, each the inverse of the other.
 * A choice whose place is outside [0, T K) gets d_weights 0; a row r of d_y with
 * place[order[r]] != r (order[r] outside [0, T K) among them) gets zeros, so
 * every output is written once, whatever the arrays hold.
 *
 *   d_out      [T][C] dtype      contiguous
 *   y          [T K][C] y_dtype  contiguous
 *   place, order [T K] int32
 *   weights    [T][K] float32    or NULL: ones
 *   d_y        [T K][C] y_dtype  out
 *   d_weights  [T][K] float32    out, or NULL (then y is not read and may be NULL)
 */
int32_t eplb_combine_rows_backward(const void* d_out, int32_t dtype, const void* y, int32_t y_dtype, int64_t C,
                                   const int32_t* place, const int32_t* order, const float* weights, int64_t T,
                                   int32_t K, void* d_y, float* d_weights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EPLB_LAYER_H_ */
