/*
 * eplb_experts.h -- C ABI of what stands before and behind the EPLB hot path
 * on AMD Instinct MI355X (gfx950), in the same library.
 *
 * Before it: the router that makes the top-k ids, its balance loss with the
 * per-expert counts, and the gradients of both.  Behind it: the redirected
 * rows grouped by physical slot, and the experts' products in 8-bit floating
 * point with a scale for each block of 128, with their gradients.
 *
 * The conventions, return codes and ownership rules are those of eplb.h.
 */
#ifndef EPLB_EXPERTS_H_
#define EPLB_EXPERTS_H_

#include "eplb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- types and choices of the router and the products -------------------- */
#define EPLB_DTYPE_F32     0  /* 32-bit floating point                             */
#define EPLB_DTYPE_BF16    1  /* bfloat16                                          */
#define EPLB_DTYPE_F16     2  /* IEEE half precision                               */
#define EPLB_SCORE_SIGMOID 0  /* s = 1 / (1 + exp(-x))                             */
#define EPLB_SCORE_SOFTMAX 1  /* s = exp(x - max x) / sum exp(x - max x)           */

/*
 * eplb_gate -- the router: for every token the K experts with the largest
 * keys, and their weights.
 *
 *   s[t][e]   = sigmoid or softmax of the token's logits, in 32 bits
 *   key[t][e] = s + bias (sigmoid) or logit + bias (softmax), one 32-bit sum
 * With G groups of E / G consecutive experts and top_groups < G, only the
 * experts of the top_groups best groups may be chosen; a group's score is the
 * sum of its group_top (1 or 2) largest keys.  Of the experts left, the K
 * largest keys are chosen, in descending order; equal keys (and equal group
 * scores) go to the lowest index.  An expert whose logit or key is minus
 * infinity or NaN is never chosen: where fewer than K experts are left, the
 * remaining ids are -1 and their weights 0.  The weights are the scores,
 * without the bias:
 *   w[t][k] = scale * s[t][ids[t][k]] / (sum over the chosen of s + 1e-20)
 * or, with normalize = 0, scale * s.  A row whose mask byte is 0 (padding)
 * gets ids -1 and weights 0.
 *
 *   logits     [T][E] dtype      router logits, rows `ld` elements apart
 *                                (ld >= E); a softmax row with a logit of plus
 *                                infinity or NaN has the formula's NaN scores
 *   dtype                        EPLB_DTYPE_* of logits
 *   T, E, K                      tokens (0 .. 2^25), experts (1 .. 4096),
 *                                choices (1 .. 64, at most E)
 *   scoring                      EPLB_SCORE_*
 *   bias       [E] float32       or NULL: added to the key only
 *   G, top_groups, group_top     G divides E, G <= 64, 1 <= top_groups <= G,
 *                                group_top 1 or 2 (at most E / G)
 *   mask       [T] uint8         or NULL: 0 marks a row to leave out
 *   ids        [T][K] int32      out: chosen experts (eplb_redirect's input)
 *   weights    [T][K] float32    out
 *
 * Errors: EPLB_E_ARG (a size outside its range, ld < E, an unknown dtype or
 * scoring, a NULL array, an output sharing a byte with an input or another
 * output), EPLB_E_DIV (E % G), EPLB_E_LIMIT (T > 2^25, E > 4096, K > 64,
 * G > 64), EPLB_E_HIP.
 */
int32_t eplb_gate(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, int32_t K, int32_t scoring,
                  const float* bias, int32_t G, int32_t top_groups, int32_t group_top, int32_t normalize, float scale,
                  const uint8_t* mask, int32_t* ids, float* weights, void* stream);

/*
 * eplb_gate_loss -- eplb_gate with the balance loss and per-expert counts of
 * S segments of rows (sequences, or one segment for the whole batch):
 *   n      = rows of the segment that the mask keeps
 *   counts[e] = how often expert e was chosen by them
 *   prob[e]   = (1 / n) sum of share[t][e], share = s / (sum over e of s +
 *               1e-20) for sigmoid, s for softmax
 *   loss   = alpha * sum over e of (E * counts[e] / (K * n)) * prob[e]
 * All are 0 for a segment with n = 0.  Sums are taken in a fixed order: equal
 * inputs give equal bits.
 *
 *   seg        [S + 1] int32     segment s holds rows seg[s] .. seg[s + 1] - 1;
 *                                non-decreasing within 0 .. T.  Rows of no
 *                                segment are routed and counted nowhere.
 *   workspace                    at least eplb_gate_loss_workspace_bytes(T, E,
 *                                S) bytes, 16-byte aligned, overwritten
 *   loss       [S] float32       out
 *   counts     [S][E] int32      out
 *   prob       [S][E] float32    out
 *   tokens     [S] int32         out: n of each segment
 * Other arguments and errors: as for eplb_gate; S is 1 .. 2^20 and S * ceil(E
 * / 64) at most 2^21 (EPLB_E_LIMIT); EPLB_E_ARG also for a workspace that is
 * too small, misaligned, or shares a byte with another array.
 */
int32_t eplb_gate_loss(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, int32_t K,
                       int32_t scoring, const float* bias, int32_t G, int32_t top_groups, int32_t group_top,
                       int32_t normalize, float scale, const uint8_t* mask, const int32_t* seg, int64_t S,
                       float alpha, void* workspace, int64_t workspace_bytes, int32_t* ids, float* weights,
                       float* loss, int32_t* counts, float* prob, int32_t* tokens, void* stream);

/* Bytes of workspace for eplb_gate_loss and eplb_balance_loss, or a negative
 * EPLB_E_* code.  Host only. */
int64_t eplb_gate_loss_workspace_bytes(int64_t T, int32_t E, int64_t S);

/*
 * eplb_balance_loss -- the loss, counts and probabilities of eplb_gate_loss
 * for choices made elsewhere: ids [T][K] is an input (an id outside [0, E) is
 * no choice).  Other arguments and errors: as for eplb_gate_loss.
 */
int32_t eplb_balance_loss(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, const int32_t* ids,
                          int32_t K, int32_t scoring, const uint8_t* mask, const int32_t* seg, int64_t S, float alpha,
                          void* workspace, int64_t workspace_bytes, float* loss, int32_t* counts, float* prob,
                          int32_t* tokens, void* stream);

/*
 * eplb_gate_backward -- gradient with respect to the logits of
 *   sum of d_weights * weights  +  sum of d_loss * loss
 * with the choices and the counts held fixed (they are piecewise constant).
 *
 *   ids        [T][K] int32      choices (an id outside [0, E): none)
 *   d_weights  [T][K] float32    or NULL: no gradient through the weights
 *   d_loss     [S] float32       or NULL: no gradient through the loss; then
 *                                seg, counts and tokens are not read
 *   counts, tokens               as eplb_gate_loss or eplb_balance_loss wrote
 *                                them
 *   d_logits   [T][E] dtype      out, contiguous; rows the mask leaves out: 0
 * Other arguments and errors: as for eplb_gate_loss.
 */
int32_t eplb_gate_backward(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, const int32_t* ids,
                           int32_t K, int32_t scoring, int32_t normalize, float scale, const uint8_t* mask,
                           const float* d_weights, const int32_t* seg, int64_t S, float alpha, const int32_t* counts,
                           const int32_t* tokens, const float* d_loss, void* d_logits, void* stream);

/*
 * eplb_group_rows -- the rows (t, k) of every layer grouped by slot, as the
 * experts' products read them: a stable counting sort of the physical ids.
 *
 *   ids        [L][n] int32      physical ids (n = T * K); slot g holds the
 *                                ids equal to first + g, 0 <= g < P
 *   first, P                     the slots kept (one rank's, for instance)
 *   offsets    [L][P + 1] int32  out: rows offsets[g] .. offsets[g + 1] - 1
 *                                of the grouped order belong to slot g
 *   order      [L][n] int32      out: position in ids of each grouped row;
 *                                ids of no slot come last, in order
 *   place      [L][n] int32      out: the inverse, order[place[i]] = i
 *   workspace                    at least eplb_group_rows_workspace_bytes(L,
 *                                n, P) bytes, 4-byte aligned (0: NULL is fine)
 *
 * Errors: EPLB_E_ARG (L or n < 0, P < 1, a NULL array, a workspace too small,
 * misaligned or sharing a byte, outputs sharing a byte), EPLB_E_LIMIT
 * (P > 8192, more than 2^22 segments: L * min(ceil(n / 2048), 256)), EPLB_E_RANGE
 * (n >= 2^31), EPLB_E_HIP.
 */
int32_t eplb_group_rows(const int32_t* ids, int64_t L, int64_t n, int32_t first, int32_t P, void* workspace,
                        int64_t workspace_bytes, int32_t* offsets, int32_t* order, int32_t* place, void* stream);
int64_t eplb_group_rows_workspace_bytes(int64_t L, int64_t n, int32_t P);

/*
 * 8-bit floating point with a scale for each block of 128: values are the
 * format with 1 sign, 4 exponent and 3 mantissa bits (largest 448, no
 * infinities), one byte each.  A block's scale and values are
 *   a = max(largest |x| of the block, 2^-100),  scale = a * (1 / 448),
 *   q = x * ((1 / a) * 448) rounded to the nearest value, ties to even
 * with each operation rounded to 32 bits, so that q * scale stands for x.  A block
 * that holds an infinity or a NaN gets the scale NaN and all its values 0:
 * whatever is computed from it is NaN.
 *
 * eplb_quantize_rows -- blocks of 128 along each row (the last one shorter).
 *   x          [R][C] dtype      rows ld elements apart
 *   q          [R][C] 8-bit      out
 *   scale      [R][ceil(C / 128)] float32  out
 *
 * Errors of the three calls: EPLB_E_ARG (a size < 1 where one is needed, ld
 * < C, an unknown dtype, a NULL array, a pointer not aligned, an output sharing
 * a byte with an input or another output, Rp not as below), EPLB_E_LIMIT (C or N
 * or K > 2^24, R or X > 2^31 - 1, Rp > 2^32, G > 8192, or more than 2^23 - 1
 * blocks of 128 x 128 of columns or weights), EPLB_E_HIP.
 */
int32_t eplb_quantize_rows(const void* x, int32_t dtype, int64_t ld, int64_t R, int64_t C, uint8_t* q, float* scale,
                           void* stream);

/*
 * eplb_quantize_columns -- the operand of a weight gradient: grouped rows
 * transposed, with blocks of 128 rows.  Group g's rows offsets[g] ..
 * offsets[g + 1] - 1 take the columns from pad[g] on, pad[0] = 0, pad[g + 1] =
 * pad[g] + its rows rounded up to 128; columns past a group's rows hold 0.
 *   x          [.][C] dtype      rows ld elements apart
 *   rows       [R] int32         or NULL: grouped row r reads row rows[r] /
 *                                K of x (eplb_group_rows' order); without it
 *                                row r reads row r
 *   X                            rows that x has: a row outside [0, X) is zero
 *   offsets    [G + 1] int32     eplb_group_rows': non-decreasing.  Values are
 *                                clamped to 0 .. R, a group that ends before it
 *                                starts is empty.  Offsets that decrease make
 *                                groups that share rows: nothing outside the
 *                                arrays is reached, but what the outputs hold
 *                                for such groups and rows is not defined
 *   Rp                           columns of q: a multiple of 128, at least
 *                                R + 127 G rounded down to one
 *   q          [C][Rp] 8-bit     out: columns below pad[G]; 16-byte aligned
 *   scale      [Rp / 128][C] float32  out: blocks below pad[G] / 128
 */
int32_t eplb_quantize_columns(const void* x, int32_t dtype, int64_t ld, int64_t X, int64_t C, const int32_t* rows,
                              int64_t R, int32_t K, const int32_t* offsets, int32_t G, int64_t Rp, uint8_t* q,
                              float* scale, void* stream);

/*
 * eplb_quantize_weights -- blocks of 128 x 128 (shorter at the ends).
 *   w          [G][N][K] dtype   contiguous
 *   q          [G][N][K] 8-bit   out
 *   scale      [G][ceil(N / 128)][ceil(K / 128)] float32  out
 *   qt, scale_t                  or NULL, both: out: the same values
 *                                transposed, [G][K][N] and [G][ceil(K / 128)]
 *                                [ceil(N / 128)], the weights of the gradient
 *                                with respect to the product's input
 */
int32_t eplb_quantize_weights(const void* w, int32_t dtype, int32_t G, int64_t N, int64_t K, uint8_t* q, float* scale,
                              uint8_t* qt, float* scale_t, void* stream);

/*
 * eplb_expert_matmul -- the experts' product: every grouped row times the
 * transposed weights of its expert,
 *   y[r][n] = sum over blocks b of scale[x(r)][b] * w_scale[g][n / 128][b]
 *             * (sum over k in b of q[x(r)][k] * w[g][n][k])
 * where g is the group of row r and x(r) = rows[r] / topk, or r without rows.
 * All sums are held in 32 bits and the result is rounded once.  Equal inputs
 * give equal bits.  Rows of no group, and rows whose x(r) is
 * outside [0, X), get zeros.
 *
 *   q          [X][K] 8-bit      and scale [X][ceil(K / 128)] float32, as
 *                                eplb_quantize_rows writes them
 *   w          [G][N][K] 8-bit   and w_scale [G][ceil(N / 128)][ceil(K / 128)]
 *                                float32, as eplb_quantize_weights writes them
 *   offsets    [G + 1] int32     eplb_group_rows'; clamped as above
 *   rows       [R] int32         or NULL
 *   N, K                         1 .. 2^24; K a multiple of 16; q, w and y
 *                                16-byte aligned
 *   y          [R][N] dtype      out
 * With G = 1 and offsets {0, R} this is the plain product of two matrices.
 *
 * Errors: EPLB_E_ARG (a size outside its range, K % 16, a pointer not
 * aligned, an unknown dtype, a NULL array, y sharing a byte with an input),
 * EPLB_E_LIMIT (N or K > 2^24, R or X > 2^31 - 1, G > 8192, or more than
 * 2^23 - 1 tiles of the output), EPLB_E_HIP.
 */
int32_t eplb_expert_matmul(const uint8_t* q, const float* scale, int64_t X, const uint8_t* w, const float* w_scale,
                           const int32_t* offsets, int32_t G, const int32_t* rows, int64_t R, int32_t topk, int64_t N,
                           int64_t K, int32_t dtype, void* y, void* stream);

/*
 * eplb_expert_wgrad -- the gradient of that product with respect to the
 * weights: for every group g, summed over its blocks b of 128 rows,
 *   dw[g][n][k] = sum over b of dy_scale[b][n] * x_scale[b][k]
 *                 * (sum over r in b of dy[n][r] * x[k][r])
 *   dy         [N][Rp] 8-bit     and dy_scale [Rp / 128][N], x [K][Rp] and
 *                                x_scale [Rp / 128][K]: eplb_quantize_columns'
 *                                outputs for the same offsets and Rp
 *   dw         [G][N][K] dtype   out: zeros for a group without rows
 * dy, x and dw are 16-byte aligned.  All sums are held in 32 bits.
 * Errors: as for eplb_expert_matmul; Rp as for eplb_quantize_columns.
 */
int32_t eplb_expert_wgrad(const uint8_t* dy, const float* dy_scale, const uint8_t* x, const float* x_scale,
                          const int32_t* offsets, int32_t G, int64_t R, int64_t Rp, int64_t N, int64_t K,
                          int32_t dtype, void* dw, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EPLB_EXPERTS_H_ */
