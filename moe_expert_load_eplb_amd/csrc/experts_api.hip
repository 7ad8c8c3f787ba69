// C ABI of the router, the grouping and the experts' products: host-side
// validation, then launches.  Declarations and the meaning of every argument:
// include/eplb_experts.h.
#include "eplb_check.h"
#include "eplb_experts.h"
#include "experts_internal.h"

using namespace eplb;

namespace {

constexpr int64_t kMaxTiles = (int64_t(1) << 23) - 1;   // workgroups of one launch (512 work-items each at most)

int32_t result(hipError_t err) { return err == hipSuccess ? EPLB_OK : EPLB_E_HIP; }

bool known_dtype(int32_t d) { return d == EPLB_DTYPE_F32 || d == EPLB_DTYPE_BF16 || d == EPLB_DTYPE_F16; }

bool aligned(const void* p, int64_t n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

// Bytes of rows of n elements, ld apart.
int64_t span(int64_t rows, int64_t ld, int64_t n, int64_t size) {
  return rows <= 0 ? 0 : bytes_of(bytes_of(rows - 1, ld, 1) > INT64_MAX - n ? INT64_MAX : (rows - 1) * ld + n, size, 1);
}

int32_t check_router(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, int32_t K,
                     int32_t scoring) {
  if (T < 0 || E < 1 || K < 1 || ld < E || !known_dtype(dtype)) return EPLB_E_ARG;
  if (scoring != EPLB_SCORE_SIGMOID && scoring != EPLB_SCORE_SOFTMAX) return EPLB_E_ARG;
  if (T > kMaxTokens || E > kMaxE || K > kMaxK || ld > INT64_MAX / 8 / (T + 1)) return EPLB_E_LIMIT;
  if (T > 0 && (logits == nullptr || !aligned(logits, dtype_size(dtype)))) return EPLB_E_ARG;
  return EPLB_OK;
}

int32_t check_choice(int32_t E, int32_t K, int32_t G, int32_t top_groups, int32_t group_top) {
  if (K > E || G < 1 || top_groups < 1 || top_groups > G || group_top < 1 || group_top > 2) return EPLB_E_ARG;
  if (G > kMaxGroups) return EPLB_E_LIMIT;
  if (E % G != 0) return EPLB_E_DIV;
  if (group_top > E / G) return EPLB_E_ARG;
  return EPLB_OK;
}

int32_t check_loss(int64_t T, int32_t E, const int32_t* seg, int64_t S, const void* workspace,
                   int64_t workspace_bytes, const void* loss, const void* counts, const void* prob,
                   const void* tokens) {
  if (S < 1 || seg == nullptr || loss == nullptr || counts == nullptr || prob == nullptr || tokens == nullptr)
    return EPLB_E_ARG;
  if (S > kMaxSegments || S * ceil_div(E, 64) > kMaxLossParts) return EPLB_E_LIMIT;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < gate_loss_part_bytes(T, E, S))
    return EPLB_E_ARG;
  return EPLB_OK;
}

}  // namespace

extern "C" {

int32_t eplb_gate(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, int32_t K, int32_t scoring,
                  const float* bias, int32_t G, int32_t top_groups, int32_t group_top, int32_t normalize, float scale,
                  const uint8_t* mask, int32_t* ids, float* weights, void* stream) {
  int32_t rc = check_router(logits, dtype, ld, T, E, K, scoring);
  if (rc == EPLB_OK) rc = check_choice(E, K, G, top_groups, group_top);
  if (rc != EPLB_OK) return rc;
  if (T == 0) return EPLB_OK;
  if (ids == nullptr || weights == nullptr) return EPLB_E_ARG;
  const Range in[3] = {{logits, span(T, ld, E, dtype_size(dtype))}, {bias, E * 4}, {mask, T}};
  const Range out[2] = {{ids, T * K * 4}, {weights, T * K * 4}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  GateArgs a = {};
  a.logits = logits; a.ld = ld; a.T = T; a.dtype = dtype; a.E = E; a.K = K; a.scoring = scoring;
  a.G = G; a.top_groups = top_groups; a.group_top = group_top; a.normalize = normalize; a.scale = scale;
  a.bias = bias; a.mask = mask; a.ids = ids; a.weights = weights;
  a.fd_group = fastdiv_make((uint32_t)(E / G));
  return result(launch_gate(a, (hipStream_t)stream));
}

int64_t eplb_gate_loss_workspace_bytes(int64_t T, int32_t E, int64_t S) {
  if (T < 0 || E < 1 || S < 1) return -EPLB_E_ARG;
  if (T > kMaxTokens || E > kMaxE || S > kMaxSegments || S * ceil_div(E, 64) > kMaxLossParts) return -EPLB_E_LIMIT;
  return gate_loss_part_bytes(T, E, S);
}

int32_t eplb_gate_loss(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, int32_t K,
                       int32_t scoring, const float* bias, int32_t G, int32_t top_groups, int32_t group_top,
                       int32_t normalize, float scale, const uint8_t* mask, const int32_t* seg, int64_t S,
                       float alpha, void* workspace, int64_t workspace_bytes, int32_t* ids, float* weights,
                       float* loss, int32_t* counts, float* prob, int32_t* tokens, void* stream) {
  int32_t rc = check_router(logits, dtype, ld, T, E, K, scoring);
  if (rc == EPLB_OK) rc = check_choice(E, K, G, top_groups, group_top);
  if (rc == EPLB_OK) rc = check_loss(T, E, seg, S, workspace, workspace_bytes, loss, counts, prob, tokens);
  if (rc != EPLB_OK) return rc;
  if (T > 0 && (ids == nullptr || weights == nullptr)) return EPLB_E_ARG;
  const Range in[4] = {{logits, span(T, ld, E, dtype_size(dtype))}, {bias, E * 4}, {mask, T}, {seg, (S + 1) * 4}};
  const Range out[7] = {{ids, T * K * 4}, {weights, T * K * 4}, {loss, S * 4}, {counts, S * E * 4},
                        {prob, S * E * 4}, {tokens, S * 4}, {workspace, gate_loss_part_bytes(T, E, S)}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  GateArgs a = {};
  a.logits = logits; a.ld = ld; a.T = T; a.S = S; a.dtype = dtype; a.E = E; a.K = K; a.scoring = scoring;
  a.G = G; a.top_groups = top_groups; a.group_top = group_top; a.normalize = normalize; a.scale = scale;
  a.alpha = alpha; a.bias = bias; a.mask = mask; a.seg = seg; a.ids = ids; a.weights = weights;
  a.part = static_cast<float*>(workspace); a.loss = loss; a.counts = counts; a.prob = prob; a.tokens = tokens;
  a.fd_group = fastdiv_make((uint32_t)(E / G));
  return result(launch_gate_loss(a, (hipStream_t)stream));
}

int32_t eplb_balance_loss(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, const int32_t* ids,
                          int32_t K, int32_t scoring, const uint8_t* mask, const int32_t* seg, int64_t S, float alpha,
                          void* workspace, int64_t workspace_bytes, float* loss, int32_t* counts, float* prob,
                          int32_t* tokens, void* stream) {
  int32_t rc = check_router(logits, dtype, ld, T, E, K, scoring);
  if (rc == EPLB_OK) rc = check_loss(T, E, seg, S, workspace, workspace_bytes, loss, counts, prob, tokens);
  if (rc != EPLB_OK) return rc;
  if (T > 0 && ids == nullptr) return EPLB_E_ARG;
  const Range in[4] = {{logits, span(T, ld, E, dtype_size(dtype))}, {ids, T * K * 4}, {mask, T}, {seg, (S + 1) * 4}};
  const Range out[5] = {{loss, S * 4}, {counts, S * E * 4}, {prob, S * E * 4}, {tokens, S * 4},
                        {workspace, gate_loss_part_bytes(T, E, S)}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  GateArgs a = {};
  a.logits = logits; a.ld = ld; a.T = T; a.S = S; a.dtype = dtype; a.E = E; a.K = K; a.scoring = scoring;
  a.G = a.top_groups = a.group_top = 1; a.alpha = alpha; a.mask = mask; a.seg = seg;
  a.given = 1; a.ids = const_cast<int32_t*>(ids);
  a.part = static_cast<float*>(workspace); a.loss = loss; a.counts = counts; a.prob = prob; a.tokens = tokens;
  return result(launch_gate_loss(a, (hipStream_t)stream));
}

int32_t eplb_gate_backward(const void* logits, int32_t dtype, int64_t ld, int64_t T, int32_t E, const int32_t* ids,
                           int32_t K, int32_t scoring, int32_t normalize, float scale, const uint8_t* mask,
                           const float* d_weights, const int32_t* seg, int64_t S, float alpha, const int32_t* counts,
                           const int32_t* tokens, const float* d_loss, void* d_logits, void* stream) {
  int32_t rc = check_router(logits, dtype, ld, T, E, K, scoring);
  if (rc != EPLB_OK) return rc;
  if (d_loss != nullptr) {
    if (S < 1 || seg == nullptr || counts == nullptr || tokens == nullptr) return EPLB_E_ARG;
    if (S > kMaxSegments) return EPLB_E_LIMIT;
  } else {
    S = 0;
  }
  if (T == 0) return EPLB_OK;
  if (d_logits == nullptr || !aligned(d_logits, dtype_size(dtype))) return EPLB_E_ARG;
  if (d_weights != nullptr && ids == nullptr) return EPLB_E_ARG;
  const Range in[8] = {{logits, span(T, ld, E, dtype_size(dtype))}, {ids, T * K * 4}, {mask, T},
                       {d_weights, T * K * 4}, {seg, S > 0 ? (S + 1) * 4 : 0}, {counts, S * E * 4}, {tokens, S * 4},
                       {d_loss, S * 4}};
  const Range out[1] = {{d_logits, T * E * dtype_size(dtype)}};
  rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  GateBackwardArgs a = {};
  a.logits = logits; a.ld = ld; a.T = T; a.S = S; a.dtype = dtype; a.E = E; a.K = K; a.scoring = scoring;
  a.normalize = normalize; a.scale = scale; a.alpha = alpha; a.mask = mask; a.ids = ids; a.d_weights = d_weights;
  a.seg = seg; a.counts = counts; a.tokens = tokens; a.d_loss = d_loss; a.d_logits = d_logits;
  return result(launch_gate_backward(a, (hipStream_t)stream));
}

int64_t eplb_group_rows_workspace_bytes(int64_t L, int64_t n, int32_t P) {
  if (L < 0 || n < 0 || P < 1) return -EPLB_E_ARG;
  if (P > kMaxSlots || L > kMaxLayers) return -EPLB_E_LIMIT;
  if (n > kMaxRows) return -EPLB_E_RANGE;
  if (!group_rows_fits(L, n, P)) return -EPLB_E_LIMIT;
  return group_rows_bytes(L, n, P);
}

int32_t eplb_group_rows(const int32_t* ids, int64_t L, int64_t n, int32_t first, int32_t P, void* workspace,
                        int64_t workspace_bytes, int32_t* offsets, int32_t* order, int32_t* place, void* stream) {
  const int64_t need = eplb_group_rows_workspace_bytes(L, n, P);
  if (need < 0) return (int32_t)-need;
  if (L == 0) return EPLB_OK;
  if (offsets == nullptr || (n > 0 && (ids == nullptr || order == nullptr || place == nullptr))) return EPLB_E_ARG;
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 4) || workspace_bytes < need)) return EPLB_E_ARG;
  const Range in[1] = {{ids, L * n * 4}};
  const Range out[4] = {{offsets, L * (P + 1) * 4}, {order, L * n * 4}, {place, L * n * 4}, {workspace, need}};
  const int32_t rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  return result(launch_group_rows(ids, L, n, first, P, static_cast<int32_t*>(workspace), offsets, order, place,
                                  (hipStream_t)stream));
}

int32_t eplb_quantize_rows(const void* x, int32_t dtype, int64_t ld, int64_t R, int64_t C, uint8_t* q, float* scale,
                           void* stream) {
  if (R < 0 || C < 1 || ld < C || !known_dtype(dtype)) return EPLB_E_ARG;
  if (C > kMaxDim || R > kMaxRows || ld > INT64_MAX / 8 / (R + 1)) return EPLB_E_LIMIT;
  if (R == 0) return EPLB_OK;
  if (!aligned(x, dtype_size(dtype))) return EPLB_E_ARG;
  const Range in[1] = {{x, span(R, ld, C, dtype_size(dtype))}};
  const Range out[2] = {{q, R * C}, {scale, R * ceil_div(C, kBlock) * 4}};
  const int32_t rc = check_buffers(in, out);
  if (rc != EPLB_OK) return rc;
  return result(launch_quantize_rows(x, dtype, ld, R, C, q, scale, (hipStream_t)stream));
}

int32_t eplb_quantize_columns(const void* x, int32_t dtype, int64_t ld, int64_t X, int64_t C, const int32_t* rows,
                              int64_t R, int32_t K, const int32_t* offsets, int32_t G, int64_t Rp, uint8_t* q,
                              float* scale, void* stream) {
  if (X < 0 || C < 1 || ld < C || R < 0 || K < 1 || G < 1 || !known_dtype(dtype)) return EPLB_E_ARG;
  if (C > kMaxDim || X > kMaxRows || R > kMaxRows || G > kMaxSlots || Rp > kMaxPadded || ld > INT64_MAX / 8 / (X + 1))
    return EPLB_E_LIMIT;
  if (Rp % kBlock != 0 || Rp < (R + (kBlock - 1) * (int64_t)G) / kBlock * kBlock) return EPLB_E_ARG;
  if (Rp / kBlock * ceil_div(C, kBlock) > kMaxTiles) return EPLB_E_LIMIT;
  if (R == 0) return EPLB_OK;
  if (offsets == nullptr || (X > 0 && x == nullptr) || q == nullptr || scale == nullptr) return EPLB_E_ARG;
  if (!aligned(x, dtype_size(dtype)) || !aligned(q, 16)) return EPLB_E_ARG;
  const Range in[3] = {{x, span(X, ld, C, dtype_size(dtype))}, {rows, R * 4}, {offsets, (G + 1) * (int64_t)4}};
  const Range out[2] = {{q, C * Rp}, {scale, Rp / kBlock * C * 4}};
  const int32_t rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  return result(launch_quantize_columns(x, dtype, ld, X, C, rows, R, K, offsets, G, Rp, q, scale,
                                        (hipStream_t)stream));
}

int32_t eplb_quantize_weights(const void* w, int32_t dtype, int32_t G, int64_t N, int64_t K, uint8_t* q, float* scale,
                              uint8_t* qt, float* scale_t, void* stream) {
  if (G < 0 || N < 1 || K < 1 || !known_dtype(dtype) || (qt == nullptr) != (scale_t == nullptr)) return EPLB_E_ARG;
  if (G > kMaxSlots || N > kMaxDim || K > kMaxDim) return EPLB_E_LIMIT;
  const int64_t blocks = ceil_div(N, kBlock) * ceil_div(K, kBlock);
  if (G * blocks > kMaxTiles) return EPLB_E_LIMIT;
  if (G == 0) return EPLB_OK;
  if (!aligned(w, dtype_size(dtype))) return EPLB_E_ARG;
  const int64_t n = G * N * K;
  const Range in[1] = {{w, n * dtype_size(dtype)}};
  const Range out[2] = {{q, n}, {scale, G * blocks * 4}};
  int32_t rc = check_buffers(in, out);
  if (rc != EPLB_OK) return rc;
  const Range outs[4] = {{q, n}, {scale, G * blocks * 4}, {qt, n}, {scale_t, G * blocks * 4}};
  rc = check_disjoint(in, outs);
  if (rc != EPLB_OK) return rc;
  return result(launch_quantize_weights(w, dtype, G, N, K, q, scale, qt, scale_t, (hipStream_t)stream));
}

int32_t eplb_expert_matmul(const uint8_t* q, const float* scale, int64_t X, const uint8_t* w, const float* w_scale,
                           const int32_t* offsets, int32_t G, const int32_t* rows, int64_t R, int32_t topk, int64_t N,
                           int64_t K, int32_t dtype, void* y, void* stream) {
  if (X < 0 || G < 1 || R < 0 || topk < 1 || N < 1 || K < 1 || K % 16 != 0 || !known_dtype(dtype)) return EPLB_E_ARG;
  if (N > kMaxDim || K > kMaxDim || R > kMaxRows || X > kMaxRows || G > kMaxSlots) return EPLB_E_LIMIT;
  if (matmul_tiles(R, N, K, G) > kMaxTiles) return EPLB_E_LIMIT;
  if (R == 0) return EPLB_OK;
  if (w == nullptr || w_scale == nullptr || offsets == nullptr || y == nullptr) return EPLB_E_ARG;
  if (X > 0 && (q == nullptr || scale == nullptr)) return EPLB_E_ARG;
  if (!aligned(q, 16) || !aligned(w, 16) || !aligned(y, 16)) return EPLB_E_ARG;
  const int64_t KB = ceil_div(K, kBlock), NB = ceil_div(N, kBlock);
  const Range in[6] = {{q, X * K}, {scale, X * KB * 4}, {w, G * N * K}, {w_scale, G * NB * KB * 4},
                       {offsets, (G + 1) * (int64_t)4}, {rows, R * 4}};
  const Range out[1] = {{y, R * N * dtype_size(dtype)}};
  const int32_t rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  MatmulArgs a = {};
  a.q = q; a.scale = scale; a.w = w; a.w_scale = w_scale; a.offsets = offsets; a.rows = rows; a.y = y;
  a.X = X; a.R = (int32_t)R; a.N = (int32_t)N; a.K = (int32_t)K; a.KB = (int32_t)KB; a.NB = (int32_t)NB; a.G = G;
  a.topk = topk; a.dtype = dtype; a.fd_topk = fastdiv_make((uint32_t)topk);
  return result(launch_expert_matmul(a, (hipStream_t)stream));
}

int32_t eplb_expert_wgrad(const uint8_t* dy, const float* dy_scale, const uint8_t* x, const float* x_scale,
                          const int32_t* offsets, int32_t G, int64_t R, int64_t Rp, int64_t N, int64_t K,
                          int32_t dtype, void* dw, void* stream) {
  if (G < 1 || R < 0 || N < 1 || K < 1 || !known_dtype(dtype)) return EPLB_E_ARG;
  if (N > kMaxDim || K > kMaxDim || R > kMaxRows || G > kMaxSlots || Rp > kMaxPadded) return EPLB_E_LIMIT;
  if (Rp % kBlock != 0 || Rp < (R + (kBlock - 1) * (int64_t)G) / kBlock * kBlock) return EPLB_E_ARG;
  if (wgrad_tiles(N, K, G) > kMaxTiles) return EPLB_E_LIMIT;
  if (offsets == nullptr || dw == nullptr || !aligned(dw, 16)) return EPLB_E_ARG;
  if (R > 0 && (dy == nullptr || dy_scale == nullptr || x == nullptr || x_scale == nullptr)) return EPLB_E_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16)) return EPLB_E_ARG;
  const int64_t blocks = R > 0 ? Rp / kBlock : 0;
  const Range in[5] = {{dy, N * blocks * kBlock}, {dy_scale, blocks * N * 4}, {x, K * blocks * kBlock},
                       {x_scale, blocks * K * 4}, {offsets, (G + 1) * (int64_t)4}};
  const Range out[1] = {{dw, G * N * K * dtype_size(dtype)}};
  const int32_t rc = check_disjoint(in, out);
  if (rc != EPLB_OK) return rc;
  WgradArgs a = {};
  a.dy = dy; a.dy_scale = dy_scale; a.x = x; a.x_scale = x_scale; a.offsets = offsets; a.dw = dw;
  a.Rp = Rp; a.R = (int32_t)R; a.N = (int32_t)N; a.K = (int32_t)K; a.G = G; a.dtype = dtype;
  return result(launch_expert_wgrad(a, (hipStream_t)stream));
}

}  // extern "C"
