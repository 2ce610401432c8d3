// capi_fp8.hip -- the extern "C" entry points of the 8-bit floating-point operators and of the
// balance loss (see include/bgt.h). Arguments are validated on the host before the first HIP
// call, as in capi.hip.
#include <stdint.h>

#include "bgt.h"
#include "launch.h"

namespace {

bool valid_type(int t) { return t == BGT_F32 || t == BGT_F16 || t == BGT_BF16; }
int type_bytes(int t) { return t == BGT_F32 ? 4 : 2; }
bool aligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}
// a launch past the grid's limits is refused by the launchers before anything runs
int hip_status(hipError_t e) {
  return e == hipSuccess ? BGT_OK : e == hipErrorInvalidConfiguration ? BGT_ERR_SHAPE : BGT_ERR_HIP;
}
hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }

constexpr int64_t kMaxRows = 1 << 24, kMaxCols = 1 << 18;

bool rows_ok(int64_t M, int64_t K) { return M >= 1 && M <= kMaxRows && K >= 1 && K <= kMaxCols; }
bool route_ok(int64_t T, int64_t E, int64_t R) {
  return T >= 1 && T <= kMaxRows && E >= 1 && E <= 256 && R >= 1 && R <= kMaxRows && R <= T * E;
}
int64_t padded(int64_t n) { return (n + BGT_GROUP - 1) / BGT_GROUP * BGT_GROUP; }

bgt::Route route_of(const int32_t* offs, const int32_t* tok, int64_t T, int64_t E, int64_t R,
                    int64_t N, int64_t K) {
  return bgt::Route{offs, tok, (int)E, (int)T, (int)R, N * padded(K),
                    padded(K) / BGT_GROUP * (padded(N) / BGT_GROUP)};
}

}  // namespace

extern "C" {

int bgt_quantize_fp8(const void* x, int x_type, int64_t M, int64_t K, int64_t ldx, uint8_t* q,
                     uint8_t* scale, void* stream) {
  if (!x || !q || !scale) return BGT_ERR_NULL;
  if (!valid_type(x_type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K) || ldx < K) return BGT_ERR_SHAPE;
  if (!aligned(x, type_bytes(x_type)) || !aligned(q, 16)) return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_rows(x, x_type, M, K, ldx, q, scale, stream_of(stream)));
}

int bgt_dequantize_fp8(const uint8_t* q, const uint8_t* scale, int64_t M, int64_t K, void* y,
                       int y_type, void* stream) {
  if (!q || !scale || !y) return BGT_ERR_NULL;
  if (!valid_type(y_type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K)) return BGT_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(y, type_bytes(y_type))) return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_values(q, scale, M, K, y, y_type, stream_of(stream)));
}

int bgt_pack_weights_fp8(const void* w, int w_type, int64_t E, int64_t K, int64_t N, uint8_t* qw,
                         uint8_t* sw, uint8_t* qt, uint8_t* st, void* stream) {
  if (!w || !qw || !sw || (!qt) != (!st)) return BGT_ERR_NULL;
  if (!valid_type(w_type)) return BGT_ERR_MODE;
  if (E < 1 || E > 256 || !rows_ok(N, K) || N > kMaxCols) return BGT_ERR_SHAPE;
  if (!aligned(w, type_bytes(w_type)) || !aligned(qw, 16) || (qt && !aligned(qt, 16)))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_weights(w, w_type, E, K, N, qw, sw, qt, st, stream_of(stream)));
}

int bgt_w8a8_gemm_fp8(const uint8_t* qx, const uint8_t* sx, const uint8_t* qw, const uint8_t* sw,
                      int64_t M, int64_t N, int64_t K, void* y, int y_type, void* stream) {
  if (!qx || !sx || !qw || !sw || !y) return BGT_ERR_NULL;
  if (!valid_type(y_type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K) || N < 1 || N > kMaxCols) return BGT_ERR_SHAPE;
  if (!aligned(qx, 16) || !aligned(qw, 16) || !aligned(y, type_bytes(y_type))) return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_w8a8_f8(qx, sx, qw, sw, M, N, padded(K), bgt::OutY{y, y_type},
                                        stream_of(stream)));
}

int bgt_w8a8_linear_fp8(const void* x, int x_type, int64_t ldx, const uint8_t* qw,
                        const uint8_t* sw, int64_t M, int64_t N, int64_t K, uint8_t* qx,
                        uint8_t* sx, void* y, int y_type, void* stream) {
  if (!x || !qw || !sw || !qx || !sx || !y) return BGT_ERR_NULL;
  if (!valid_type(x_type) || !valid_type(y_type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K) || N < 1 || N > kMaxCols || ldx < K) return BGT_ERR_SHAPE;
  if (!aligned(x, type_bytes(x_type)) || !aligned(qx, 16) || !aligned(qw, 16) ||
      !aligned(y, type_bytes(y_type)))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_w8a8_f8_linear(x, x_type, ldx, K, qw, sw, M, N, padded(K), qx, sx,
                                               bgt::OutY{y, y_type}, stream_of(stream)));
}

int bgt_w8a8_moe_gemm_fp8(const uint8_t* qx, const uint8_t* sx, int64_t T,
                          const int32_t* expert_offsets, const int32_t* slot_token, int64_t E,
                          int64_t R, const uint8_t* qw, const uint8_t* sw, int64_t N, int64_t K,
                          void* y, int y_type, void* stream) {
  if (!qx || !sx || !expert_offsets || !slot_token || !qw || !sw || !y) return BGT_ERR_NULL;
  if (!valid_type(y_type)) return BGT_ERR_MODE;
  if (!route_ok(T, E, R) || N < 1 || N > kMaxCols || K < 1 || K > kMaxCols) return BGT_ERR_SHAPE;
  if (!aligned(qx, 16) || !aligned(qw, 16) || !aligned(y, type_bytes(y_type)) ||
      !aligned(expert_offsets, 4) || !aligned(slot_token, 4))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_w8a8_f8_moe(qx, sx, qw, sw, N, padded(K),
                                            route_of(expert_offsets, slot_token, T, E, R, N, K),
                                            bgt::OutY{y, y_type}, stream_of(stream)));
}

int64_t bgt_wgrad_fp8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (!rows_ok(M, K) || N < 1 || N > kMaxCols) return BGT_ERR_SHAPE;
  return bgt::f8_wgrad_ws_bytes(M, K, N);
}

int bgt_wgrad_fp8(const uint8_t* qx, const uint8_t* sx, const void* dy, int type, int64_t lddy,
                  int64_t M, int64_t K, int64_t N, void* dw, void* ws, int64_t ws_bytes,
                  void* stream) {
  if (!qx || !sx || !dy || !dw) return BGT_ERR_NULL;
  if (!valid_type(type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K) || N < 1 || N > kMaxCols || lddy < N) return BGT_ERR_SHAPE;
  const int64_t need = bgt::f8_wgrad_ws_bytes(M, K, N);
  if (need > 0 && !ws) return BGT_ERR_NULL;
  if (ws_bytes < need) return BGT_ERR_SHAPE;
  const int b = type_bytes(type);
  if (!aligned(qx, 16) || !aligned(dy, b) || !aligned(dw, b) || (need > 0 && !aligned(ws, 4)))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_wgrad(qx, sx, dy, lddy, M, K, N, bgt::Route{},
                                         bgt::OutY{dw, type}, ws, stream_of(stream)));
}

int bgt_moe_wgrad_fp8(const uint8_t* qx, const uint8_t* sx, int64_t T,
                      const int32_t* expert_offsets, const int32_t* slot_token, int64_t E,
                      int64_t R, const void* dy, int type, int64_t lddy, int64_t K, int64_t N,
                      void* dw, void* stream) {
  if (!qx || !sx || !expert_offsets || !slot_token || !dy || !dw) return BGT_ERR_NULL;
  if (!valid_type(type)) return BGT_ERR_MODE;
  if (!route_ok(T, E, R) || N < 1 || N > kMaxCols || K < 1 || K > kMaxCols || lddy < N)
    return BGT_ERR_SHAPE;
  const int b = type_bytes(type);
  if (!aligned(qx, 16) || !aligned(dy, b) || !aligned(dw, b) || !aligned(expert_offsets, 4) ||
      !aligned(slot_token, 4))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_wgrad(qx, sx, dy, lddy, T, K, N,
                                         route_of(expert_offsets, slot_token, T, E, R, N, K),
                                         bgt::OutY{dw, type}, nullptr, stream_of(stream)));
}

int bgt_silu_mul_fp8(const void* gate, int64_t ldg, const void* up, int64_t ldu, int type,
                     int64_t M, int64_t K, uint8_t* hq, uint8_t* hs, uint8_t* gq, uint8_t* gs,
                     uint8_t* uq, uint8_t* us, void* stream) {
  if (!gate || !up || !hq || !hs || !gq || !gs || !uq || !us) return BGT_ERR_NULL;
  if (!valid_type(type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K) || ldg < K || ldu < K) return BGT_ERR_SHAPE;
  const int b = type_bytes(type);
  if (!aligned(gate, b) || !aligned(up, b) || !aligned(hq, 16) || !aligned(gq, 16) ||
      !aligned(uq, 16))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_gate(gate, ldg, up, ldu, type, M, K, hq, hs, gq, gs, uq, us,
                                        stream_of(stream)));
}

int bgt_silu_mul_fp8_backward(const void* dh, int type, int64_t ld, const uint8_t* gq,
                              const uint8_t* gs, const uint8_t* uq, const uint8_t* us, int64_t M,
                              int64_t K, void* dg, void* du, void* stream) {
  if (!dh || !gq || !gs || !uq || !us || !dg || !du) return BGT_ERR_NULL;
  if (!valid_type(type)) return BGT_ERR_MODE;
  if (!rows_ok(M, K) || ld < K) return BGT_ERR_SHAPE;
  const int b = type_bytes(type);
  if (!aligned(dh, b) || !aligned(dg, b) || !aligned(du, b) || !aligned(gq, 16) || !aligned(uq, 16))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_f8_gate_grad(dh, ld, type, gq, gs, uq, us, M, K, dg, du,
                                             stream_of(stream)));
}

namespace {

int check_balance(int64_t T, int64_t E, int64_t k) {
  if (E < 1 || E > 256 || k < 1 || k > 16 || k > E) return BGT_ERR_SHAPE;
  return T >= 1 && T <= kMaxRows / k ? BGT_OK : BGT_ERR_SHAPE;
}

}  // namespace

int64_t bgt_moe_balance_workspace_bytes(int64_t T, int64_t E) {
  const int st = check_balance(T, E, 1);
  return st != BGT_OK ? st : bgt::moe_balance_ws_bytes(T, E);
}

int bgt_moe_balance(const void* logits, int type, int64_t ld, const int32_t* ids, int64_t T,
                    int64_t E, int64_t k, float* loss, int32_t* counts, float* probs,
                    int32_t* tokens, void* ws, int64_t ws_bytes, void* stream) {
  if (!logits || !ids || !loss || !counts || !probs || !tokens || !ws) return BGT_ERR_NULL;
  if (!valid_type(type)) return BGT_ERR_MODE;
  const int st = check_balance(T, E, k);
  if (st != BGT_OK) return st;
  if (ld < E || ws_bytes < bgt::moe_balance_ws_bytes(T, E)) return BGT_ERR_SHAPE;
  if (!aligned(logits, type_bytes(type)) || !aligned(ids, 4) || !aligned(loss, 4) ||
      !aligned(counts, 4) || !aligned(probs, 4) || !aligned(tokens, 4) || !aligned(ws, 4))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_moe_balance(logits, type, ld, ids, T, E, k, loss, counts, probs,
                                            tokens, ws, stream_of(stream)));
}

int bgt_moe_balance_backward(const float* dloss, const void* logits, int type, int64_t ld,
                             const int32_t* counts, const int32_t* tokens, int64_t T, int64_t E,
                             void* dlogits, void* stream) {
  if (!dloss || !logits || !counts || !tokens || !dlogits) return BGT_ERR_NULL;
  if (!valid_type(type)) return BGT_ERR_MODE;
  const int st = check_balance(T, E, 1);
  if (st != BGT_OK) return st;
  if (ld < E) return BGT_ERR_SHAPE;
  if (!aligned(logits, type_bytes(type)) || !aligned(dlogits, type_bytes(type)) ||
      !aligned(dloss, 4) || !aligned(counts, 4) || !aligned(tokens, 4))
    return BGT_ERR_ALIGN;
  return hip_status(bgt::launch_moe_balance_backward(dloss, logits, type, ld, counts, tokens, T, E,
                                                     dlogits, stream_of(stream)));
}

}  // extern "C"
