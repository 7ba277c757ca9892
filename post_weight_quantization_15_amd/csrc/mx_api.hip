// Host side of the operators on 4-bit floating-point layers and of the token
// statistics: argument validation and workspace checks.
#include "mx.h"

using namespace gptq;

namespace {

constexpr int64_t kMaxDim = 65535;

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool valid_sizes(int64_t n, int64_t m, int64_t d) {
  return n >= 0 && n <= kMaxRows && m > 0 && d > 0 && m <= kMaxDim && d <= kMaxDim;
}

bool valid_layer(const uint8_t* codes, const uint8_t* scales) {
  return codes && scales && aligned16(codes);
}

bool valid_form(int32_t f) {
  return f == GPTQ_MX_BF16 || f == GPTQ_MX_ROUND || f == GPTQ_MX_CODES;
}

bool valid_input(const void* X, int32_t form, const uint8_t* x_scales, int64_t d, int64_t ldx) {
  if (form == GPTQ_MX_CODES) return X && x_scales && aligned16(X);
  return X && ldx >= d;
}

bool bad_ws(const void* ws, size_t have, size_t need) {
  return have < need || (need > 0 && (!ws || !aligned16(ws)));
}

bool valid_act(int32_t a) {
  return a == GPTQ_ACT_NONE || a == GPTQ_ACT_RELU || a == GPTQ_ACT_SILU;
}

bool valid_tokens(gptq_dtype dt, int64_t n, int64_t vocab, int64_t ldl, float temp) {
  return (dt == GPTQ_BF16 || dt == GPTQ_F16 || dt == GPTQ_F32) && n >= 0 &&
         n <= (int64_t(1) << 21) && vocab >= 1 && vocab <= kDistillMaxVocab && ldl >= vocab &&
         temp >= kDistillMinTemp && temp <= 1.0f / kDistillMinTemp;
}

}  // namespace

extern "C" {

gptq_status gptq_mx_quantize(const void* X, gptq_dtype dtype, int64_t n, int64_t d, int64_t ldx,
                                uint8_t* codes, uint8_t* scales, void* hat, int64_t ldh,
                                void* stream) {
  if ((dtype != GPTQ_BF16 && dtype != GPTQ_F16 && dtype != GPTQ_F32) || !valid_sizes(n, 1, d) ||
      ldx < d || (hat && ldh < d) || (n > 0 && (!X || !codes || !scales)) || !aligned16(codes))
    return GPTQ_ERR_INVALID_ARG;
  return launch_mx_quantize(X, dtype, n, d, ldx, codes, scales, hat, ldh,
                            static_cast<hipStream_t>(stream));
}

size_t gptq_mx_matmul_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t x_form) {
  if (!valid_sizes(n, m, d) || !valid_form(x_form)) return 0;
  return mx_matmul_ws_bytes(n, m, d, x_form, false);
}

gptq_status gptq_mx_matmul(const void* X, int32_t x_form, const uint8_t* x_scales, int64_t n,
                              int64_t d, int64_t ldx, const uint8_t* codes, const uint8_t* scales,
                              int64_t m, void* Y, gptq_dtype y_dtype, int64_t ldy, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, m, d) || !valid_form(x_form) ||
      (y_dtype != GPTQ_F32 && y_dtype != GPTQ_BF16) || ldy < m)
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_input(X, x_form, x_scales, d, ldx) || !valid_layer(codes, scales) || !Y)
    return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes, mx_matmul_ws_bytes(n, m, d, x_form, false))) return GPTQ_ERR_WORKSPACE;
  const int64_t nb = mx_blocks(d);
  const MxOutput y{Y, ldy, y_dtype == GPTQ_BF16, GPTQ_ACT_NONE, nullptr, nullptr, 0};
  return launch_mx_matmul(MxInput{x_form, X, ldx, x_scales, n, d}, Mx{codes, scales, m, nb}, Mx{},
                          y, ws, static_cast<hipStream_t>(stream));
}

size_t gptq_mx_matmul_t_workspace_bytes(int64_t n, int64_t m, int64_t d) {
  return valid_sizes(n, m, d) ? mx_matmul_t_ws_bytes(n, m, d, false) : 0;
}

gptq_status gptq_mx_matmul_t(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                                int64_t lddy, const uint8_t* codes, const uint8_t* scales,
                                int64_t d, void* dX, int64_t lddx, void* ws, size_t ws_bytes,
                                void* stream) {
  if (dy_dtype != GPTQ_BF16 || !valid_sizes(n, m, d) || lddy < m || lddx < d)
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!dY || !valid_layer(codes, scales) || !dX) return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes, mx_matmul_t_ws_bytes(n, m, d, false))) return GPTQ_ERR_WORKSPACE;
  return launch_mx_matmul_t(static_cast<const uint16_t*>(dY), lddy, n,
                            Mx{codes, scales, m, mx_blocks(d)}, d, static_cast<uint16_t*>(dX), lddx,
                            ws, static_cast<hipStream_t>(stream));
}

size_t gptq_mx_gated_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t x_form) {
  if (!valid_sizes(n, m, d) || !valid_form(x_form)) return 0;
  return mx_matmul_ws_bytes(n, m, d, x_form, true);
}

gptq_status gptq_mx_gated(const void* X, int32_t x_form, const uint8_t* x_scales, int64_t n,
                             int64_t d, int64_t ldx, const uint8_t* gate_codes,
                             const uint8_t* gate_scales, const uint8_t* up_codes,
                             const uint8_t* up_scales, int64_t m, int32_t activation, void* Y,
                             int64_t ldy, void* G, void* U, int64_t ldg, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!valid_sizes(n, m, d) || !valid_form(x_form) || !valid_act(activation) || ldy < m ||
      !G != !U || (G && ldg < m))
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_input(X, x_form, x_scales, d, ldx) || !valid_layer(gate_codes, gate_scales) ||
      !valid_layer(up_codes, up_scales) || !Y)
    return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes, mx_matmul_ws_bytes(n, m, d, x_form, true))) return GPTQ_ERR_WORKSPACE;
  const int64_t nb = mx_blocks(d);
  const MxOutput y{Y, ldy, 1, activation, static_cast<uint16_t*>(G), static_cast<uint16_t*>(U), ldg};
  return launch_mx_matmul(MxInput{x_form, X, ldx, x_scales, n, d},
                          Mx{gate_codes, gate_scales, m, nb}, Mx{up_codes, up_scales, m, nb}, y, ws,
                          static_cast<hipStream_t>(stream));
}

size_t gptq_mx_gated_backward_workspace_bytes(int64_t n, int64_t m, int64_t d) {
  return valid_sizes(n, m, d) ? mx_matmul_t_ws_bytes(n, m, d, true) : 0;
}

gptq_status gptq_mx_gated_backward(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                                      int64_t lddy, const void* G, const void* U, int64_t ldg,
                                      const uint8_t* gate_codes, const uint8_t* gate_scales,
                                      const uint8_t* up_codes, const uint8_t* up_scales, int64_t d,
                                      int32_t activation, void* dX, int64_t lddx, void* dGU,
                                      void* ws, size_t ws_bytes, void* stream) {
  if (dy_dtype != GPTQ_BF16 || !valid_sizes(n, m, d) || !valid_act(activation) || lddy < m ||
      ldg < m || (dX && lddx < d))
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!dY || !G || !U || !dGU || !aligned16(dGU) ||
      (dX && (!valid_layer(gate_codes, gate_scales) || !valid_layer(up_codes, up_scales))))
    return GPTQ_ERR_INVALID_ARG;
  if (dX && bad_ws(ws, ws_bytes, mx_matmul_t_ws_bytes(n, m, d, true))) return GPTQ_ERR_WORKSPACE;
  const int64_t nb = mx_blocks(d);
  return launch_mx_gated_backward(
      static_cast<const uint16_t*>(dY), lddy, n, static_cast<const uint16_t*>(G),
      static_cast<const uint16_t*>(U), ldg, Mx{gate_codes, gate_scales, m, nb},
      Mx{up_codes, up_scales, m, nb}, d, activation, static_cast<uint16_t*>(dX), lddx,
      static_cast<uint16_t*>(dGU), ws, static_cast<hipStream_t>(stream));
}

size_t gptq_token_logprobs_workspace_bytes(int64_t n, int64_t vocab, int64_t k) {
  if (!valid_tokens(GPTQ_F32, n, vocab, vocab, 1.0f) || k < 0 || k > kTokensMaxK || k > vocab)
    return 0;
  return tokens_ws_bytes(n, vocab, k);
}

gptq_status gptq_token_logprobs(const void* logits, gptq_dtype dtype, int64_t n, int64_t vocab,
                                int64_t ldl, const int32_t* tokens, float temperature, int64_t k,
                                float* logp, float* entropy, float* lse, float* stats,
                                float* top_logits, int32_t* top_idx, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!valid_tokens(dtype, n, vocab, ldl, temperature) || k < 0 || k > kTokensMaxK || k > vocab)
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!logits || (logp && !tokens) || (k > 0 && (!top_logits || !top_idx)))
    return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes, tokens_ws_bytes(n, vocab, k))) return GPTQ_ERR_WORKSPACE;
  return launch_tokens(logits, dtype, n, vocab, ldl, tokens, temperature, k, logp, entropy, lse,
                       stats, top_logits, top_idx, ws, static_cast<hipStream_t>(stream));
}

gptq_status gptq_token_logprobs_backward(const void* logits, gptq_dtype dtype, int64_t n,
                                         int64_t vocab, int64_t ldl, const float* stats,
                                         const int32_t* tokens, float temperature,
                                         const float* grad_logp, const float* grad_entropy,
                                         void* dlogits, int64_t ldd, void* stream) {
  if (!valid_tokens(dtype, n, vocab, ldl, temperature) || ldd < vocab ||
      (n > 0 && dlogits == logits && ldd != ldl))
    return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!logits || !stats || !dlogits || (grad_logp && !tokens)) return GPTQ_ERR_INVALID_ARG;
  return launch_tokens_grad(logits, dtype, n, vocab, ldl, stats, tokens, temperature, grad_logp,
                            grad_entropy, dlogits, ldd, static_cast<hipStream_t>(stream));
}

}  // extern "C"
