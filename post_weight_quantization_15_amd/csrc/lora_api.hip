// Host side of the adapter products, the transposed dequantizing product and
// the distillation loss: argument validation and workspace checks.
#include "common.h"

using namespace gptq;

namespace {

constexpr int64_t kMaxDim = 65535;

bool valid_bits(int32_t b) { return b == 2 || b == 3 || b == 4 || b == 8; }

// The sizes and types every product on the packed format checks; pointers
// are needed only where there are rows.
bool valid_packed(int64_t n, int64_t m, int64_t d, const uint32_t* qw, const void* scales,
                  gptq_dtype sdt, const uint8_t* zeros, const int32_t* g_idx, int32_t bits,
                  int32_t group, int32_t sgn) {
  if (n < 0 || n > kMaxRows || m <= 0 || d <= 0 || m > kMaxDim || d > kMaxDim ||
      (sdt != GPTQ_F32 && sdt != GPTQ_F16) || !valid_bits(bits) ||
      !(group == -1 || group > 0) || (sgn != 0 && sgn != 1))
    return false;
  return n == 0 || (qw && scales && zeros && g_idx);
}

Packed make_packed(int64_t m, int64_t d, const uint32_t* qw, const void* scales, gptq_dtype sdt,
                   const uint8_t* zeros, const int32_t* g_idx, int32_t bits, int32_t group,
                   int32_t sgn) {
  return Packed{qw, scales, zeros, g_idx, m, d, group > 0 ? (d + group - 1) / group : 1,
                bits, group, sdt == GPTQ_F16, sgn};
}

bool valid_adapters(const gptq_adapters* a) {
  return a && a->n_adapters >= 1 && a->n_adapters <= kMaxDim && a->rank >= 1 &&
         a->rank <= kMaxRank;
}

// Too small, missing, or not aligned as its parts' 16-byte accesses need.
bool bad_ws(const void* ws, size_t have, size_t need) {
  return have < need || (need > 0 && (!ws || reinterpret_cast<uintptr_t>(ws) % 16));
}

}  // namespace

extern "C" {

size_t gptq_dequant_matmul_t_workspace_bytes(int64_t n, int64_t m, int64_t d) {
  if (n < 0 || n > kMaxRows || m <= 0 || d <= 0 || m > kMaxDim || d > kMaxDim) return 0;
  return lora_backward_ws_bytes(n, m, d, 0, 0);
}

gptq_status gptq_dequant_matmul_t(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                                  int64_t lddy, const uint32_t* qweight, const void* scales,
                                  gptq_dtype scale_dtype, const uint8_t* zeros,
                                  const int32_t* g_idx, int64_t d, int32_t bits,
                                  int32_t group_size, int32_t signed_codes, void* dX,
                                  int64_t lddx, void* ws, size_t ws_bytes, void* stream) {
  if (dy_dtype != GPTQ_BF16 ||
      !valid_packed(n, m, d, qweight, scales, scale_dtype, zeros, g_idx, bits, group_size,
                    signed_codes) ||
      lddy < m || lddx < d || (n > 0 && (!dY || !dX)))
    return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes, lora_backward_ws_bytes(n, m, d, 0, 0))) return GPTQ_ERR_WORKSPACE;
  const Packed w = make_packed(m, d, qweight, scales, scale_dtype, zeros, g_idx, bits, group_size,
                               signed_codes);
  return launch_lora_backward(static_cast<const uint16_t*>(dY), lddy, n, nullptr, 0, nullptr, w,
                              nullptr, static_cast<uint16_t*>(dX), lddx, nullptr, nullptr, 0, ws,
                              static_cast<hipStream_t>(stream));
}

size_t gptq_lora_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t group_size,
                                 int32_t rank) {
  if (n < 0 || n > kMaxRows || m <= 0 || d <= 0 || m > kMaxDim || d > kMaxDim || rank < 1 ||
      rank > kMaxRank || !(group_size == -1 || group_size > 0))
    return 0;
  return lora_ws_bytes(n, m, d, group_size, rank);
}

gptq_status gptq_lora_matmul(const void* X, gptq_dtype x_dtype, int64_t n, int64_t d, int64_t ldx,
                             const uint32_t* qweight, const void* scales, gptq_dtype scale_dtype,
                             const uint8_t* zeros, const int32_t* g_idx, int64_t m, int32_t bits,
                             int32_t group_size, int32_t signed_codes,
                             const gptq_adapters* adapters, float* H, void* Y, gptq_dtype y_dtype,
                             int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  if (x_dtype != GPTQ_BF16 || (y_dtype != GPTQ_F32 && y_dtype != GPTQ_BF16) ||
      !valid_packed(n, m, d, qweight, scales, scale_dtype, zeros, g_idx, bits, group_size,
                    signed_codes) ||
      !valid_adapters(adapters) || ldx < d || ldy < m)
    return GPTQ_ERR_INVALID_ARG;
  if (n > 0 && (!X || !Y || !adapters->A || !adapters->B || !adapters->alpha || !adapters->row))
    return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes, lora_ws_bytes(n, m, d, group_size, adapters->rank)))
    return GPTQ_ERR_WORKSPACE;
  if (n == 0) return GPTQ_OK;
  const Packed w = make_packed(m, d, qweight, scales, scale_dtype, zeros, g_idx, bits, group_size,
                               signed_codes);
  return launch_lora(static_cast<const uint16_t*>(X), ldx, n, w, *adapters, H, Y,
                     y_dtype == GPTQ_BF16, ldy, ws, static_cast<hipStream_t>(stream));
}

size_t gptq_lora_backward_workspace_bytes(int64_t n, int64_t m, int64_t d, int32_t rank,
                                          int32_t n_adapters) {
  if (n < 0 || n > kMaxRows || m <= 0 || d <= 0 || m > kMaxDim || d > kMaxDim || rank < 1 ||
      rank > kMaxRank || n_adapters < 1 || n_adapters > kMaxDim)
    return 0;
  return lora_backward_ws_bytes(n, m, d, rank, n_adapters);
}

gptq_status gptq_lora_backward(const void* dY, gptq_dtype dy_dtype, int64_t n, int64_t m,
                               int64_t lddy, const void* X, int64_t ldx, const float* H,
                               const uint32_t* qweight, const void* scales,
                               gptq_dtype scale_dtype, const uint8_t* zeros, const int32_t* g_idx,
                               int64_t d, int32_t bits, int32_t group_size, int32_t signed_codes,
                               const gptq_adapters* adapters, void* dX, int64_t lddx, float* dA,
                               float* dB, int32_t accumulate, void* ws, size_t ws_bytes,
                               void* stream) {
  if (dy_dtype != GPTQ_BF16 || n < 0 || n > kMaxRows || m <= 0 || d <= 0 || m > kMaxDim ||
      d > kMaxDim || !valid_adapters(adapters) || lddy < m || (dA && ldx < d) ||
      (dX && lddx < d) || (accumulate != 0 && accumulate != 1))
    return GPTQ_ERR_INVALID_ARG;
  // the packed weights are read for dX alone
  if (!valid_packed(dX ? n : 0, m, d, qweight, scales, scale_dtype, zeros, g_idx, bits,
                    group_size, signed_codes))
    return GPTQ_ERR_INVALID_ARG;
  if (n > 0 && (!dY || !adapters->alpha || !adapters->row || ((dX || dA) && !adapters->B) ||
                (dX && !adapters->A) || (dA && !X) || (dB && !H)))
    return GPTQ_ERR_INVALID_ARG;
  if (bad_ws(ws, ws_bytes,
               lora_backward_ws_bytes(n, m, d, adapters->rank, adapters->n_adapters)))
    return GPTQ_ERR_WORKSPACE;
  const Packed w = make_packed(m, d, qweight, scales, scale_dtype, zeros, g_idx, bits, group_size,
                               signed_codes);
  return launch_lora_backward(static_cast<const uint16_t*>(dY), lddy, n,
                              static_cast<const uint16_t*>(X), ldx, H, w, adapters,
                              static_cast<uint16_t*>(dX), lddx, dA, dB, accumulate, ws,
                              static_cast<hipStream_t>(stream));
}

static bool valid_distill(const void* logits, gptq_dtype dt, int64_t n, int64_t vocab,
                          int64_t ldl, const int32_t* t_idx, const float* t_logits, int64_t k,
                          float temp) {
  if ((dt != GPTQ_BF16 && dt != GPTQ_F16 && dt != GPTQ_F32) || n < 0 || n > (int64_t(1) << 21) ||
      vocab < 1 || vocab > kDistillMaxVocab || ldl < vocab || k < 1 || k > kDistillMaxK ||
      !(temp >= kDistillMinTemp && temp <= 1.0f / kDistillMinTemp))
    return false;
  return n == 0 || (logits && t_idx && t_logits);
}

gptq_status gptq_distill_loss(const void* logits, gptq_dtype dtype, int64_t n, int64_t vocab,
                              int64_t ldl, const int32_t* t_idx, const float* t_logits, int64_t k,
                              float temperature, const float* t_lse, const float* weight,
                              float* loss, float* stats, void* dlogits, int64_t ldd,
                              void* stream) {
  if (!valid_distill(logits, dtype, n, vocab, ldl, t_idx, t_logits, k, temperature) ||
      (n > 0 && !loss) || (dlogits && ldd < vocab) ||
      (dlogits && dlogits == logits && ldd != ldl))
    return GPTQ_ERR_INVALID_ARG;
  return launch_distill(logits, dtype, n, vocab, ldl, t_idx, t_logits, k, temperature, t_lse,
                        weight, nullptr, loss, stats, dlogits, ldd,
                        static_cast<hipStream_t>(stream));
}

gptq_status gptq_distill_backward(const void* logits, gptq_dtype dtype, int64_t n, int64_t vocab,
                                  int64_t ldl, const float* stats, const int32_t* t_idx,
                                  const float* t_logits, int64_t k, float temperature,
                                  const float* t_lse, const float* weight, const float* grad,
                                  void* dlogits, int64_t ldd, void* stream) {
  if (!valid_distill(logits, dtype, n, vocab, ldl, t_idx, t_logits, k, temperature) ||
      (n > 0 && (!stats || !grad || !dlogits)) || ldd < vocab ||
      (n > 0 && dlogits == logits && ldd != ldl))
    return GPTQ_ERR_INVALID_ARG;
  return launch_distill(logits, dtype, n, vocab, ldl, t_idx, t_logits, k, temperature, t_lse,
                        weight, grad, nullptr, const_cast<float*>(stats), dlogits, ldd,
                        static_cast<hipStream_t>(stream));
}

}  // extern "C"
