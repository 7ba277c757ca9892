// Shared by the operators on 4-bit floating-point layers (MXFP4): the stored
// format on the device and the pieces that the entry points put together.
#pragma once

#include "lora.h"

namespace gptq {

constexpr int kMxBlock = 32;                 // values that share a power of two

inline int64_t mx_blocks(int64_t d) { return (d + kMxBlock - 1) / kMxBlock; }

// A matrix [rows, 32 nb] of 4-bit values: 16 bytes a block (lower half of a
// byte first), rows of nb blocks without gaps, and a scale byte a block.
struct Mx {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, nb;
};

// The activations of a product: bf16 as they are, bf16 that the call rounds to
// 4 bits, or 4-bit values (gptq_mx_input).
struct MxInput {
  int form;
  const void* X;                             // bf16 [n][ldx], or codes
  int64_t ldx;
  const uint8_t* scales;                     // of the codes
  int64_t n, d;
};

// Y = X W^T (up.codes NULL), or bf16 Y = act(X W^T) * (X up^T) with, where G
// is given, both factors in bf16 (rows of ldg).
struct MxOutput {
  void* Y;
  int64_t ldy;
  int out_bf16;
  int act;
  uint16_t* G;
  uint16_t* U;
  int64_t ldg;
};

gptq_status launch_mx_quantize(const void* X, gptq_dtype dt, int64_t n, int64_t d, int64_t ldx,
                               uint8_t* codes, uint8_t* scales, void* hat, int64_t ldh,
                               hipStream_t st);
size_t mx_matmul_ws_bytes(int64_t n, int64_t m, int64_t d, int form, bool gated);
gptq_status launch_mx_matmul(const MxInput& x, const Mx& w, const Mx& up, const MxOutput& y,
                             void* ws, hipStream_t st);
size_t mx_matmul_t_ws_bytes(int64_t n, int64_t m, int64_t d, bool gated);
gptq_status launch_mx_matmul_t(const uint16_t* dY, int64_t lddy, int64_t n, const Mx& w, int64_t d,
                               uint16_t* dX, int64_t lddx, void* ws, hipStream_t st);
// dGU [n][2 mp], mp = m padded to 64: the gradients of both factors.
gptq_status launch_mx_gated_backward(const uint16_t* dY, int64_t lddy, int64_t n,
                                     const uint16_t* G, const uint16_t* U, int64_t ldg,
                                     const Mx& gate, const Mx& up, int64_t d, int act,
                                     uint16_t* dX, int64_t lddx, uint16_t* dGU, void* ws,
                                     hipStream_t st);

// Few rows (mx_decode.hip): no workspace.  Up to 16 rows, and up to 64 where it takes less time
// than tiles.
bool mx_decode_takes(int64_t n, int64_t m, int64_t d, int form, bool gated);
gptq_status launch_mx_decode(const MxInput& x, const Mx& w, const Mx& up, const MxOutput& y,
                             hipStream_t st);

// Many rows (mx_gemm.hip).
size_t mx_gemm_ws_bytes(int64_t n, int64_t m, int64_t d, int form, bool gated);
double mx_gemm_time(int64_t n, int64_t m, int64_t d, int form, bool gated);   // us, estimated
gptq_status launch_mx_gemm(const MxInput& x, const Mx& w, const Mx& up, const MxOutput& y, void* ws,
                           hipStream_t st);

size_t mx_dense_floats(int64_t n, int64_t m, int64_t k);
gptq_status launch_mx_dense(const uint16_t* V, int64_t ldv, int64_t n, const uint16_t* M,
                            int64_t ldm, int64_t m, int64_t k, const MxOutput& y, float* part,
                            hipStream_t st);

#ifdef __HIPCC__
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Scale byte of a block whose largest magnitude has these fp32 bits: the
// largest value's power of two comes to lie at 4 = 2^2, the format's last.  255 (NaN)
// where the block holds a value that is not finite.
__device__ inline uint32_t mx_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}
// A scale byte as the fp32 number whose exponent field the conversions read.
__device__ inline float mx_scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight 4-bit values of a word times their scale, as bf16: exact (up to
// 2^127, inf beyond), NaN for a scale byte of 255.
__device__ inline u32x4 mx_expand8(uint32_t word, float scale) {
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3));
  return v;
}

// A pair of 16-bit values, by value: a bit cast of a vector's element itself
// reads its first one with this compiler.
__device__ inline bf16x2 mx_pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// Eight bf16 values to 4 bits: to nearest even, saturating at 6 times the scale.
__device__ inline uint32_t mx_round8(const u32x4& v, float scale) {
  uint32_t w = 0u;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, mx_pair(v[0]), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, mx_pair(v[1]), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, mx_pair(v[2]), scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, mx_pair(v[3]), scale, 3);
  return w;
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The larger magnitudes of two pairs of bf16 (as integers they order alike).
__device__ inline uint32_t mx_amax2(uint32_t m, uint32_t v) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                          __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu)));
}

// acc += A B^T over 128 values of 16 rows each: a lane holds block lane / 16 of
// its operands' row lane % 16, with the block's scale in byte B.
template <int B>
__device__ inline f32x4 mx_mfma(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                const f32x4& c) {
  i32x8 va = {}, vb = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    va[i] = static_cast<int>(a[i]);
    vb[i] = static_cast<int>(b[i]);
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, B, static_cast<int>(sa),
                                                          B, static_cast<int>(sb));
}

// The gate's activation and its slope.  The reciprocal is the hardware's (1 ulp).
__device__ inline float mx_sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}
__device__ inline float mx_act(float g, int act) {
  if (act == GPTQ_ACT_SILU) return g * mx_sigmoid(g);
  if (act == GPTQ_ACT_RELU) return g < 0.0f ? 0.0f : g;      // NaN stays
  return g;
}
__device__ inline float mx_slope(float g, int act) {
  if (act == GPTQ_ACT_SILU) {
    const float s = mx_sigmoid(g);
    return s * fmaf(g, 1.0f - s, 1.0f);
  }
  if (act == GPTQ_ACT_RELU) return g > 0.0f ? 1.0f : g != g ? g : 0.0f;
  return 1.0f;
}

}  // namespace
#endif

}  // namespace gptq
