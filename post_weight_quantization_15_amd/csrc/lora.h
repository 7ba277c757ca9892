// Shared by the adapter products: small device helpers and the pieces that
// the orchestration in k_lora.hip puts together.
#pragma once

#include "common.h"
#include "lora_sizes.h"

namespace gptq {

inline unsigned ceil_div(int64_t a, int64_t b) { return static_cast<unsigned>((a + b - 1) / b); }
inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

// A launch holds fewer than 2^32 threads in one dimension (more are cut off
// without an error), and some launches here have a workgroup for every part
// of every adapter: those go into two dimensions, and the kernel reads the
// index off both (flat_block; the last row may run past the end).
inline dim3 flat_grid(int64_t blocks) {
  const int64_t y = (blocks + (int64_t(1) << 23) - 1) >> 23;
  return dim3(ceil_div(blocks, y), unsigned(y));
}

// ---------------------------------------------------------------------------
// The products Y[t][j] = sum_k V[t][k] M[j][k] (+ the adapters' part) of
// lora_gemm.hip.  Both operands are bf16 with k contiguous, rows 16-byte
// aligned, k in blocks of 64.
struct GemmArgs {
  const uint16_t* V;       // activations [n][ldv]
  int64_t ldv, n;
  const uint16_t* V2;      // the same in group order, when the plan asks for it
  int64_t ldv2;
  const uint16_t* M;       // [m][ldm]
  int64_t ldm, m;
  int kblocks, kwrap;      // blocks of 64 of M; V repeats after kwrap blocks
  // groups: per unit of columns the group whose step Delta multiplies its sums
  const int32_t* plan;     // header {in order, kblocks}, then the group per unit
  const float* scale_t;    // [ng][mpad] steps (without a plan: [mpad], or NULL)
  int64_t mpad;
  // the adapters' part: parts [n][3 rp] (three bf16 parts of alpha H), L_a [m][rank] rows
  const uint16_t* parts;
  const uint16_t* L;       // [n_adapters][m][rank], or NULL
  const int32_t* row;
  int n_adapters, rank, rp;
  void* Y;
  int64_t ldy;
  int out_bf16;
};
constexpr int kPlanHeader = 16;   // words before the plan's group list

// Columns in group order, every group padded to whole units (64
// columns where they divide the group size, else 32), and all to whole blocks.
int fold_unit(int64_t group);
int64_t plan_cols(int64_t d, int64_t ng, int64_t group);
size_t plan_words(int64_t d, int64_t ng, int64_t group);
gptq_status launch_plan(const Packed& w, int32_t* plan, hipStream_t st);
// M[j][k] = code - zero, exact in bf16, in the plan's column order; scale_t =
// steps transposed; V2[t][k] = V[t][order[k]] where the plan is not the natural
// order (or always).  M NULL: the activations alone.
gptq_status launch_layout(const Packed& w, const int32_t* plan, uint16_t* M, int64_t ldm,
                          float* scale_t, int64_t mpad, const uint16_t* V, int64_t ldv, int64_t n,
                          int always, uint16_t* V2, int64_t ldv2, hipStream_t st);
// The same for the whole-row grid, in the columns' own order.
gptq_status launch_expand_row(const Packed& w, uint16_t* M, int64_t ldm, float* scale,
                              hipStream_t st);
// M[j][p ldp + c] = part p of three of W_hat[j][c] in bf16 (their sum is exact in fp32).
gptq_status launch_expand_parts(const Packed& w, uint16_t* M, int64_t ldp, hipStream_t st);
// What the backward pass lays out (NULL: not asked for).
struct PrepareArgs {
  Packed w;
  int64_t mp;          // m padded to 64
  uint16_t* Wt;        // [d][mp] W_hat^T rounded to bf16, zeros past m
  gptq_adapters ad;
  int rp;
  uint16_t* Bt;        // [n_adapters][rank][mp]
  uint16_t* At;        // [n_adapters][d][rank]
  const float* H;
  int64_t n;
  uint16_t* hparts;    // [n][3 rp] parts of alpha H
};
gptq_status launch_prepare(const PrepareArgs& a, hipStream_t st);
// V2[t][0 .. cols) = V[t][0 .. len) and zeros.
gptq_status launch_pad_rows(const uint16_t* V, int64_t ldv, int64_t n, int64_t len, uint16_t* V2,
                            int64_t cols, hipStream_t st);
// fold: the unit of columns whose sums one step multiplies; 0: none.
gptq_status launch_gemm(const GemmArgs& a, int fold, hipStream_t st);

// Few rows (lora_decode.hip): no workspace but H [n][rank].  4096 columns into 4096
// / 11008 into 4096 in 4 bits: 128 rows 34 / 68 us against 50 / 100 by laid-out
// tiles (act-order 53 / 112 and 58 / 117), 160 rows 52 / 115 and 49 / 102.
constexpr int64_t kDecodeMaxRows = 128;
bool decode_takes(int64_t n, int64_t ng);
gptq_status launch_lora_decode(const uint16_t* X, int64_t ldx, int64_t n, const Packed& w,
                               const gptq_adapters& ad, float* H, void* Y, int out_bf16,
                               int64_t ldy, hipStream_t st);

#ifdef __HIPCC__
namespace {

__device__ inline unsigned flat_block() { return blockIdx.y * gridDim.x + blockIdx.x; }

typedef const void __attribute__((address_space(1)))* gvoid;
typedef void __attribute__((address_space(3)))* lvoid;

__device__ inline float bf16_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ inline uint16_t f32_bf16(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// The three bf16 parts of an fp32 number: each the rounding of what the
// parts before leave, so that (normal range) their sum is the number itself:
// 8 + 8 + 8 significant bits.  inf and NaN go into the first part alone.
__device__ inline void split3(float v, uint16_t p[3]) {
  p[0] = f32_bf16(v);
  const float a = bf16_f32(p[0]);
  const float r1 = (__float_as_uint(a) & 0x7F800000u) == 0x7F800000u ? 0.0f : v - a;
  p[1] = f32_bf16(r1);
  const float r2 = r1 - bf16_f32(p[1]);
  p[2] = f32_bf16(r2);
}

__device__ inline f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight values [c, c + 8) of a row of len bf16 values, zeros past its end; vec: the row's
// 16-byte loads are aligned.
__device__ inline u32x4 load8(const uint16_t* __restrict__ p, int64_t c, int64_t len, bool vec) {
  if (vec && c + 8 <= len) return *reinterpret_cast<const u32x4*>(p + c);
  u32x4 v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < len) v[i >> 1] |= uint32_t(p[c + i]) << (16 * (i & 1));
  return v;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ inline float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a),
                                         __builtin_bit_cast(bf16x2, b), c, false);
}
__device__ inline float dot8(const u32x4& a, const u32x4& b, float c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = dot2(a[i], b[i], c);
  return c;
}

// Dot product of two rows by a wave, the sum in every lane; vec: 16-byte aligned.
__device__ inline float dot_wave(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w,
                                 int64_t len, bool vec, int lane) {
  float s = 0.0f;
  int64_t b = 0;
  if (vec) {                               // whole 512-column rounds, loads back to back
#pragma unroll 8
    for (; b + 512 <= len; b += 512)
      s = dot8(*reinterpret_cast<const u32x4*>(x + b + 8 * lane),
               *reinterpret_cast<const u32x4*>(w + b + 8 * lane), s);
  }
  for (int64_t c = b + 8 * lane; c < len; c += 512)
    s = dot8(load8(x, c, len, vec), load8(w, c, len, vec), s);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  return s;
}

// Group of column c, always one of the row's: an id outside counts as the nearest.
__device__ inline int group_at(const Packed& w, int64_t c) {
  return min(max(w.g_idx[c], 0), static_cast<int>(w.ng) - 1);
}
// Step Delta and code minus zero of weight (r, c).
__device__ inline float step_at(const Packed& w, int64_t i) {
  return w.scale_f16 ? static_cast<float>(static_cast<const _Float16*>(w.scales)[i])
                     : static_cast<const float*>(w.scales)[i];
}
__device__ inline int code_at(const Packed& w, int64_t words, int64_t r, int64_t c) {
  const int64_t p = c * w.bits;
  const int64_t i = p >> 5;
  const int off = static_cast<int>(p & 31);
  uint32_t v = w.qw[r * words + i] >> off;
  if (off + w.bits > 32) v |= w.qw[r * words + i + 1] << (32 - off);
  v &= (1u << w.bits) - 1u;
  const int hb = 1 << (w.bits - 1);
  return w.sgn ? static_cast<int>(v ^ hb) - hb : static_cast<int>(v);
}

template <int n>
__device__ inline void wait_vmcnt() {
  // vmcnt = n (split field), expcnt and lgkmcnt at maximum
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

}  // namespace
#endif

}  // namespace gptq
