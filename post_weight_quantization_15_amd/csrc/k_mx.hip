// Layers and activations in 4-bit floating point (e2m1: 0, 1/2, 1, 3/2, 2, 3,
// 4, 6 and their negatives) in blocks of 32 with a power of two each: rounding
// to it, and the products that read it.
#include <algorithm>

#include "mx.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------
// Rounding.  A thread takes eight values of a row, four threads a block; the
// block's largest magnitude goes round by two exchanges.  A wave takes runs of
// 512 values.  All of it exact but the rounding itself, which the hardware's
// conversion does (nearest even, saturating).  One reading and one writing: bound by
// bytes (11008 x 4096 with the rounded values too: fp32 70 us, 5.5 TB/s, bf16 33 us, 6.2 TB/s, as part
// of it stays in the last cache; small ones by the launch).
// ---------------------------------------------------------------------------
struct QuantizeArgs {
  const void* X;
  int64_t ldx;
  uint32_t n, runs;       // rows, runs of 512 values a row
  int64_t d, nb;
  uint8_t* codes;
  uint8_t* scales;
  void* hat;
  int64_t ldh;
  bool vec, vec_h;
};

template <int DT>
struct Eight {                               // eight values as stored
  u32x4 v[DT == GPTQ_F32 ? 2 : 1];
};

template <int DT>
__device__ inline Eight<DT> load_eight(const void* X, int64_t at, int64_t c, int64_t d, bool vec) {
  Eight<DT> e;
  if (DT == GPTQ_F32) {
    const float* p = static_cast<const float*>(X) + at;
    if (vec && c + 8 <= d) {
      e.v[0] = *reinterpret_cast<const u32x4*>(p + c);
      e.v[DT == GPTQ_F32] = *reinterpret_cast<const u32x4*>(p + c + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        e.v[DT == GPTQ_F32 ? i >> 2 : 0][i & 3] = c + i < d ? __float_as_uint(p[c + i]) : 0u;
    }
  } else {
    e.v[0] = load8(static_cast<const uint16_t*>(X) + at, c, d, vec);
  }
  return e;
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(QuantizeArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const uint32_t row = wave / a.runs, run = wave % a.runs;
  if (row >= a.n) return;
  const int64_t c = int64_t(run) * 512 + 8 * lane;
  if (c >= a.nb * kMxBlock) return;          // whole blocks leave: four lanes each
  const Eight<DT> e = load_eight<DT>(a.X, int64_t(row) * a.ldx, c, a.d, a.vec);
  uint32_t m = 0u;                           // largest magnitude as fp32 bits
  if (DT == GPTQ_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m = max(m, e.v[DT == GPTQ_F32 ? i >> 2 : 0][i & 3] & 0x7FFFFFFFu);
  } else {
    uint32_t p = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) p = mx_amax2(p, e.v[0][i]);
    p = max(p & 0xFFFFu, p >> 16);
    m = DT == GPTQ_BF16
            ? p << 16
            : p >= 0x7C00u ? 0x7F800000u
                           : __float_as_uint(static_cast<float>(
                                 __builtin_bit_cast(_Float16, static_cast<uint16_t>(p))));
  }
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2)));
  const uint32_t byte = mx_scale_byte(m);
  const float scale = mx_scale_f32(byte);
  uint32_t word = 0u;
  if (byte != 255u) {
    if (DT == GPTQ_F32) {
      auto f = [&](int i) { return __uint_as_float(e.v[DT == GPTQ_F32 ? i >> 2 : 0][i & 3]); };
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f(0), f(1), scale, 0);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f(2), f(3), scale, 1);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f(4), f(5), scale, 2);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f(6), f(7), scale, 3);
    } else if (DT == GPTQ_F16) {
      auto f = [&](int i) {
        const uint32_t w = e.v[0][i];        // by value: see mx_pair
        return __builtin_bit_cast(f16x2, w);
      };
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, f(0), scale, 0);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, f(1), scale, 1);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, f(2), scale, 2);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(word, f(3), scale, 3);
    } else {
      word = mx_round8(e.v[0], scale);
    }
  }
  const int64_t block = int64_t(row) * a.nb + c / kMxBlock;
  reinterpret_cast<uint32_t*>(a.codes)[4 * block + (lane & 3)] = word;
  if ((lane & 3) == 0) a.scales[block] = static_cast<uint8_t>(byte);
  if (!a.hat) return;
  const int64_t left = a.d - c;
  const int64_t at = int64_t(row) * a.ldh + c;
  if (DT == GPTQ_F32) {
    u32x4 h[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      f32x2 v;
      if (i == 0) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, scale, 0);
      else if (i == 1) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, scale, 1);
      else if (i == 2) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, scale, 2);
      else v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, scale, 3);
      h[i >> 1][2 * (i & 1)] = __float_as_uint(v[0]);
      h[i >> 1][2 * (i & 1) + 1] = __float_as_uint(v[1]);
    }
    float* p = static_cast<float*>(a.hat) + at;
    if (a.vec_h && left >= 8) {
      *reinterpret_cast<u32x4*>(p) = h[0];
      *reinterpret_cast<u32x4*>(p + 4) = h[1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = __uint_as_float(h[i >> 2][i & 3]);
    }
  } else {
    u32x4 h;
    if (DT == GPTQ_BF16) {
      h = mx_expand8(word, scale);
    } else {
      h[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, scale, 0));
      h[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, scale, 1));
      h[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, scale, 2));
      h[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(word, scale, 3));
    }
    uint16_t* p = static_cast<uint16_t*>(a.hat) + at;
    if (a.vec_h && left >= 8) {
      *reinterpret_cast<u32x4*>(p) = h;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// Layout in bf16 (exact) for the gradient's product
// ---------------------------------------------------------------------------

// Wt[c][j0 + j] = W[j][c] for 64 rows x 256 columns a workgroup, zeros for
// rows past the matrix.  A thread takes the same block of two neighbouring
// rows and writes pairs to the turned tile in LDS, 32 lanes to 32 consecutive words of a
// column; a wave's second block takes the other column of two first, whose words lie in other
// banks.  Bound by the writing: 4096 x 11008 values in 28 us (4 TB/s with the codes), a gated
// pair of them in 49; a product of 4096 rows behind it takes ten times that.
__global__ __launch_bounds__(256) void mx_turn_kernel(Mx w, Mx up, unsigned by_one, int64_t d,
                                                      uint16_t* __restrict__ Wt, int64_t ldt) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[256][36];
  const int tid = threadIdx.x, pair = tid & 31, run = tid >> 5;
  const bool second = blockIdx.y >= by_one;
  const Mx& src = second ? up : w;
  const int64_t c0 = int64_t(blockIdx.x) * 256, j0 = int64_t(blockIdx.y - (second ? by_one : 0)) * 64;
  const int64_t b = c0 / kMxBlock + run;
  u32x4 code[2];
  float scale[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t j = j0 + 2 * pair + h;
    code[h] = u32x4{0u, 0u, 0u, 0u};
    scale[h] = 1.0f;
    if (j < src.rows && b < src.nb) {
      code[h] = *reinterpret_cast<const u32x4*>(src.codes + (j * src.nb + b) * 16);
      scale[h] = mx_scale_f32(src.scales[j * src.nb + b]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const u32x4 lo = mx_expand8(code[0][e], scale[0]), hi = mx_expand8(code[1][e], scale[1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t even = (lo[i] & 0xFFFFu) | (hi[i] << 16);
      const uint32_t uneven = (lo[i] >> 16) | (hi[i] & 0xFFFF0000u);
      const int c = 32 * run + 8 * e + 2 * i, odd = run & 1;
      tile[c + odd][pair] = odd ? uneven : even;
      tile[c + 1 - odd][pair] = odd ? even : uneven;
    }
  }
  __syncthreads();
  const int64_t at = int64_t(blockIdx.y) * 64;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int cl = run + 8 * (4 * e + (pair >> 3)), u = pair & 7;
    if (c0 + cl < d)
      *reinterpret_cast<u32x4*>(Wt + (c0 + cl) * ldt + at + 8 * u) =
          *reinterpret_cast<const u32x4*>(&tile[cl][4 * u]);
  }
}

// ---------------------------------------------------------------------------
// The gated block's elementwise gradient
// ---------------------------------------------------------------------------
// dGU[t][j] = dY U act'(G), dGU[t][mp + j] = dY act(G); zeros in the padding.  Computed in fp32
// and rounded to bf16 once, for the next product as for the layers' weight gradients, so that
// both see the same factors.  dX is off by 0.0023 of itself for that (mean square), 0.0017 of which
// is its own rounding; two bf16 parts of each factor would leave that alone at twice the product's
// operations.  Bound by bytes.
__global__ __launch_bounds__(256) void mx_gate_grad_kernel(const uint16_t* __restrict__ dY,
                                                           int64_t lddy,
                                                           const uint16_t* __restrict__ G,
                                                           const uint16_t* __restrict__ U,
                                                           int64_t ldg, int64_t n, int64_t m,
                                                           int act, uint32_t per,
                                                           uint16_t* __restrict__ dGU, bool vec) {
  const uint64_t e = uint64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = static_cast<int64_t>(e / per);
  const int64_t c = 8 * static_cast<int64_t>(e % per);
  if (t >= n) return;
  const u32x4 vy = load8(dY + t * lddy, c, m, vec), vg = load8(G + t * ldg, c, m, vec),
              vu = load8(U + t * ldg, c, m, vec);
  u32x4 og = u32x4{0u, 0u, 0u, 0u}, ou = og;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int s = 16 * (i & 1);
    const float y = bf16_f32((vy[i >> 1] >> s) & 0xFFFFu), g = bf16_f32((vg[i >> 1] >> s) & 0xFFFFu),
                u = bf16_f32((vu[i >> 1] >> s) & 0xFFFFu);
    if (c + i >= m) continue;
    og[i >> 1] |= uint32_t(f32_bf16(y * u * mx_slope(g, act))) << s;
    ou[i >> 1] |= uint32_t(f32_bf16(y * mx_act(g, act))) << s;
  }
  uint16_t* row = dGU + t * (16 * int64_t(per));
  *reinterpret_cast<u32x4*>(row + c) = og;
  *reinterpret_cast<u32x4*>(row + 8 * int64_t(per) + c) = ou;
}

bool as_is(const uint16_t* V, int64_t ldv, int64_t len) {
  return ldv % 8 == 0 && reinterpret_cast<uintptr_t>(V) % 16 == 0 && len % 64 == 0 &&
         ldv < (int64_t(1) << 22);
}

struct TurnWs {
  float* part;
  uint16_t* Wt;
  uint16_t* V2;
};

TurnWs carve_turn(Carver& c, int64_t n, int64_t m, int64_t d, bool gated) {
  TurnWs w{};
  if (n == 0) return w;
  const int64_t mp = round_up(m, 64), k = mp * (gated ? 2 : 1);
  // a last, shorter chunk of rows may want more parts than a whole one
  size_t floats = mx_dense_floats(std::min<int64_t>(n, kRowChunk), d, k);
  if (n % kRowChunk) floats = std::max(floats, mx_dense_floats(n % kRowChunk, d, k));
  w.part = c.take<float>(floats);
  w.Wt = c.take<uint16_t>(size_t(d) * k);
  if (!gated) w.V2 = c.take<uint16_t>(size_t(std::min<int64_t>(n, kRowChunk)) * mp);
  return w;
}

gptq_status launch_turn(const Mx& w, const Mx& up, int64_t d, uint16_t* Wt, hipStream_t st) {
  const unsigned by = ceil_div(w.rows, 64), two = up.codes ? 2 : 1;
  mx_turn_kernel<<<dim3(ceil_div(d, 256), by * two), 256, 0, st>>>(w, up, by, d, Wt,
                                                                   int64_t(by) * 64 * two);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace

gptq_status launch_mx_quantize(const void* X, gptq_dtype dt, int64_t n, int64_t d, int64_t ldx,
                               uint8_t* codes, uint8_t* scales, void* hat, int64_t ldh,
                               hipStream_t st) {
  if (n == 0) return GPTQ_OK;
  const int item = dt == GPTQ_F32 ? 4 : 2;
  QuantizeArgs a{X, ldx, uint32_t(n), uint32_t((d + 511) / 512), d, mx_blocks(d), codes, scales,
                 hat, ldh, ldx * item % 16 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0,
                 ldh * item % 16 == 0 && reinterpret_cast<uintptr_t>(hat) % 16 == 0};
  const unsigned grid = ceil_div(n * a.runs, 4);
  switch (dt) {
    case GPTQ_F32: mx_quantize_kernel<GPTQ_F32><<<grid, 256, 0, st>>>(a); break;
    case GPTQ_F16: mx_quantize_kernel<GPTQ_F16><<<grid, 256, 0, st>>>(a); break;
    default: mx_quantize_kernel<GPTQ_BF16><<<grid, 256, 0, st>>>(a); break;
  }
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

size_t mx_matmul_ws_bytes(int64_t n, int64_t m, int64_t d, int form, bool gated) {
  return mx_decode_takes(n, m, d, form, gated) ? 0 : mx_gemm_ws_bytes(n, m, d, form, gated);
}

gptq_status launch_mx_matmul(const MxInput& x, const Mx& w, const Mx& up, const MxOutput& y,
                             void* ws, hipStream_t st) {
  return mx_decode_takes(x.n, w.rows, x.d, x.form, up.codes) ? launch_mx_decode(x, w, up, y, st)
                                                             : launch_mx_gemm(x, w, up, y, ws, st);
}

size_t mx_matmul_t_ws_bytes(int64_t n, int64_t m, int64_t d, bool gated) {
  Carver c(nullptr);
  carve_turn(c, n, m, d, gated);
  return c.bytes();
}

gptq_status launch_mx_matmul_t(const uint16_t* dY, int64_t lddy, int64_t n, const Mx& w, int64_t d,
                               uint16_t* dX, int64_t lddx, void* ws, hipStream_t st) {
  Carver c(ws);
  const TurnWs b = carve_turn(c, n, w.rows, d, false);
  const int64_t mp = round_up(w.rows, 64);
  gptq_status s;
  if ((s = launch_turn(w, Mx{}, d, b.Wt, st)) != GPTQ_OK) return s;
  const bool direct = as_is(dY, lddy, w.rows);
  for (int64_t t0 = 0; t0 < n; t0 += kRowChunk) {
    const int64_t nc = std::min<int64_t>(kRowChunk, n - t0);
    const uint16_t* V = dY + t0 * lddy;
    if (!direct) {
      if ((s = launch_pad_rows(V, lddy, nc, w.rows, b.V2, mp, st)) != GPTQ_OK) return s;
      V = b.V2;
    }
    const MxOutput y{dX + t0 * lddx, lddx, 1, GPTQ_ACT_NONE, nullptr, nullptr, 0};
    if ((s = launch_mx_dense(V, direct ? lddy : mp, nc, b.Wt, mp, d, mp, y, b.part, st)) != GPTQ_OK)
      return s;
  }
  return GPTQ_OK;
}

gptq_status launch_mx_gated_backward(const uint16_t* dY, int64_t lddy, int64_t n,
                                     const uint16_t* G, const uint16_t* U, int64_t ldg,
                                     const Mx& gate, const Mx& up, int64_t d, int act,
                                     uint16_t* dX, int64_t lddx, uint16_t* dGU, void* ws,
                                     hipStream_t st) {
  const int64_t m = gate.rows, mp = round_up(m, 64);
  const bool vec = lddy % 8 == 0 && ldg % 8 == 0 && reinterpret_cast<uintptr_t>(dY) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(G) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(U) % 16 == 0;
  mx_gate_grad_kernel<<<ceil_div(n * (mp / 8), 256), 256, 0, st>>>(dY, lddy, G, U, ldg, n, m, act,
                                                                   uint32_t(mp / 8), dGU, vec);
  GPTQ_CHECK_LAUNCH();
  if (!dX) return GPTQ_OK;
  Carver c(ws);
  const TurnWs b = carve_turn(c, n, m, d, true);
  gptq_status s;
  if ((s = launch_turn(gate, up, d, b.Wt, st)) != GPTQ_OK) return s;
  for (int64_t t0 = 0; t0 < n; t0 += kRowChunk) {
    const MxOutput y{dX + t0 * lddx, lddx, 1, GPTQ_ACT_NONE, nullptr, nullptr, 0};
    if ((s = launch_mx_dense(dGU + t0 * 2 * mp, 2 * mp, std::min<int64_t>(kRowChunk, n - t0), b.Wt,
                             2 * mp, d, 2 * mp, y, b.part, st)) != GPTQ_OK)
      return s;
  }
  return GPTQ_OK;
}

}  // namespace gptq
