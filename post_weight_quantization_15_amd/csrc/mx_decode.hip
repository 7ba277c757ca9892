// The 4-bit floating-point products for few activation rows.
//
// Bound by the weights' bytes, and at one token by latency: nothing is laid
// out, no weight passes through LDS.  A wave takes 16 output rows (or 16 of
// either layer of a gated block) and a share of k; lane 16 q + r loads the 16
// bytes that are block 4 s + q of row r, for slabs s of 128 columns, which is
// the operand that the scaled matrix instruction takes, one block's scale a lane
// (4-bit activations), or four operands of the bf16 one after a conversion that
// is exact (bf16 activations; column 32 q + 8 i + v of a slab is then place 8 q
// + v of product i, in both operands).  Activations to be rounded are rounded
// on the way: a lane holds a whole block, so its scale needs no exchange.  The
// waves' sums meet in LDS in the order of k.
//
// Up to 16 rows mx_stream_kernel: a workgroup stays on its CU and goes through tiles, which keeps
// its weights' loads in flight across them and the activations in registers.  Measured, kernel
// alone, 4096 columns: into 11008 one row 12.4 us (1.9 TB/s), 16 rows 15.5; gated 18.9 and 21.4
// (2.3 TB/s; a workgroup a tile took 25); into 4096 5.9 and 8.3.  The bytes at a large copy's rate
// would take half of that; the first loads' and the last sums' latencies are the rest.
#include <algorithm>

#include "mx.h"

namespace gptq {
namespace {

struct DecodeArgs {
  MxInput x;
  Mx w, up;
  MxOutput y;
  bool vec;               // 16-byte loads of bf16 rows are aligned
};

constexpr int kWaves = 8;
constexpr int kSlabs = 4;                    // slabs whose loads are under way at once

// Up to 16 NT rows, a workgroup for each 16 output columns.  FORM: gptq_mx_input.
template <int FORM, int NT, bool GATED>
__global__ __launch_bounds__(kWaves * 64) void mx_decode_kernel(DecodeArgs a) {
  constexpr int JT = GATED ? 2 : 1;                      // layers
  __shared__ f32x4 sums[kWaves][JT * NT][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int64_t j0 = int64_t(blockIdx.x) * 16;
  const int nb = static_cast<int>(a.w.nb), slabs = (nb + 3) / 4;
  const int s0 = slabs * wv / kWaves, s1 = slabs * (wv + 1) / kWaves;
  const uint8_t* wc[JT];
  const uint8_t* wsc[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const Mx& w = j ? a.up : a.w;
    const int64_t row = min(j0 + r, w.rows - 1);
    wc[j] = w.codes + row * nb * 16;
    wsc[j] = w.scales + row * nb;
  }
  const char* xp[NT];
  const uint8_t* xs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t row = min<int64_t>(16 * t + r, a.x.n - 1);
    if (FORM == GPTQ_MX_CODES) {
      xp[t] = static_cast<const char*>(a.x.X) + row * nb * 16;
      xs[t] = a.x.scales + row * nb;
    } else {
      xp[t] = static_cast<const char*>(a.x.X) + row * a.x.ldx * 2;
    }
  }
  f32x4 acc[JT][NT];
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kX = FORM == GPTQ_MX_CODES ? 1 : 4;      // 16-byte loads of a block
  for (int s = s0; s < s1; s += kSlabs) {
    u32x4 w[kSlabs][JT];
    uint32_t sc[kSlabs][JT];
#pragma unroll
    for (int u = 0; u < kSlabs; ++u) {
      const int b = 4 * (s + u) + q;
      // past the share's end or the row's: zeros times 1
      const bool in = s + u < s1 && b < nb;
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        w[u][j] = u32x4{0u, 0u, 0u, 0u};
        sc[u][j] = 127u;
        if (in) {
          w[u][j] = *reinterpret_cast<const u32x4*>(wc[j] + 16 * b);
          sc[u][j] = wsc[j][b];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kSlabs; ++u) {
      if (s + u >= s1) break;
      const int b = 4 * (s + u) + q;
      u32x4 x[NT][kX];
      uint32_t sx[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sx[t] = 127u;
        if (FORM == GPTQ_MX_CODES) {
          x[t][0] = u32x4{0u, 0u, 0u, 0u};
          if (b < nb) {
            x[t][0] = *reinterpret_cast<const u32x4*>(xp[t] + 16 * b);
            sx[t] = xs[t][b];
          }
        } else {
#pragma unroll
          for (int i = 0; i < kX; ++i)
            x[t][i] = load8(reinterpret_cast<const uint16_t*>(xp[t]), 32 * int64_t(b) + 8 * i, a.x.d,
                            a.vec);
        }
      }
      if (FORM == GPTQ_MX_ROUND) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t m = 0u;
#pragma unroll
          for (int i = 0; i < kX; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = mx_amax2(m, x[t][i][e]);
          sx[t] = mx_scale_byte(max(m & 0xFFFFu, m >> 16) << 16);
          const float scale = mx_scale_f32(sx[t]);
          u32x4 c;
#pragma unroll
          for (int i = 0; i < kX; ++i) c[i] = mx_round8(x[t][i], scale);
          x[t][0] = c;
        }
      }
      if (FORM == GPTQ_MX_BF16) {
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const float scale = mx_scale_f32(sc[u][j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const u32x4 f = mx_expand8(w[u][j][i], scale);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[j][t] = mfma16(f, x[t][i % kX], acc[j][t]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
            acc[j][t] = mx_mfma<0>(w[u][j], sc[u][j], x[t][0], sx[t], acc[j][t]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[wv][j * NT + t][lane] = acc[j][t];
  __syncthreads();
  // lane 16 q + r holds columns 4 q .. + 3 of activation row r
  for (int p = wv; p < NT; p += kWaves) {
    f32x4 v = sums[0][p][lane];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v += sums[k][p][lane];
    const int64_t t = 16 * p + r, j = j0 + 4 * q;
    if (t >= a.x.n) continue;
    if constexpr (GATED) {
      f32x4 u = sums[0][NT + p][lane];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) u += sums[k][NT + p][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (j + e >= a.w.rows) break;
        static_cast<uint16_t*>(a.y.Y)[t * a.y.ldy + j + e] = f32_bf16(mx_act(v[e], a.y.act) * u[e]);
        if (a.y.G) {
          a.y.G[t * a.y.ldg + j + e] = f32_bf16(v[e]);
          a.y.U[t * a.y.ldg + j + e] = f32_bf16(u[e]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (j + e >= a.w.rows) break;
        if (a.y.out_bf16) static_cast<uint16_t*>(a.y.Y)[t * a.y.ldy + j + e] = f32_bf16(v[e]);
        else static_cast<float*>(a.y.Y)[t * a.y.ldy + j + e] = v[e];
      }
    }
  }
}

// Up to 16 activation rows, where the weights' stream is the whole of it: one workgroup a CU
// goes through row tiles, the next loads under way beside the products, the sums in two sets
// of LDS in turn.  KEEP: a wave's share of the activations (at most kSlabs slabs) stays in
// registers (4096 columns; longer rows read them again for every tile).
template <int FORM, bool GATED, bool KEEP>
__global__ __launch_bounds__(kWaves * 64, 2) void mx_stream_kernel(DecodeArgs a, int tiles) {
  constexpr int JT = GATED ? 2 : 1;
  __shared__ f32x4 sums[2][kWaves][JT][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int nb = static_cast<int>(a.w.nb), slabs = (nb + 3) / 4;
  const int s0 = slabs * wv / kWaves, s1 = slabs * (wv + 1) / kWaves;
  const int64_t row = min<int64_t>(r, a.x.n - 1);
  const char* xp = static_cast<const char*>(a.x.X) + (FORM == GPTQ_MX_CODES ? row * nb * 16 : row * a.x.ldx * 2);
  const uint8_t* xs = FORM == GPTQ_MX_CODES ? a.x.scales + row * nb : nullptr;
  constexpr int kX = FORM == GPTQ_MX_BF16 ? 4 : 1;       // operands of a slab
  // the activations of one slab (zeros past the share's end), as operands
  auto load_x = [&](int s, u32x4 (&x)[kX], uint32_t& sx) {
    const int b = 4 * s + q;
    sx = 127u;
    if (FORM == GPTQ_MX_CODES) {
      x[0] = u32x4{0u, 0u, 0u, 0u};
      if (s < s1 && b < nb) {
        x[0] = *reinterpret_cast<const u32x4*>(xp + 16 * b);
        sx = xs[b];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kX; ++i) x[i] = u32x4{0u, 0u, 0u, 0u};
      if (s >= s1) return;
      u32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = load8(reinterpret_cast<const uint16_t*>(xp), 32 * int64_t(b) + 8 * i, a.x.d, a.vec);
      if (FORM == GPTQ_MX_ROUND) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = mx_amax2(m, v[i][e]);
        sx = mx_scale_byte(max(m & 0xFFFFu, m >> 16) << 16);
        const float scale = mx_scale_f32(sx);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[0][i] = mx_round8(v[i], scale);
      } else {
#pragma unroll
        for (int i = 0; i < kX; ++i) x[i] = v[i];
      }
    }
  };
  // the weights of kSlabs slabs of a tile (past the share's end or the row's: zeros times 1)
  auto load_w = [&](int tile, int s, u32x4 (&w)[kSlabs][JT], uint32_t (&sc)[kSlabs][JT]) {
    const int64_t j = min(int64_t(tile) * 16 + r, a.w.rows - 1) * nb;
#pragma unroll
    for (int u = 0; u < kSlabs; ++u) {
      const int b = 4 * (s + u) + q;
      const bool in = s + u < s1 && b < nb;
#pragma unroll
      for (int l = 0; l < JT; ++l) {
        const Mx& m = l ? a.up : a.w;
        w[u][l] = u32x4{0u, 0u, 0u, 0u};
        sc[u][l] = 127u;
        if (in) {
          w[u][l] = *reinterpret_cast<const u32x4*>(m.codes + (j + b) * 16);
          sc[u][l] = m.scales[j + b];
        }
      }
    }
  };
  u32x4 w[kSlabs][JT], nw[kSlabs][JT];
  uint32_t sc[kSlabs][JT], nsc[kSlabs][JT];
  int tile = blockIdx.x;
  load_w(tile, s0, w, sc);
  u32x4 x[KEEP ? kSlabs : 1][kX];
  uint32_t sx[KEEP ? kSlabs : 1];
  if (KEEP) {
#pragma unroll
    for (int u = 0; u < (KEEP ? kSlabs : 1); ++u) load_x(s0 + u, x[u], sx[u]);
  }
  for (int turn = 0; tile < tiles; ++turn) {
    f32x4 acc[JT];
#pragma unroll
    for (int l = 0; l < JT; ++l) acc[l] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int next = tile + static_cast<int>(gridDim.x);
    for (int s = s0; s < s1; s += kSlabs) {
      const bool over = s + kSlabs >= s1;
      if (!over || next < tiles) load_w(over ? next : tile, over ? s0 : s + kSlabs, nw, nsc);
#pragma unroll
      for (int u = 0; u < kSlabs; ++u) {
        if (s + u >= s1) break;
        if (!KEEP) load_x(s + u, x[0], sx[0]);
        const int k = KEEP ? u : 0;
#pragma unroll
        for (int l = 0; l < JT; ++l) {
          if (FORM == GPTQ_MX_BF16) {
            const float scale = mx_scale_f32(sc[u][l]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[l] = mfma16(mx_expand8(w[u][l][i], scale), x[k][i % kX], acc[l]);
          } else {
            acc[l] = mx_mfma<0>(w[u][l], sc[u][l], x[k][0], sx[k], acc[l]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kSlabs; ++u)
#pragma unroll
        for (int l = 0; l < JT; ++l) {
          w[u][l] = nw[u][l];
          sc[u][l] = nsc[u][l];
        }
    }
#pragma unroll
    for (int l = 0; l < JT; ++l) sums[turn & 1][wv][l][lane] = acc[l];
    __syncthreads();
    // one wave, another one each turn; lane 16 q + r holds columns 4 q .. + 3 of row r
    if (wv == turn % kWaves) {
      f32x4 v[JT];
#pragma unroll
      for (int l = 0; l < JT; ++l) {
        v[l] = sums[turn & 1][0][l][lane];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) v[l] += sums[turn & 1][k][l][lane];
      }
      const int64_t j = int64_t(tile) * 16 + 4 * q;
      if (r < a.x.n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (j + e >= a.w.rows) break;
          const int64_t at = r * a.y.ldy + j + e;
          if (GATED) {
            static_cast<uint16_t*>(a.y.Y)[at] = f32_bf16(mx_act(v[0][e], a.y.act) * v[JT - 1][e]);
            if (a.y.G) {
              a.y.G[r * a.y.ldg + j + e] = f32_bf16(v[0][e]);
              a.y.U[r * a.y.ldg + j + e] = f32_bf16(v[JT - 1][e]);
            }
          } else if (a.y.out_bf16) {
            static_cast<uint16_t*>(a.y.Y)[at] = f32_bf16(v[0][e]);
          } else {
            static_cast<float*>(a.y.Y)[at] = v[0][e];
          }
        }
      }
    }
    tile = next;
  }
}

template <int FORM, bool GATED>
gptq_status launch_stream(const DecodeArgs& a, hipStream_t st) {
  const int tiles = static_cast<int>(ceil_div(a.w.rows, 16));
  const unsigned grid = static_cast<unsigned>(std::min(tiles, 256));
  // every wave's share: at most kSlabs slabs
  if ((a.w.nb + 3) / 4 <= kSlabs * kWaves)
    mx_stream_kernel<FORM, GATED, true><<<grid, kWaves * 64, 0, st>>>(a, tiles);
  else
    mx_stream_kernel<FORM, GATED, false><<<grid, kWaves * 64, 0, st>>>(a, tiles);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <int FORM, int NT>
gptq_status launch_rows(const DecodeArgs& a, hipStream_t st) {
  const int64_t m = a.w.rows;
  if (a.up.codes)
    mx_decode_kernel<FORM, NT, true><<<ceil_div(m, 16), kWaves * 64, 0, st>>>(a);
  else
    mx_decode_kernel<FORM, NT, false><<<ceil_div(m, 16), kWaves * 64, 0, st>>>(a);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <int FORM>
gptq_status launch_form(const DecodeArgs& a, hipStream_t st) {
  if (a.x.n <= 16)
    return a.up.codes ? launch_stream<FORM, true>(a, st) : launch_stream<FORM, false>(a, st);
  if (a.x.n <= 32) return launch_rows<FORM, 2>(a, st);
  return launch_rows<FORM, 4>(a, st);
}

}  // namespace

// Every 16 output columns read all activations again, which takes over from 16
// rows on (7.5 TB/s from the L2s, as measured: 64 rows of 4096 into 11008 take 54 us here, 24 in
// tiles; of 1024 into 1024 columns 7 and 9).  The same for both 4-bit forms, whose results are the
// same bits: by blocks, as codes tell no more of their width.
bool mx_decode_takes(int64_t n, int64_t m, int64_t d, int form, bool gated) {
  if (n <= 16) return true;
  if (n > 64) return false;
  const double cols = double(form == GPTQ_MX_BF16 ? d : mx_blocks(d) * kMxBlock);
  const double bytes = double(ceil_div(m, 16)) * double(round_up(n, 16)) * cols * 2.0 +
                       double(m) * cols * (gated ? 1.06 : 0.53);
  return 3.0 + bytes / 7.5e6 < 2.5 + mx_gemm_time(n, m, d, form, gated);
}

gptq_status launch_mx_decode(const MxInput& x, const Mx& w, const Mx& up, const MxOutput& y,
                             hipStream_t st) {
  const DecodeArgs a{x, w, up, y, x.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(x.X) % 16 == 0};
  switch (x.form) {
    case GPTQ_MX_BF16: return launch_form<GPTQ_MX_BF16>(a, st);
    case GPTQ_MX_ROUND: return launch_form<GPTQ_MX_ROUND>(a, st);
    default: return launch_form<GPTQ_MX_CODES>(a, st);
  }
}

}  // namespace gptq
