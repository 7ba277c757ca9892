// Low-rank adapters beside the packed weights, and the gradients of the sum:
//   H = X A_a^T,  Y = X W_hat^T + alpha_a H B_a^T,
//   G = alpha_a dY B_a,  dX = dY W_hat + G A_a,
//   dA_a = sum_t G[t]^T X[t],  dB_a = alpha_a sum_t dY[t]^T H[t]
// with a the adapter of each row (outside [0, n_adapters): none).
//
// The simplest form of each: dot products per wave, one thread per output.
#include "common.h"

namespace gptq {
namespace {

__device__ inline float bf16f(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ inline uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

unsigned cdiv(int64_t a, int64_t b) { return static_cast<unsigned>((a + b - 1) / b); }

// Weight (r, c) in fp32.
__device__ inline float weight_at(const Packed& w, int64_t words, int64_t r, int64_t c) {
  const int64_t p = c * w.bits;
  const int64_t i = p >> 5;
  const int off = static_cast<int>(p & 31);
  uint32_t v = w.qw[r * words + i] >> off;
  if (off + w.bits > 32) v |= w.qw[r * words + i + 1] << (32 - off);
  v &= (1u << w.bits) - 1u;
  const int64_t g = r * w.ng + w.g_idx[c];
  const float s = w.scale_f16 ? static_cast<float>(static_cast<const _Float16*>(w.scales)[g])
                              : static_cast<const float*>(w.scales)[g];
  const int hb = 1 << (w.bits - 1);
  const int k = w.sgn ? static_cast<int>(v ^ hb) - hb : static_cast<int>(v) - int(w.zeros[g]);
  return s * static_cast<float>(k);
}

// out[t][q] = scale_a sum_c V[t][c] M_a[q][c], M_a at stride (sq, sc); one wave per q.
__global__ __launch_bounds__(256) void dots_kernel(const uint16_t* __restrict__ V, int64_t ldv,
                                                   int64_t len, const uint16_t* __restrict__ M,
                                                   int64_t per, int64_t sq, int64_t sc,
                                                   gptq_adapters ad, int scaled,
                                                   float* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int a = ad.row[t];
  const bool on = a >= 0 && a < ad.n_adapters;
  for (int q = threadIdx.x >> 6; q < ad.rank; q += 4) {
    float s = 0.0f;
    if (on)
      for (int64_t c = lane; c < len; c += 64)
        s = fmaf(bf16f(V[t * ldv + c]), bf16f(M[a * per + q * sq + c * sc]), s);
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) out[t * ad.rank + q] = on && scaled ? s * ad.alpha[a] : s;
  }
}

// Y[t][j] = base[t][j] + alpha_a sum_q H[t][q] B_a[j][q]
__global__ __launch_bounds__(256) void expand_kernel(const float* base, int64_t ldb,
                                                     const float* __restrict__ H,
                                                     gptq_adapters ad, int64_t m, void* Y,
                                                     int64_t ldy, int out_bf16, int64_t t0) {
  const int64_t t = t0 + blockIdx.y, j = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (j >= m) return;
  float y = base[t * ldb + j];
  const int a = ad.row[t];
  if (a >= 0 && a < ad.n_adapters) {
    const uint16_t* b = static_cast<const uint16_t*>(ad.B) + (a * m + j) * ad.rank;
    float s = 0.0f;
    for (int q = 0; q < ad.rank; ++q) s = fmaf(H[t * ad.rank + q], bf16f(b[q]), s);
    y = fmaf(ad.alpha[a], s, y);
  }
  if (out_bf16) static_cast<uint16_t*>(Y)[t * ldy + j] = to_bf16(y);
  else static_cast<float*>(Y)[t * ldy + j] = y;
}

// dX[t][c] = sum_j dY[t][j] W_hat[j][c] + sum_q G[t][q] A_a[q][c]
__global__ __launch_bounds__(256) void back_kernel(const uint16_t* __restrict__ dY, int64_t lddy,
                                                   int64_t n, Packed w, const float* __restrict__ G,
                                                   gptq_adapters ad, uint16_t* __restrict__ dX,
                                                   int64_t lddx) {
  __shared__ float Ys[32][33], Ws[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c0 = int64_t(blockIdx.x) * 32, t0 = int64_t(blockIdx.y) * 32;
  const int64_t words = (w.d * w.bits + 31) / 32;
  float acc[4] = {};
  for (int64_t j0 = 0; j0 < w.m; j0 += 32) {
    for (int u = 0; u < 4; ++u) {
      const int64_t t = t0 + ty + 8 * u, j = j0 + ty + 8 * u;
      Ys[ty + 8 * u][tx] = t < n && j0 + tx < w.m ? bf16f(dY[t * lddy + j0 + tx]) : 0.0f;
      Ws[ty + 8 * u][tx] = j < w.m && c0 + tx < w.d ? weight_at(w, words, j, c0 + tx) : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
      for (int u = 0; u < 4; ++u) acc[u] = fmaf(Ys[ty + 8 * u][k], Ws[k][tx], acc[u]);
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u) {
    const int64_t t = t0 + ty + 8 * u, c = c0 + tx;
    if (t >= n || c >= w.d) continue;
    float v = acc[u];
    if (G) {
      const int a = ad.row[t];
      if (a >= 0 && a < ad.n_adapters)
        for (int q = 0; q < ad.rank; ++q)
          v = fmaf(G[t * ad.rank + q],
                   bf16f(static_cast<const uint16_t*>(ad.A)[(int64_t(a) * ad.rank + q) * w.d + c]), v);
    }
    dX[t * lddx + c] = to_bf16(v);
  }
}

// out[a][...] (+)= sum over the rows t of a of scale_a L[t][q] V[t][c]; out at
// a * rank * len + q * oq + c * oc.
__global__ __launch_bounds__(256) void outer_kernel(const float* __restrict__ L,
                                                    const uint16_t* __restrict__ V, int64_t ldv,
                                                    int64_t n, int64_t len, gptq_adapters ad,
                                                    int scaled, int64_t oq, int64_t oc,
                                                    int accumulate, float* __restrict__ out) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int q = blockIdx.y, a = blockIdx.z;
  if (c >= len) return;
  float s = 0.0f;
  bool any = false;      // an adapter without a row gets 0, whatever its alpha holds
  for (int64_t t = 0; t < n; ++t)
    if (ad.row[t] == a) {
      s = fmaf(L[t * ad.rank + q], bf16f(V[t * ldv + c]), s);
      any = true;
    }
  if (scaled && any) s *= ad.alpha[a];
  float* o = out + int64_t(a) * ad.rank * len + q * oq + c * oc;
  *o = accumulate ? *o + s : s;
}

}  // namespace

size_t lora_ws_bytes(int64_t n, int64_t m, int64_t d, int rank) {
  if (n == 0) return 0;
  Carver c(nullptr);
  c.take<float>(size_t(n) * rank);
  c.take<float>(size_t(n) * m);
  return c.bytes();
}

gptq_status launch_lora(const uint16_t* X, int64_t ldx, int64_t n, const Packed& w,
                        const gptq_adapters& ad, float* H, void* Y, int out_bf16, int64_t ldy,
                        void* ws, hipStream_t st) {
  Carver c(ws);
  float* h = c.take<float>(size_t(n) * ad.rank);
  float* base = c.take<float>(size_t(n) * w.m);
  int64_t ldb = w.m;
  if (H) h = H;
  if (!out_bf16) {
    base = static_cast<float*>(Y);
    ldb = ldy;
  }
  gptq_status s;
  if ((s = launch_dequant_matmul(X, ldx, n, w.qw, w.m, w.d, w.bits, w.scales, w.scale_f16, w.zeros,
                                 w.ng, w.g_idx, w.sgn, base, ldb, 0, 0, st)) != GPTQ_OK)
    return s;
  dots_kernel<<<unsigned(n), 256, 0, st>>>(X, ldx, w.d, static_cast<const uint16_t*>(ad.A),
                                           ad.rank * w.d, w.d, 1, ad, 0, h);
  GPTQ_CHECK_LAUNCH();
  for (int64_t t0 = 0; t0 < n; t0 += 65535) {
    const dim3 grid(cdiv(w.m, 256), unsigned(n - t0 < 65535 ? n - t0 : 65535));
    expand_kernel<<<grid, 256, 0, st>>>(base, ldb, h, ad, w.m, Y, ldy, out_bf16, t0);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

size_t lora_backward_ws_bytes(int64_t n, int64_t m, int64_t d, int rank, int n_adapters) {
  if (n == 0 || rank == 0) return 0;
  Carver c(nullptr);
  c.take<float>(size_t(n) * rank);
  return c.bytes();
}

gptq_status launch_lora_backward(const uint16_t* dY, int64_t lddy, int64_t n, const uint16_t* X,
                                 int64_t ldx, const float* H, const Packed& w,
                                 const gptq_adapters* adp, uint16_t* dX, int64_t lddx, float* dA,
                                 float* dB, int accumulate, void* ws, hipStream_t st) {
  const gptq_adapters ad = adp ? *adp : gptq_adapters{};
  Carver c(ws);
  float* G = nullptr;
  if (adp && n > 0 && (dX || dA)) {
    G = c.take<float>(size_t(n) * ad.rank);
    dots_kernel<<<unsigned(n), 256, 0, st>>>(dY, lddy, w.m, static_cast<const uint16_t*>(ad.B),
                                             w.m * ad.rank, 1, ad.rank, ad, 1, G);
    GPTQ_CHECK_LAUNCH();
  }
  if (dX && n > 0) {
    back_kernel<<<dim3(cdiv(w.d, 32), cdiv(n, 32)), 256, 0, st>>>(dY, lddy, n, w, G, ad, dX, lddx);
    GPTQ_CHECK_LAUNCH();
  }
  if (dA) {
    outer_kernel<<<dim3(cdiv(w.d, 256), ad.rank, ad.n_adapters), 256, 0, st>>>(
        G, X, ldx, n, w.d, ad, 0, w.d, 1, accumulate, dA);
    GPTQ_CHECK_LAUNCH();
  }
  if (dB) {
    outer_kernel<<<dim3(cdiv(w.m, 256), ad.rank, ad.n_adapters), 256, 0, st>>>(
        H, dY, lddy, n, w.m, ad, 1, 1, ad.rank, accumulate, dB);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

}  // namespace gptq
