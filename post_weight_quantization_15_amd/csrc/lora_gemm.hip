// The matrix-core product behind the adapter operators, and the passes that
// lay its operands out.
//
//   Y[t][j] = sum_k V[t][k] M[j][k]  (+ sum_q (alpha H)[t][q] L_a[j][q])
//
// Forward (Y = X W_hat^T): M holds code - zero, an integer of at most 8
// bits and so exact in bf16, with the columns in group order (act-order
// scatters a group's columns; a sum takes its terms in any order) and every
// group padded to whole 32-column steps.  A 32-step then lies in one group,
// the matrix cores form P = sum x (code - zero) over the group exactly as
// products with fp32 sums, and the group's step folds in once at its end:
// acc += Delta P.  No weight is rounded.  Groups narrower than a step
// (g < 32) would pad to several times the work; there M holds Delta (code -
// zero) as three bf16 parts instead (their sum is the fp32 value), three
// products per weight and no fold.
// Backward (dX = dY W_hat): the sum runs over output rows, each with its own
// step, so no step factors out of it; M is W_hat^T rounded to bf16.  That
// rounding (2^-9 of a weight in the mean) is of the size of the result's own;
// a second part of every weight would take it out and double the product.
#include <algorithm>

#include "lora.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------
// The plan: order[k] = column at place k (-1: padding) and the group of every
// unit of 32 or 64 places.  A wave places one group's columns, in their own order; every
// workgroup counts all groups for itself (g_idx is small and stays in L2).
// In natural order with whole steps per group the order is the identity and
// the activations are used where they lie.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxGroups = 2048;      // groups of at least 32 columns, d <= 65535

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int32_t* __restrict__ g_idx,
                                                            int d, int ng, int unit, int cols_max,
                                                            int32_t* __restrict__ plan) {
  extern __shared__ uint16_t of[];         // the columns' groups
  __shared__ int32_t cnt[kPlanMaxGroups];
  __shared__ int32_t start[kPlanMaxGroups + 1];
  __shared__ int ident;
  const int tid = threadIdx.x, lane = tid & 63;
  int32_t* grp = plan + kPlanHeader;
  int32_t* order = grp + cols_max / unit;
  const int block = max(unit, 64);
  for (int i = tid; i < ng; i += kPlanThreads) cnt[i] = 0;
  if (tid == 0) ident = d % block == 0;
  __syncthreads();
  bool inc = true;
  for (int c0 = 0; c0 < d; c0 += 8 * kPlanThreads) {        // eight loads at a time
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = g_idx[min(c0 + kPlanThreads * i + tid, d - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + kPlanThreads * i + tid;
      if (c >= d) break;
      const int g = min(max(v[i], 0), ng - 1);
      of[c] = static_cast<uint16_t>(g);
      atomicAdd(&cnt[g], 1);
    }
  }
  __syncthreads();
  for (int c = tid + 1; c < d; c += kPlanThreads) inc = inc && of[c] >= of[c - 1];
  if (!inc) ident = 0;
  __syncthreads();
  if (tid < 64) {                          // padded starts: one wave's running sum
    int run = 0;
    for (int b = 0; b < ng; b += 64) {
      const int g = b + lane;
      const int c = g < ng ? cnt[g] : 0;
      if (c % unit) ident = 0;
      int s = (c + unit - 1) / unit * unit;
      const int own = s;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o);
        if (lane >= o) s += u;
      }
      if (g < ng) start[g] = run + s - own;
      run += __shfl(s, 63);
    }
    if (lane == 0) start[ng] = run;
  }
  __syncthreads();
  const int total = start[ng];
  const int padded = (total + block - 1) / block * block;
  if (blockIdx.x == 0) {
    if (tid == 0) {
      plan[0] = ident;
      plan[1] = padded / 64;
    }
    if (tid == 0 && padded > total) grp[total / unit] = -1;   // fills the last block
    for (int k = total + tid; k < padded; k += kPlanThreads) order[k] = -1;
  }
  const int nw = gridDim.x * (kPlanThreads / 64);
  for (int g = blockIdx.x * (kPlanThreads / 64) + (tid >> 6); g < ng; g += nw) {
    const int s = start[g], e = start[g + 1], n = cnt[g];
    for (int k = s / unit + lane; k < e / unit; k += 64) grp[k] = g;
    if (ident) {
      for (int k = s + lane; k < e; k += 64) order[k] = k;
      continue;
    }
    int at = s;
    for (int c0 = 0; c0 < d && at < s + n; c0 += 512) {     // eight reads at a time
      int v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = of[min(c0 + 64 * i + lane, d - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + 64 * i + lane;
        const bool mine = c < d && v[i] == g;
        const uint64_t b = __ballot(mine);
        if (mine) order[at + __popcll(b & ((uint64_t(1) << lane) - 1))] = c;
        at += __popcll(b);
      }
    }
    for (int k = s + n + lane; k < e; k += 64) order[k] = -1;
  }
}

// ---------------------------------------------------------------------------
// Layout passes
// ---------------------------------------------------------------------------

// The eight codes of run ch (columns 8 ch .. + 7) of a row, as integers.
template <int BITS>
__device__ inline void codes8(const uint32_t* __restrict__ p, int64_t words, int64_t ch, int c[8]) {
  uint32_t lo, hi = 0u;
  if (BITS == 4) {
    lo = p[min<int64_t>(ch, words - 1)];
  } else if (BITS == 2) {
    lo = p[min<int64_t>(ch >> 1, words - 1)] >> (16 * (ch & 1));
  } else if (BITS == 8) {
    lo = p[min<int64_t>(2 * ch, words - 1)];
    hi = p[min<int64_t>(2 * ch + 1, words - 1)];
  } else {
    const int64_t bit = 24 * ch;
    const int64_t i = min<int64_t>(bit >> 5, words - 1);
    lo = __builtin_amdgcn_alignbit(p[min<int64_t>(i + 1, words - 1)], p[i],
                                   static_cast<uint32_t>(bit & 31));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = BITS == 8 ? (i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) : lo >> (BITS * i);
    c[i] = static_cast<int>(v & ((1u << BITS) - 1u));
  }
}

__device__ inline int signed_code(int c, int bits) {
  const int hb = 1 << (bits - 1);
  return (c ^ hb) - hb;
}

// One launch lays out everything the plan orders: the first blocks R rows of M
// each (out of natural order through the rows' words in LDS), then the steps
// transposed, then the activations (a block a row at a time, through LDS; nothing to
// do where they are used as they lie).
struct LayoutArgs {
  Packed w;
  int64_t words;
  const int32_t* plan;
  int unit, cols_max;
  uint16_t* M;
  int64_t ldm;
  float* scale_t;
  int64_t mpad;
  const uint16_t* V;
  int64_t ldv, n;
  int always;
  uint16_t* V2;
  int64_t ldv2;
  unsigned blocks_m, blocks_s, blocks_v;
};

template <int BITS, int R>
__global__ __launch_bounds__(256) void layout_kernel(LayoutArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lay_lds[];
  const Packed& w = a.w;
  const int tid = threadIdx.x;
  const int32_t* grp = a.plan + kPlanHeader;
  const int32_t* order = grp + a.cols_max / a.unit;
  const bool ident = a.plan[0];
  const int units = a.plan[1] * 8;
  if (blockIdx.x < a.blocks_m) {
    const int64_t j0 = int64_t(blockIdx.x) * R;
    if (!ident) {
      for (int r = 0; r < R; ++r) {
        const uint32_t* src = w.qw + min<int64_t>(j0 + r, w.m - 1) * a.words;
        for (int i = tid; i < a.words; i += 256) lay_lds[r * a.words + i] = src[i];
      }
      __syncthreads();
    }
    for (int u = tid; u < units; u += 256) {
      const int g = grp[8 * u / a.unit];
      int at[8];
      if (!ident) {
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i] = order[8 * u + i];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t j = j0 + r;
        if (j >= w.m) break;
        u32x4 out = u32x4{0u, 0u, 0u, 0u};
        if (g >= 0) {
          const int z = w.sgn ? 0 : w.zeros[j * w.ng + g];
          int c[8];
          if (ident) {
            codes8<BITS>(w.qw + j * a.words, a.words, u, c);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int p = max(at[i], 0) * BITS;
              const uint32_t* word = lay_lds + r * a.words + (p >> 5);
              uint32_t v = word[0] >> (p & 31);
              if (BITS == 3 && (p & 31) > 29) v |= word[1] << (32 - (p & 31));
              c[i] = static_cast<int>(v & ((1u << BITS) - 1u));
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int v = (w.sgn ? signed_code(c[i], BITS) : c[i]) - z;
            const uint32_t h = __float_as_uint(static_cast<float>(v)) >> 16;
            out[i >> 1] |= (ident || at[i] >= 0 ? h : 0u) << (16 * (i & 1));
          }
        }
        *reinterpret_cast<u32x4*>(a.M + j * a.ldm + 8 * u) = out;
      }
    }
    return;
  }
  if (blockIdx.x < a.blocks_m + a.blocks_s) {
    const int64_t e = int64_t(blockIdx.x - a.blocks_m) * 256 + tid;
    const int64_t j = e / w.ng, g = e % w.ng;
    if (j < w.m) a.scale_t[g * a.mpad + j] = step_at(w, j * w.ng + g);
    return;
  }
  if (ident && !a.always) return;
  uint16_t* rowbuf = reinterpret_cast<uint16_t*>(lay_lds);
  for (int64_t t = blockIdx.x - a.blocks_m - a.blocks_s; t < a.n; t += a.blocks_v) {
    const uint16_t* src = a.V + t * a.ldv;
    __syncthreads();
    for (int c = tid; c < w.d; c += 256) rowbuf[c] = src[c];
    __syncthreads();
    for (int u = tid; u < units; u += 256) {
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = order[8 * u + i];
        v[i >> 1] |= (c >= 0 ? uint32_t(rowbuf[c]) : 0u) << (16 * (i & 1));
      }
      *reinterpret_cast<u32x4*>(a.V2 + t * a.ldv2 + 8 * u) = v;
    }
  }
}

// The whole-row grid: the columns stay as they are.
template <int BITS>
__global__ __launch_bounds__(256) void expand_row_kernel(Packed w, int64_t words,
                                                         uint16_t* __restrict__ M, int64_t ldm,
                                                         float* __restrict__ scale,
                                                         unsigned blocks) {
  if (blockIdx.x >= blocks) {
    const int64_t j = int64_t(blockIdx.x - blocks) * 256 + threadIdx.x;
    if (j < w.m) scale[j] = step_at(w, j);
    return;
  }
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t per = ldm / 8, j = e / per, u = e % per;
  if (j >= w.m) return;
  const int z = w.sgn ? 0 : w.zeros[j];
  int c[8];
  codes8<BITS>(w.qw + j * words, words, u, c);
  u32x4 out = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int v = 8 * u + i < w.d ? (w.sgn ? signed_code(c[i], BITS) : c[i]) - z : 0;
    out[i >> 1] |= (__float_as_uint(static_cast<float>(v)) >> 16) << (16 * (i & 1));
  }
  *reinterpret_cast<u32x4*>(M + j * ldm + 8 * u) = out;
}

__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ V, int64_t ldv,
                                                       int64_t n, int64_t len,
                                                       uint16_t* __restrict__ V2, int64_t cols,
                                                       bool vec) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t per = cols / 8, t = e / per, u = e % per;
  if (t >= n) return;
  *reinterpret_cast<u32x4*>(V2 + t * cols + 8 * u) = load8(V + t * ldv, 8 * u, len, vec);
}

__global__ __launch_bounds__(256) void expand_parts_kernel(Packed w, int64_t words,
                                                           uint16_t* __restrict__ M, int64_t ldp) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t per = ldp / 8, j = e / per, u = e % per;
  if (j >= w.m) return;
  u32x4 out[3] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = 8 * u + i;
    if (c >= w.d) continue;
    const int64_t g = j * w.ng + group_at(w, c);
    const int k = code_at(w, words, j, c) - (w.sgn ? 0 : w.zeros[g]);
    uint16_t p[3];
    split3(step_at(w, g) * static_cast<float>(k), p);
#pragma unroll
    for (int q = 0; q < 3; ++q) out[q][i >> 1] |= uint32_t(p[q]) << (16 * (i & 1));
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
    *reinterpret_cast<u32x4*>(M + j * 3 * ldp + q * ldp + 8 * u) = out[q];
}

// 64 weight rows x 128 columns per workgroup.  A thread takes the same 8-column
// run of two neighbouring rows, so that it writes pairs (two bf16 of one
// column) to the turned tile in LDS: 32 lanes write 32 consecutive words, and
// a column's stride of 144 bytes puts the wave's two runs in different halves
// of the banks.  The tile leaves as 128 contiguous bytes of a column.
constexpr int kTurnCols = 128;

template <int BITS>
__device__ inline void expand_transposed(const Packed& w, int64_t words, uint16_t* __restrict__ M,
                                         int64_t ldm, unsigned bx, unsigned by, char* lds) {
  constexpr int kCols = kTurnCols;
  auto tile = reinterpret_cast<uint32_t(*)[36]>(lds);
  const int tid = threadIdx.x;
  const int64_t c0 = int64_t(bx) * kCols, j0 = int64_t(by) * 64;
  const int pair = tid & 31;
#pragma unroll
  for (int e = 0; e < kCols / 64; ++e) {
    const int run = (tid >> 5) + 8 * e;
    if (c0 + 8 * run >= w.d) break;
    int g[8];
    bool one = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = group_at(w, min<int64_t>(c0 + 8 * run + i, w.d - 1));
      one = one && g[i] == g[0];
    }
    uint32_t out[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t j = j0 + 2 * pair + h;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (j < w.m) {
        int c[8];
        codes8<BITS>(w.qw + j * words, words, c0 / 8 + run, c);
        if (one) {
          const float s = step_at(w, j * w.ng + g[0]);
          const int z = w.sgn ? 0 : w.zeros[j * w.ng + g[0]];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = s * static_cast<float>((w.sgn ? signed_code(c[i], BITS) : c[i]) - z);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = step_at(w, j * w.ng + g[i]) *
                   static_cast<float>((w.sgn ? signed_code(c[i], BITS) : c[i]) -
                                      (w.sgn ? 0 : w.zeros[j * w.ng + g[i]]));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (h == 0) out[i] = f32_bf16(v[i]);
        else out[i] |= uint32_t(f32_bf16(v[i])) << 16;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[8 * run + i][pair] = out[i];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kCols * 8 / 256; ++e) {
    const int cl = (tid >> 3) + 32 * e, u = tid & 7;
    if (c0 + cl < w.d && j0 + 8 * u < ldm)
      *reinterpret_cast<u32x4*>(M + (c0 + cl) * ldm + j0 + 8 * u) =
          *reinterpret_cast<const u32x4*>(&tile[cl][4 * u]);
  }
}

// out[b][x][y] = in[b][y][x], a 64 x 64 tile; rows of `out` at stride ldo, zeros past ny.
__device__ inline void turn_tile(const uint16_t* __restrict__ in, int64_t ny, int64_t nx,
                                 uint16_t* __restrict__ out, int64_t ldo, int64_t b, int64_t x0,
                                 int64_t y0, char* lds) {
  auto tile = reinterpret_cast<uint16_t(*)[66]>(lds);
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int r = w; r < 64; r += 4)
    tile[r][l] = y0 + r < ny && x0 + l < nx ? in[(b * ny + y0 + r) * nx + x0 + l] : uint16_t(0);
  __syncthreads();
  for (int r = w; r < 64; r += 4)
    if (x0 + r < nx && y0 + l < ldo) out[(b * nx + x0 + r) * ldo + y0 + l] = tile[l][r];
}

// Everything the backward pass lays out, one launch: W_hat^T, B and A turned,
// alpha H as parts; each by its range of blocks (0: not asked for).
template <int BITS>
__global__ __launch_bounds__(256) void prepare_kernel(PrepareArgs a, unsigned nw, unsigned wx,
                                                      unsigned nb, unsigned nta, unsigned nh) {
  __shared__ __attribute__((aligned(16))) char lds[kTurnCols * 36 * 4];
  unsigned b = flat_block();
  if (b < nw) {
    expand_transposed<BITS>(a.w, (a.w.d * BITS + 31) / 32, a.Wt, a.mp, b % wx, b / wx, lds);
    return;
  }
  b -= nw;
  const int rank = a.ad.rank;
  if (b < nb) {                              // Bt[a][q][j] = B[a][j][q]
    const unsigned tx = (rank + 63) / 64, ty = static_cast<unsigned>(a.mp / 64);
    turn_tile(static_cast<const uint16_t*>(a.ad.B), a.w.m, rank, a.Bt, a.mp, b / (tx * ty),
              int64_t(b % tx) * 64, int64_t(b / tx % ty) * 64, lds);
    return;
  }
  b -= nb;
  if (b < nta) {                             // At[a][c][q] = A[a][q][c]
    const unsigned tx = static_cast<unsigned>((a.w.d + 63) / 64), ty = (rank + 63) / 64;
    turn_tile(static_cast<const uint16_t*>(a.ad.A), rank, a.w.d, a.At, rank, b / (tx * ty),
              int64_t(b % tx) * 64, int64_t(b / tx % ty) * 64, lds);
    return;
  }
  b -= nta;
  if (b >= nh) return;
  const int64_t e = int64_t(b) * 256 + threadIdx.x;
  const int64_t t = e / a.rp;
  const int p = static_cast<int>(e % a.rp);
  if (t >= a.n) return;
  const int id = a.ad.row[t];                // rows without an adapter are never read
  if (id < 0 || id >= a.ad.n_adapters) return;
  uint16_t part[3];
  split3(p < rank ? a.ad.alpha[id] * a.H[t * rank + p] : 0.0f, part);
#pragma unroll
  for (int u = 0; u < 3; ++u) a.hparts[t * 3 * a.rp + u * a.rp + p] = part[u];
}

// ---------------------------------------------------------------------------
// The product.  A workgroup of WM x WN waves owns TM activation rows x TN
// rows of M; k goes by in blocks of 64 through a ring of S stages in LDS,
// both operands copied by global_load_lds_dwordx4 (no registers) S - 1
// blocks ahead, one barrier per block.  Rows are stored as eight 16-byte
// units, unit c of row r at c ^ ((r / 2) % 8), which the fragment reads (16
// consecutive rows, one unit each) and the copies (8 rows of 8 units) both
// pass without bank conflicts.  M is the matrix instruction's first operand:
// a lane then holds four consecutive j of one activation row, 16 bytes that
// turn through LDS at the end into whole lines of the result.
//
// Reaches 1370 TFLOP/s without a fold on 256 x 256 tiles (8192 rows of 11008
// into 4096: 539 us; 8192 rows of 4096 into 11008: 586, 1260 TFLOP/s) and 764
// with a fold every 64 columns (256 x 128, two sets of accumulators; 16384
// rows of 4096 into 11008: 1.93 ms), against 1430 of a large library product.
// These are times among calls that have run for a while; in the first some
// twenty after a pause the card's clock drops, and they are up to a quarter
// longer.  Measured so, the second took 695, on 256 x 128 tiles 781: matrix
// instructions alone 474 of it, with the barriers 542, with either the copies
// or the LDS reads about 700: no one of them bounds it, their overlap does.
// ---------------------------------------------------------------------------
constexpr int kBk = 64;

__device__ inline uint32_t unit_off(int r, int c) {
  return static_cast<uint32_t>((r * (kBk / 8) + (c ^ ((r >> 1) & 7))) * 16);
}

// P = A B and P += A B.  With two sets of accumulators the register allocator
// moves whole sets about; IN_PLACE pins each to its registers (the product
// written out, P tied).  The compiler then does not know that a matrix
// instruction writes P: what reads P comes behind a barrier (its steps are
// loaded there), or behind wait states written out.
template <bool IN_PLACE>
__device__ inline void open_sum(f32x4& P, const u32x4& a, const u32x4& b) {
  if (IN_PLACE) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "+v"(P) : "v"(a), "v"(b));
  else P = mfma16(a, b, f32x4{0.f, 0.f, 0.f, 0.f});
}
template <bool IN_PLACE>
__device__ inline void add_sum(f32x4& P, const u32x4& a, const u32x4& b) {
  if (IN_PLACE) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(P) : "v"(a), "v"(b));
  else P = mfma16(a, b, P);
}

// KS shares of k, each with its own waves and ring, take the blocks of a tile
// side by side where tiles are few and small: a block's time is then latency
// (barrier, LDS read, a short chain of products), not work.
// FOLD = 0: one sum per output (times a row's step at the end where scale_t
// is given); FOLD = 1, 2: every FOLD 32-steps are one group's, whose step
// folds in.  The fold of a finished group runs fragment by fragment between
// the matrix instructions that open the next one over its registers, so its
// vector work hides behind them.
template <int TM, int TN, int WM, int WN, int KS, int S, int FOLD, bool LORA>
__global__ __launch_bounds__(WM* WN* KS * 64) void gemm_kernel(GemmArgs a, unsigned tiles_j,
                                                           unsigned tiles, int vec_y, int vec_l) {
  constexpr int kWaves = WM * WN;            // of one share of k
  constexpr int kFi = TM / WM / 16;          // activation fragments of a wave
  constexpr int kFj = TN / WN / 16;          // fragments of M
  constexpr int kRows = TM + TN;
  constexpr int kLoads = kRows / 8 / kWaves; // copies per wave and block
  static_assert(kRows % (8 * kWaves) == 0, "copies divide evenly");
  constexpr int kStage = kRows * kBk * 2;
  constexpr int kScale = FOLD ? kWaves * 512 : 0;       // a block's steps, per wave
  constexpr int kOut = kLoads + (FOLD ? 1 : 0);         // copies in flight per block
  constexpr bool kInPlace = kFi * kFj >= 16;
  static_assert((TN / WN) <= 64, "a wave's steps fit its slot");
  // S stages, then S + 1 blocks' steps: those of the block before the one in
  // work are still there when its group folds
  constexpr int kRing = S * kStage + (FOLD ? (S + 1) * kScale : 0);
  extern __shared__ __attribute__((aligned(16))) char lds_all[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int kg = __builtin_amdgcn_readfirstlane((tid >> 6) / kWaves);   // the wave's share of k
  const int wv = __builtin_amdgcn_readfirstlane((tid >> 6) % kWaves);
  char* lds = lds_all + kg * kRing;
  const int q = lane >> 4, c16 = lane & 15;
  // Each XCD (blocks b, b + 8, ...) walks a contiguous range of tiles, in bands
  // of kBand activation tiles: the tiles it runs at once then form a block of
  // them, and its L2 takes in the fewest rows per step.
  constexpr unsigned kBand = 4;
  unsigned tile = blockIdx.x;
  const unsigned per = tiles / 8;
  if (tile < 8 * per) tile = (tile % 8) * per + tile / 8;
  const unsigned tiles_t = tiles / tiles_j, band = tile / (kBand * tiles_j);
  const unsigned high = min(kBand, tiles_t - band * kBand), rest = tile - band * kBand * tiles_j;
  // first row of M, first activation row (divided on the vector unit: made uniform)
  const int64_t jb = int64_t(__builtin_amdgcn_readfirstlane(rest / high)) * TN;
  const int64_t tb = int64_t(__builtin_amdgcn_readfirstlane(band * kBand + rest % high)) * TM;
  const int wi = (wv % WM) * (TM / WM), wj = (wv / WM) * (TN / WN);

  int kblocks = a.kblocks;
  const uint16_t* V = a.V;
  int64_t ldv = a.ldv;
  if (FOLD) {
    kblocks = __builtin_amdgcn_readfirstlane(a.plan[1]);
    if (!__builtin_amdgcn_readfirstlane(a.plan[0]) || !V) {
      V = a.V2;
      ldv = a.ldv2;
    }
  }
  // this share's blocks; all shares turn as often as the longest
  const int kb0 = kblocks * kg / KS, kb1 = kblocks * (kg + 1) / KS;
  const int turns = (kblocks + KS - 1) / KS;
  // the units' groups, through the scalar cache (uniform, and no vector load
  // whose wait would drain the copies in flight)
  const auto grp = (const int32_t __attribute__((address_space(4)))*)(a.plan + kPlanHeader);
  const char* vbase = reinterpret_cast<const char*>(V + tb * ldv);
  const char* mbase = reinterpret_cast<const char*>(a.M + jb * a.ldm);
  // copy i of this wave fills rows 8 (kLoads wv + i) .. + 7 of the stage:
  // activation rows first, then rows of M
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 8 * (kLoads * wv + i) + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    const int64_t row = r < TM ? min<int64_t>(tb + r, a.n - 1) - tb
                               : min<int64_t>(jb + r - TM, a.m - 1) - jb;
    off[i] = static_cast<uint32_t>(row * (r < TM ? ldv : a.ldm) * 2 + 16 * c);
  }
  // groups of a block (past the end: the last one's)
  auto groups_of = [&](int kb, int& ga, int& gb) {
    const int k = max(min(kb0 + kb, kb1 - 1), 0);
    ga = gb = 0;
    if (FOLD == 1) {
      ga = max(grp[2 * k], 0);
      gb = max(grp[2 * k + 1], 0);
    } else if (FOLD) {
      ga = max(grp[k], 0);
    }
  };
  // copies of block kb into its stage (past the end: the last block again,
  // into a stage nobody reads any more, so that every block counts alike)
  auto fetch = [&](int kb, int ga, int gb) {
    const int st = kb % S;
    const int k = __builtin_amdgcn_readfirstlane(max(min(kb0 + kb, kb1 - 1), 0));
    // V repeats for each of up to three parts of M
    const int kv = FOLD ? k : k - (k >= 2 * a.kwrap ? 2 * a.kwrap : k >= a.kwrap ? a.kwrap : 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool act = 8 * (kLoads * wv + i) < TM;
      const char* base = act ? vbase + int64_t(kv) * (kBk * 2) : mbase + int64_t(k) * (kBk * 2);
      // opaque here, so that the copy takes a scalar base and a 32-bit offset
      uint32_t o = off[i];
      asm volatile("" : "+s"(base), "+v"(o));
      __builtin_amdgcn_global_load_lds((gvoid)(base + o),
                                       (lvoid)(lds + st * kStage +
                                               8 * (kLoads * wv + i) * (kBk * 2)),
                                       16, 0, 0);
    }
    if (FOLD) {
      // the wave's rows' steps for the block's group (FOLD = 1: its two groups,
      // lanes 0 .. 15 the first, 16 .. 31 the second), four rows a lane
      const char* base = reinterpret_cast<const char*>(a.scale_t + int64_t(ga) * a.mpad + jb + wj);
      uint32_t o = 16 * c16;
      if (FOLD == 1 && gb != ga) {
        const char* second = reinterpret_cast<const char*>(a.scale_t + int64_t(gb) * a.mpad + jb + wj);
        if (lane & 16) base = second;
      }
      asm volatile("" : "+v"(o));
      if (lane < 32)
        __builtin_amdgcn_global_load_lds((gvoid)(base + o),
                                         (lvoid)(lds + S * kStage + (kb % (S + 1)) * kScale + wv * 512),
                                         16, 0, 0);
    }
  };
  // the lane's unit of its operand rows: 16 rows further is 2048 bytes on
  // (the swizzle repeats), the second 32-step flips bit 2 of the unit
  const uint32_t oa = unit_off(wi + c16, q), om = TM * kBk * 2 + unit_off(wj + c16, q);
  f32x4 acc[kFi][kFj];
  f32x4 P[FOLD ? kFi : 1][FOLD ? kFj : 1];
  const f32x4 zero = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kFj; ++j) {
#pragma unroll
    for (int i = 0; i < kFi; ++i) {
      acc[i][j] = zero;
      if (FOLD) P[i][j] = zero;
    }
  }
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    int ga, gb;
    groups_of(s, ga, gb);
    fetch(s, ga, gb);
  }
  if (FOLD) {                                // steps of the block before the first
    float* none = reinterpret_cast<float*>(lds + S * kStage + S * kScale + wv * 512);
    none[lane] = none[lane + 64] = 0.0f;
  }
  int na, nb;                                // groups of the next block to fetch
  groups_of(S - 1, na, nb);
  for (int kb = 0; kb < turns; ++kb) {
    wait_vmcnt<(S - 2) * kOut>();
    // LDS reads of the stage that is filled next are done as well
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fetch(kb + S - 1, na, nb);
    groups_of(kb + S, na, nb);
    const char* la = lds + (kb % S) * kStage;
    // steps of this block and of the one before
    const char* sc = lds + S * kStage + wv * 512 + 16 * q;
    const char* sc0 = sc + ((kb + S) % (S + 1)) * kScale;
    const char* sc1 = sc + (kb % (S + 1)) * kScale;
    if (KS > 1 && kb >= kb1 - kb0) continue;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      // sums opened by this block's first step are read in its second: all
      // of them behind the wait states a matrix result needs
      if (FOLD == 1 && s && kInPlace) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 7\n\ts_nop 7" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
      u32x4 fa[kFi], fm[kFj];
#pragma unroll
      for (int i = 0; i < kFi; ++i)
        fa[i] = *reinterpret_cast<const u32x4*>(la + (oa ^ (64 * s)) + 2048 * i);
#pragma unroll
      for (int j = 0; j < kFj; ++j)
        fm[j] = *reinterpret_cast<const u32x4*>(la + (om ^ (64 * s)) + 2048 * j);
      if (FOLD && s % (FOLD ? FOLD : 1) == 0) {
#pragma unroll
        for (int j = 0; j < kFj; ++j) {
          // the closing group's steps: the block before's (its second group
          // where a block has two), or this block's first
          const f32x4 d = *reinterpret_cast<const f32x4*>(
              (FOLD == 1 && s ? sc1 : sc0 + (FOLD == 1 ? 256 : 0)) + 64 * j);
#pragma unroll
          for (int i = 0; i < kFi; ++i) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[i][j][v] = fmaf(d[v], P[i][j][v], acc[i][j][v]);
            open_sum<kInPlace>(P[i][j], fm[j], fa[i]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kFj; ++j)
#pragma unroll
          for (int i = 0; i < kFi; ++i) {
            if (FOLD) add_sum<kInPlace>(P[FOLD ? i : 0][FOLD ? j : 0], fm[j], fa[i]);
            else add_sum<kInPlace>(acc[i][j], fm[j], fa[i]);
          }
      }
    }
  }
  wait_vmcnt<0>();
  if (kInPlace) {
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }
  if (FOLD) {
    const char* sc = lds + S * kStage + ((kb1 - kb0 + S) % (S + 1)) * kScale + wv * 512 + 16 * q;
#pragma unroll
    for (int j = 0; j < kFj; ++j) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(sc + (FOLD == 1 ? 256 : 0) + 64 * j);
#pragma unroll
      for (int i = 0; i < kFi; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[v], P[i][j][v], acc[i][j][v]);
    }
  } else if (a.scale_t) {
#pragma unroll
    for (int j = 0; j < kFj; ++j) {
      const f32x4 d = *reinterpret_cast<const f32x4*>(a.scale_t + jb + wj + 16 * j + 4 * q);
#pragma unroll
      for (int i = 0; i < kFi; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] *= d[v];
    }
  }

  // ---- the shares of k, added in their order
  if constexpr (KS > 1) {
    __syncthreads();
    f32x4* sums = reinterpret_cast<f32x4*>(lds_all) + wv * kFi * kFj * 64 + lane;
    constexpr int kAll = kWaves * kFi * kFj * 64;
    static_assert((KS - 1) * kAll * 16 <= KS * kRing, "the shares' sums fit the rings");
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < kFi; ++i)
#pragma unroll
        for (int j = 0; j < kFj; ++j) sums[(kg - 1) * kAll + (i * kFj + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KS - 1; ++g)
#pragma unroll
      for (int i = 0; i < kFi; ++i)
#pragma unroll
        for (int j = 0; j < kFj; ++j) {
          const f32x4 o = sums[g * kAll + (i * kFj + j) * 64];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += o[v];
        }
  }

  // ---- the adapters' part: per adapter among the wave's rows one small
  //      product, added to the rows of that adapter alone
  if (LORA) {
    int ids[kFi];                              // every row's adapter: one wait for all
#pragma unroll
    for (int i = 0; i < kFi; ++i) {
      const int64_t t = tb + wi + 16 * i + c16;
      ids[i] = t < a.n ? a.row[t] : -1;
    }
    auto part_of = [&](int i) {
      int row = wi + 16 * i;                   // opaque: no addresses ahead of their use
      asm volatile("" : "+s"(row));
      return a.parts + min<int64_t>(tb + row + c16, a.n - 1) * 3 * a.rp + 8 * q;
    };
    // the hidden values of the next 16 rows are loaded beside the product of
    // these, an adapter's factors once for rows that follow each other
    u32x4 fn[3], fm[kFj];
#pragma unroll
    for (int p = 0; p < 3; ++p) fn[p] = *reinterpret_cast<const u32x4*>(part_of(0) + p * a.rp);
    int held = -1;
#pragma unroll
    for (int i = 0; i < kFi; ++i) {
      const int id = ids[i];
      u32x4 f0[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) f0[p] = fn[p];
      if (i + 1 < kFi) {
        const uint16_t* next = part_of(i + 1);
#pragma unroll
        for (int p = 0; p < 3; ++p) fn[p] = *reinterpret_cast<const u32x4*>(next + p * a.rp);
      }
      uint32_t left = static_cast<uint32_t>(__ballot(id >= 0 && id < a.n_adapters)) & 0xFFFFu;
      while (left) {
        const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
        const bool mine = id == ad;
        left &= ~static_cast<uint32_t>(__ballot(mine));
        const uint16_t* Lm = a.L + int64_t(ad) * a.m * a.rank;
        f32x4 D[kFj];
#pragma unroll
        for (int j = 0; j < kFj; ++j) D[j] = zero;
        for (int b = 0; b < a.rp; b += 32) {
          u32x4 fa[3];
#pragma unroll
          for (int p = 0; p < 3; ++p) fa[p] = f0[p];
          if (b) {
            const uint16_t* part = part_of(i) + b;
#pragma unroll
            for (int p = 0; p < 3; ++p) fa[p] = *reinterpret_cast<const u32x4*>(part + p * a.rp);
          }
          if (ad != held || a.rp > 32) {
            int col = wj;
            asm volatile("" : "+s"(col));
#pragma unroll
            for (int j = 0; j < kFj; ++j) {
              const int64_t r = min<int64_t>(jb + col + 16 * j + c16, a.m - 1);
              fm[j] = load8(Lm + r * a.rank, b + 8 * q, a.rank, vec_l);
            }
            held = ad;
          }
#pragma unroll
          for (int j = 0; j < kFj; ++j)
#pragma unroll
            for (int p = 0; p < 3; ++p) D[j] = mfma16(fm[j], fa[p], D[j]);
        }
#pragma unroll
        for (int j = 0; j < kFj; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (mine) acc[i][j][v] += D[j][v];
      }
    }
  }
  // ---- results, turned through LDS 16 rows at a time: a lane holds 4 columns
  //      of a row, 4 lanes a row; stored from there, each of a wave's stores
  //      would open 16 rows for 32 bytes each
  constexpr int kCols = TN / WN, kPitch = kCols + 4;
  constexpr int kTurn = KS > 1 ? (KS - 1) * kWaves * kFi * kFj * 1024 : 0;   // behind the sums
  static_assert(kTurn + kWaves * 16 * kPitch * 4 <= KS * kRing, "the turned rows fit the rings");
  if (KS == 1) __syncthreads();                // the last stage is read
  float* out = reinterpret_cast<float*>(lds_all + kTurn) + wv * (16 * kPitch);
  const int64_t r0 = jb + wj;
  const bool wide = vec_y && r0 + kCols <= a.m;
#pragma unroll
  for (int i = 0; i < kFi; ++i) {
#pragma unroll
    for (int j = 0; j < kFj; ++j)
      *reinterpret_cast<f32x4*>(out + c16 * kPitch + 16 * j + 4 * q) = acc[i][j];
    int row = wi + 16 * i;                     // opaque: these rows' addresses only now
    asm volatile("s_waitcnt lgkmcnt(0)" : "+s"(row)::"memory");
    const int64_t t0 = tb + row;
    if (wide && a.out_bf16) {
      constexpr int kPer = kCols / 8;          // lanes a row
#pragma unroll
      for (int r = lane / kPer; r < 16; r += 64 / kPer) {
        const int c = 8 * (lane % kPer);
        const f32x4 lo = *reinterpret_cast<const f32x4*>(out + r * kPitch + c);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(out + r * kPitch + c + 4);
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[e] = uint32_t(f32_bf16(lo[2 * e])) | (uint32_t(f32_bf16(lo[2 * e + 1])) << 16);
          v[e + 2] = uint32_t(f32_bf16(hi[2 * e])) | (uint32_t(f32_bf16(hi[2 * e + 1])) << 16);
        }
        if (t0 + r < a.n)
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.Y) + (t0 + r) * a.ldy + r0 + c) = v;
      }
    } else if (wide) {
      constexpr int kPer = kCols / 4;
#pragma unroll
      for (int r = lane / kPer; r < 16; r += 64 / kPer) {
        const int c = 4 * (lane % kPer);
        const f32x4 v = *reinterpret_cast<const f32x4*>(out + r * kPitch + c);
        if (t0 + r < a.n)
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.Y) + (t0 + r) * a.ldy + r0 + c) = v;
      }
    } else {
      const int c = lane % kCols;
      if (r0 + c < a.m)
        for (int r = lane / kCols; r < 16 && t0 + r < a.n; r += 64 / kCols) {
          const float v = out[r * kPitch + c];
          const int64_t at = (t0 + r) * a.ldy + r0 + c;
          if (a.out_bf16) static_cast<uint16_t*>(a.Y)[at] = f32_bf16(v);
          else static_cast<float*>(a.Y)[at] = v;
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next rows' writes
  }
}

template <int TM, int TN, int WM, int WN, int KS, int S, int FOLD, bool LORA>
gptq_status launch_tile(const GemmArgs& a, hipStream_t st) {
  constexpr int lds =
      KS * (S * (TM + TN) * kBk * 2 + (FOLD ? (S + 1) * WM * WN * 512 : 0));
  static_assert(lds <= 160 * 1024, "the ring fits the LDS");
  const unsigned tj = ceil_div(a.m, TN);
  const unsigned tiles = tj * ceil_div(a.n, TM);
  const int item = a.out_bf16 ? 2 : 4;
  const int vec_y = a.ldy * item % 16 == 0 && reinterpret_cast<uintptr_t>(a.Y) % 16 == 0;
  const int vec_l = a.L && a.rank % 8 == 0 && reinterpret_cast<uintptr_t>(a.L) % 16 == 0;
  gemm_kernel<TM, TN, WM, WN, KS, S, FOLD, LORA><<<tiles, WM * WN * KS * 64, lds, st>>>(a, tj, tiles, vec_y, vec_l);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

// Tiles by the time they take on 256 CUs: rounds of workgroups times a tile's
// area over the rate measured for its shape (relative; wide tiles read less
// per product).  Narrow tiles run several workgroups a CU.
template <int FOLD, bool LORA>
gptq_status launch_fold(const GemmArgs& a, hipStream_t st) {
  auto cost = [&](int tm, int tn, int per_cu, double rate) {
    const int64_t tiles = int64_t(ceil_div(a.n, tm)) * ceil_div(a.m, tn);
    const int64_t rounds = (tiles + 256 * per_cu - 1) / (256 * per_cu);
    // a last round that leaves CUs with fewer workgroups than others is as long
    const int64_t left = tiles - (rounds - 1) * 256 * per_cu;
    const int64_t last = (left + 255) / 256;
    return double((rounds - 1) * per_cu + last) * tm * tn / rate;
  };
  const double c256 = FOLD == 0 ? cost(256, 256, 1, 1.2) : 1e30, cw = cost(256, 128, 1, 1.0);
  const double c128 = cost(128, 128, 1, 0.75), c64 = cost(64, 64, 3, 0.40), c32 = cost(32, 32, 6, 0.18);
  const double best = std::min(std::min(std::min(c256, cw), std::min(c128, c64)), c32);
  if constexpr (FOLD == 0)
    if (best == c256) return launch_tile<256, 256, 2, 4, 1, 2, 0, LORA>(a, st);
  if (best == cw) return launch_tile<256, 128, 4, 2, 1, 3, FOLD, LORA>(a, st);
  if (best == c128) return launch_tile<128, 128, 2, 2, 2, 2, FOLD, LORA>(a, st);
  if (best == c64) return launch_tile<64, 64, 2, 2, 4, 2, FOLD, LORA>(a, st);
  return launch_tile<32, 32, 1, 2, 8, 2, FOLD, LORA>(a, st);
}

}  // namespace

int fold_unit(int64_t group) {
  return group % 64 == 0 ? 64 : 32;
}

int64_t plan_cols(int64_t d, int64_t ng, int64_t group) {
  const int u = fold_unit(group);
  return round_up(d + (u - 1) * ng, std::max(u, 64));
}

size_t plan_words(int64_t d, int64_t ng, int64_t group) {
  const int64_t cols = plan_cols(d, ng, group);
  return size_t(kPlanHeader + cols / fold_unit(group) + cols);
}

gptq_status launch_plan(const Packed& w, int32_t* plan, hipStream_t st) {
  const unsigned grid = w.ng < 512 ? ceil_div(w.ng, 8) : 64;
  plan_kernel<<<grid, kPlanThreads, size_t(w.d) * 2, st>>>(w.g_idx, int(w.d), int(w.ng), fold_unit(w.group),
                                             int(plan_cols(w.d, w.ng, w.group)), plan);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status launch_layout(const Packed& w, const int32_t* plan, uint16_t* M, int64_t ldm,
                          float* scale_t, int64_t mpad, const uint16_t* V, int64_t ldv, int64_t n,
                          int always, uint16_t* V2, int64_t ldv2, hipStream_t st) {
  LayoutArgs a{w, (w.d * w.bits + 31) / 32, plan, fold_unit(w.group),
               int(plan_cols(w.d, w.ng, w.group)), M, ldm, scale_t, mpad, V, ldv, n, always, V2,
               ldv2, 0, 0, 0};
  // four rows share the loads of the order where their words fit in LDS
  const int rows = a.words * 16 <= 64 * 1024 ? 4 : 1;
  if (M) {
    a.blocks_m = ceil_div(w.m, rows);
    a.blocks_s = ceil_div(w.m * w.ng, 256);
  }
  a.blocks_v = unsigned(std::min<int64_t>(n, 2048));
  const size_t lds = std::max<size_t>(M ? size_t(a.words) * 4 * rows : 0, size_t(w.d) * 2);
  const unsigned grid = a.blocks_m + a.blocks_s + a.blocks_v;
#define GPTQ_LAY(B)                                                     \
  do {                                                                  \
    if (rows == 4) layout_kernel<B, 4><<<grid, 256, lds, st>>>(a);      \
    else layout_kernel<B, 1><<<grid, 256, lds, st>>>(a);                \
  } while (0)
  switch (w.bits) {
    case 2: GPTQ_LAY(2); break;
    case 3: GPTQ_LAY(3); break;
    case 4: GPTQ_LAY(4); break;
    default: GPTQ_LAY(8); break;
  }
#undef GPTQ_LAY
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status launch_expand_row(const Packed& w, uint16_t* M, int64_t ldm, float* scale,
                              hipStream_t st) {
  const int64_t words = (w.d * w.bits + 31) / 32;
  const unsigned blocks = ceil_div(w.m * (ldm / 8), 256);
  const unsigned grid = blocks + ceil_div(w.m, 256);
#define GPTQ_EX(B) \
  expand_row_kernel<B><<<grid, 256, 0, st>>>(w, words, M, ldm, scale, blocks)
  switch (w.bits) {
    case 2: GPTQ_EX(2); break;
    case 3: GPTQ_EX(3); break;
    case 4: GPTQ_EX(4); break;
    default: GPTQ_EX(8); break;
  }
#undef GPTQ_EX
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status launch_pad_rows(const uint16_t* V, int64_t ldv, int64_t n, int64_t len, uint16_t* V2,
                            int64_t cols, hipStream_t st) {
  const bool vec = ldv % 8 == 0 && reinterpret_cast<uintptr_t>(V) % 16 == 0;
  pad_rows_kernel<<<ceil_div(n * (cols / 8), 256), 256, 0, st>>>(V, ldv, n, len, V2, cols, vec);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status launch_expand_parts(const Packed& w, uint16_t* M, int64_t ldp, hipStream_t st) {
  expand_parts_kernel<<<ceil_div(w.m * (ldp / 8), 256), 256, 0, st>>>(
      w, (w.d * w.bits + 31) / 32, M, ldp);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status launch_prepare(const PrepareArgs& a, hipStream_t st) {
  const unsigned wx = ceil_div(a.w.d, kTurnCols);
  const unsigned nw = a.Wt ? wx * ceil_div(a.mp, 64) : 0;
  const unsigned count = static_cast<unsigned>(a.ad.n_adapters), tr = (a.ad.rank + 63) / 64;
  const unsigned nb = a.Bt ? tr * ceil_div(a.mp, 64) * count : 0;
  const unsigned na = a.At ? tr * ceil_div(a.w.d, 64) * count : 0;
  const unsigned nh = a.hparts ? ceil_div(a.n * a.rp, 256) : 0;
  if (!(nw + nb + na + nh)) return GPTQ_OK;
  const dim3 grid = flat_grid(int64_t(nw) + nb + na + nh);
  switch (a.w.bits) {
    case 2: prepare_kernel<2><<<grid, 256, 0, st>>>(a, nw, wx, nb, na, nh); break;
    case 3: prepare_kernel<3><<<grid, 256, 0, st>>>(a, nw, wx, nb, na, nh); break;
    case 4: prepare_kernel<4><<<grid, 256, 0, st>>>(a, nw, wx, nb, na, nh); break;
    default: prepare_kernel<8><<<grid, 256, 0, st>>>(a, nw, wx, nb, na, nh); break;
  }
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

gptq_status launch_gemm(const GemmArgs& a, int fold, hipStream_t st) {
  switch (fold) {
    case 64: return launch_fold<2, true>(a, st);
    case 32: return launch_fold<1, true>(a, st);
  }
  return a.L ? launch_fold<0, true>(a, st) : launch_fold<0, false>(a, st);
}

}  // namespace gptq
