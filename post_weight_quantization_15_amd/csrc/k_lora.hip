// Low-rank adapters beside the packed weights, and the gradients of the sum:
//   H = X A_a^T,  Y = X W_hat^T + alpha_a H B_a^T,
//   G = alpha_a dY B_a,  dX = dY W_hat + G A_a,
//   dA_a = sum_t G[t]^T X[t],  dB_a = alpha_a sum_t dY[t]^T H[t]
// with a the adapter of each row (outside [0, n_adapters): none).
//
// The hidden values H and G are fp32; where they meet a matrix instruction
// they go in as three bf16 parts, whose sum is the fp32 value, so that no
// output depends on a rounding of them.  This file holds the two narrow
// products (n x rank from the activations; rank x width over the rows) and
// the order of the launches; the wide one is in lora_gemm.hip.
#include <algorithm>

#include "lora.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------
// Down to the hidden values: out[t][p] = sum_k V[t][k] M_a[p][k].
//
// A workgroup owns 32 rows; its four waves take every fourth 32-step of k
// (and grid.y a share of the steps where there are few rows), and their
// sums meet in LDS.  Rows are independent in the product, so a tile with
// several adapters runs once per adapter and keeps each adapter's rows.
// Read once per adapter of the tile: 32 rows of V from HBM, rank rows of
// M from L2.
// ---------------------------------------------------------------------------
constexpr int kShrinkRows = 32;

struct ShrinkArgs {
  const uint16_t* V;
  int64_t ldv, n, len;
  const uint16_t* M;        // [n_adapters][rank][ldm], k contiguous
  int64_t ldm;
  const int32_t* row;
  int n_adapters, rank, rp;
  const float* alpha;
  int scaled;               // H holds alpha out (G), else out (H); the parts are of alpha out
  float* H;                 // [n][rank] or NULL
  uint16_t* parts;          // [n][3 rp]
  float* sums;              // [grid.y][n][rank] when grid.y > 1
};

// Value q of row t: to H, and alpha times it as parts.
__device__ inline void put_hidden(const ShrinkArgs& a, int64_t t, int p, float v, float al) {
  if (p >= a.rank) v = 0.0f;
  const float s = p < a.rank ? al * v : 0.0f;
  if (a.H && p < a.rank) a.H[t * a.rank + p] = a.scaled ? s : v;
  uint16_t part[3];
  split3(s, part);
#pragma unroll
  for (int u = 0; u < 3; ++u) a.parts[t * 3 * a.rp + u * a.rp + p] = part[u];
}

template <int NF>
__global__ __launch_bounds__(256) void shrink_kernel(ShrinkArgs a, bool vec_v, bool vec_m) {
  __shared__ float red[4][kShrinkRows][16 * NF + 4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int q = lane >> 4, c16 = lane & 15;
  const int64_t t0 = int64_t(blockIdx.x) * kShrinkRows;
  const int id = lane < kShrinkRows && t0 + lane < a.n ? a.row[t0 + lane] : -1;
  const bool valid = id >= 0 && id < a.n_adapters;
  uint32_t left = static_cast<uint32_t>(__ballot(valid));
  const uint32_t none = ~left;
  const int64_t steps = (a.len + 31) / 32;
  const int64_t s0 = steps * blockIdx.y / gridDim.y, s1 = steps * (blockIdx.y + 1) / gridDim.y;
  const uint16_t* vr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) vr[i] = a.V + min<int64_t>(t0 + 16 * i + c16, a.n - 1) * a.ldv;
  while (left) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t in = static_cast<uint32_t>(__ballot(id == ad));
    left &= ~in;
    const uint16_t* Ma = a.M + int64_t(ad) * a.rank * a.ldm;
    f32x4 acc[2][NF];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    int64_t s = s0 + wv;
    if (vec_v && vec_m) {                  // whole steps, loads back to back
      const int64_t whole = min(s1, a.len / 32);
      const uint16_t* mr[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f)
        mr[f] = Ma + int64_t(min(16 * f + c16, a.rank - 1)) * a.ldm + 8 * q;
#pragma unroll(NF > 2 ? 2 : 4)
      for (; s < whole; s += 4) {
        u32x4 fv[2], fm[NF];
#pragma unroll
        for (int i = 0; i < 2; ++i) fv[i] = *reinterpret_cast<const u32x4*>(vr[i] + 32 * s + 8 * q);
#pragma unroll
        for (int f = 0; f < NF; ++f) fm[f] = *reinterpret_cast<const u32x4*>(mr[f] + 32 * s);
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[i][f] = mfma16(fm[f], fv[i], acc[i][f]);
      }
    }
    for (; s < s1; s += 4) {
      u32x4 fv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) fv[i] = load8(vr[i], 32 * s + 8 * q, a.len, vec_v);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const u32x4 fm = load8(Ma + int64_t(min(16 * f + c16, a.rank - 1)) * a.ldm, 32 * s + 8 * q,
                               a.len, vec_m);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i][f] = mfma16(fm, fv[i], acc[i][f]);
      }
    }
    __syncthreads();          // the previous adapter's sums are read
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        *reinterpret_cast<f32x4*>(&red[wv][16 * i + c16][16 * f + 4 * q]) = acc[i][f];
    __syncthreads();
    for (int e = tid; e < kShrinkRows * a.rp; e += 256) {
      const int tl = e / a.rp, p = e % a.rp;
      if (!((in >> tl) & 1u)) continue;
      const int64_t t = t0 + tl;
      float v = 0.0f;
      if (p < a.rank) v = (red[0][tl][p] + red[1][tl][p]) + (red[2][tl][p] + red[3][tl][p]);
      if (gridDim.y > 1) {
        if (p < a.rank) a.sums[(int64_t(blockIdx.y) * a.n + t) * a.rank + p] = v;
      } else {
        put_hidden(a, t, p, v, a.alpha[ad]);
      }
    }
  }
  // rows without an adapter
  if (blockIdx.y == 0 && a.H)
    for (int e = tid; e < kShrinkRows * a.rank; e += 256) {
      const int tl = e / a.rank;
      if (((none >> tl) & 1u) && t0 + tl < a.n) a.H[(t0 + tl) * a.rank + e % a.rank] = 0.0f;
    }
}

// The shares of grid.y, added in their order.
__global__ __launch_bounds__(256) void shrink_sum_kernel(ShrinkArgs a, int shares) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = e / a.rp;
  const int p = static_cast<int>(e % a.rp);
  if (t >= a.n) return;
  const int id = a.row[t];
  if (id < 0 || id >= a.n_adapters) return;
  float v = 0.0f;
  if (p < a.rank)
    for (int s = 0; s < shares; ++s) v += a.sums[(int64_t(s) * a.n + t) * a.rank + p];
  put_hidden(a, t, p, v, a.alpha[id]);
}

// Shares of k per row tile: enough workgroups for the chip where rows are
// few, at least 16 steps each.
int shrink_shares(int64_t n, int64_t len) {
  const int64_t tiles = (n + kShrinkRows - 1) / kShrinkRows;
  return tiles >= 128 ? 1 : int(std::max<int64_t>(1, std::min<int64_t>(512 / tiles, (len + 511) / 512)));
}

gptq_status launch_shrink(const ShrinkArgs& a, hipStream_t st) {
  const bool vv = a.ldv % 8 == 0 && reinterpret_cast<uintptr_t>(a.V) % 16 == 0;
  const bool vm = a.ldm % 8 == 0 && reinterpret_cast<uintptr_t>(a.M) % 16 == 0;
  const int shares = shrink_shares(a.n, a.len);
  const dim3 grid(ceil_div(a.n, kShrinkRows), shares);
  if (a.rank <= 16) shrink_kernel<1><<<grid, 256, 0, st>>>(a, vv, vm);
  else if (a.rank <= 32) shrink_kernel<2><<<grid, 256, 0, st>>>(a, vv, vm);
  else if (a.rank <= 64) shrink_kernel<4><<<grid, 256, 0, st>>>(a, vv, vm);
  else shrink_kernel<8><<<grid, 256, 0, st>>>(a, vv, vm);
  GPTQ_CHECK_LAUNCH();
  if (shares > 1) {
    shrink_sum_kernel<<<ceil_div(a.n * a.rp, 256), 256, 0, st>>>(a, shares);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

// parts[t] = the three parts of alpha_a H[t] (dB); rows without an adapter are never read.
__global__ __launch_bounds__(256) void split_kernel(ShrinkArgs a, const float* __restrict__ H) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = e / a.rp;
  const int p = static_cast<int>(e % a.rp);
  if (t >= a.n) return;
  const int id = a.row[t];
  if (id < 0 || id >= a.n_adapters) return;
  put_hidden(a, t, p, p < a.rank ? H[t * a.rank + p] : 0.0f, a.alpha[id]);
}

// out[b][x][y] = in[b][y][x], 64 x 64 tiles; rows of `out` at stride ldo, zeros past `ny`.
__global__ __launch_bounds__(256) void turn_kernel(const uint16_t* __restrict__ in, int64_t ny,
                                                   int64_t nx, uint16_t* __restrict__ out,
                                                   int64_t ldo) {
  __shared__ uint16_t tile[64][66];
  const int64_t x0 = int64_t(blockIdx.x) * 64, y0 = int64_t(blockIdx.y) * 64;
  const int64_t b = blockIdx.z;
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int r = w; r < 64; r += 4)
    tile[r][l] = y0 + r < ny && x0 + l < nx ? in[(b * ny + y0 + r) * nx + x0 + l] : uint16_t(0);
  __syncthreads();
  for (int r = w; r < 64; r += 4)
    if (x0 + r < nx && y0 + l < ldo) out[(b * nx + x0 + r) * ldo + y0 + l] = tile[l][r];
}

// ---------------------------------------------------------------------------
// Over the rows of an adapter: out_a[p][c] = sum_t L[t][p] V[t][c], L given
// as three bf16 parts.
//
// A workgroup owns one adapter, 128 columns and a share of the rows.  It
// lists its adapter's rows (in their order, 4096 row ids at a time), and
// takes them 32 a step: the rows' 256-byte pieces of V and the rows' parts go
// through LDS and come back transposed (ds_read_b64_tr_b16: the sum runs
// over rows, which is the slow direction of both).  The parts of V outside
// the list are never read.  Where the shares of an adapter are several, each
// leaves its sums and a last pass adds them in order: no atomics, the same
// bits every time.
// ---------------------------------------------------------------------------
constexpr int kOuterCols = 128;
constexpr int kOuterList = 4096;

struct OuterArgs {
  const uint16_t* V;
  int64_t ldv, n, len;
  const uint16_t* parts;     // [n][3 rp]
  const int32_t* row;
  int rank, rp, shares;
  int by_column;             // 1: out_a [len][rank] (dB), 0: [rank][len] (dA)
  int accumulate;
  float* out;                // shares == 1: the result, else [a][share] sums
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ inline uint2 tr_read(const char* p) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)p);
  return __builtin_bit_cast(uint2, v);
}

// 16-byte chunk c of row r of the V tile is stored at chunk c ^ swz(r): the
// eight rows that a half wave's transposing read touches then lie in
// different banks.
__device__ inline int swz(int r) { return 2 * ((r & 3) | (((r >> 3) & 1) << 2)); }

template <int NF>
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs a, bool vec_v) {
  constexpr int kRp = NF <= 2 ? 32 : 16 * NF;               // padded rank
  constexpr int kPartRow = kRp * 2 + 16;                    // bytes of a row of one part in LDS
  __shared__ __attribute__((aligned(16))) char lv[32 * kOuterCols * 2];
  __shared__ __attribute__((aligned(16))) char lp[3][32 * kPartRow];
  __shared__ int32_t list[kOuterList];
  __shared__ int wcount[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int kg = lane >> 4, c16 = lane & 15;
  const int64_t c0 = int64_t(blockIdx.x) * kOuterCols;
  const int ad = blockIdx.z, share = blockIdx.y;
  const int64_t r0 = a.n * share / a.shares, r1 = a.n * (share + 1) / a.shares;
  f32x4 acc[NF][2];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int rr = 8 * kg + (c16 >> 2);                       // row the lane points a read at
  for (int64_t p0 = r0; p0 < r1; p0 += kOuterList) {
    // ---- the adapter's rows of this piece, in order
    const int piece = static_cast<int>(min<int64_t>(kOuterList, r1 - p0));
    int count = 0;
    for (int b = 0; b < piece; b += 256) {
      const int e = b + tid;
      const bool mine = e < piece && a.row[p0 + e] == ad;
      const uint64_t m = __ballot(mine);
      __syncthreads();
      if (lane == 0) wcount[wv] = __popcll(m);
      __syncthreads();
      int at = count;
      for (int w = 0; w < wv; ++w) at += wcount[w];
      if (mine) list[at + __popcll(m & ((uint64_t(1) << lane) - 1))] = e;
      count += wcount[0] + wcount[1] + wcount[2] + wcount[3];
    }
    __syncthreads();
    for (int s = 0; s < count; s += 32) {
      // ---- stage the step: thread t the two 16-byte chunks 2 (t % 8), + 1 of row t / 8 of V
      const int rl = tid >> 3;
      const bool have = s + rl < count;
      const int64_t t = p0 + (have ? list[s + rl] : 0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ch = 2 * (tid & 7) + h;
        u32x4 v = u32x4{0u, 0u, 0u, 0u};
        if (have) v = load8(a.V + t * a.ldv, c0 + 8 * ch, a.len, vec_v);
        *reinterpret_cast<u32x4*>(lv + rl * (kOuterCols * 2) + 16 * (ch ^ swz(rl))) = v;
      }
      for (int ch = tid & 7; ch < 3 * kRp / 8; ch += 8) {
        u32x4 v = u32x4{0u, 0u, 0u, 0u};
        if (have) v = *reinterpret_cast<const u32x4*>(a.parts + t * 3 * a.rp + 8 * ch);
        *reinterpret_cast<u32x4*>(lp[ch / (kRp / 8)] + rl * kPartRow + 16 * (ch % (kRp / 8))) = v;
      }
      __syncthreads();
      u32x4 fv[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int f8 = (32 * wv + 16 * j + 4 * (c16 & 3)) * 2;      // byte of the lane's columns
        const uint2 lo = tr_read(lv + rr * (kOuterCols * 2) + 16 * ((f8 >> 4) ^ swz(rr)) + (f8 & 15));
        const uint2 hi = tr_read(lv + (rr + 4) * (kOuterCols * 2) + 16 * ((f8 >> 4) ^ swz(rr + 4)) + (f8 & 15));
        fv[j] = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          const char* b = lp[p] + rr * kPartRow + (16 * f + 4 * (c16 & 3)) * 2;
          const uint2 lo = tr_read(b), hi = tr_read(b + 4 * kPartRow);
          const u32x4 fl = u32x4{lo.x, lo.y, hi.x, hi.y};
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[f][j] = a.by_column ? mfma16(fv[j], fl, acc[f][j]) : mfma16(fl, fv[j], acc[f][j]);
        }
      __syncthreads();
    }
  }
  // ---- by row (dA): lane holds p = 16 f + 4 kg + v, column c16; by column
  //      (dB): lane holds columns 4 kg + v, p = 16 f + c16
  float* out = a.out + (int64_t(ad) * a.shares + share) * a.rank * a.len;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int p = 16 * f + (a.by_column ? c16 : 4 * kg + v);
        const int64_t c = c0 + 32 * wv + 16 * j + (a.by_column ? 4 * kg + v : c16);
        if (p >= a.rank || c >= a.len) continue;
        float* o = out + (a.by_column ? c * a.rank + p : p * a.len + c);
        *o = a.accumulate && a.shares == 1 ? *o + acc[f][j][v] : acc[f][j][v];
      }
}

__global__ __launch_bounds__(256) void outer_sum_kernel(const float* __restrict__ sums, int shares,
                                                        int64_t per, int64_t total, int accumulate,
                                                        float* __restrict__ out) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (e >= total) return;
  const float* s = sums + e / per * shares * per + e % per;
  float v = s[0];
  for (int i = 1; i < shares; ++i) v += s[i * per];
  out[e] = accumulate ? out[e] + v : v;
}

__global__ void zero_kernel(float* __restrict__ p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// Shares of the rows per adapter: enough workgroups, at least 256 rows each,
// and sums of at most 64 (adapter, share) pairs and 256 MB.
int outer_shares(int64_t n, int64_t len, int rank, int count) {
  int64_t s = 1024 / int64_t(ceil_div(len, kOuterCols));
  s = std::min<int64_t>(s, (n + 255) / 256);
  s = std::min<int64_t>(s, 64 / count);
  s = std::min<int64_t>(s, (int64_t(256) << 20) / (int64_t(count) * rank * len * 4));
  return int(std::max<int64_t>(s, 1));
}

size_t outer_floats(int64_t n, int64_t len, int rank, int count) {
  const int s = outer_shares(n, len, rank, count);
  return s > 1 ? size_t(s) * count * rank * len : 0;
}

gptq_status launch_outer(OuterArgs a, int count, float* sums, float* out, hipStream_t st) {
  const bool vec = a.ldv % 8 == 0 && reinterpret_cast<uintptr_t>(a.V) % 16 == 0;
  a.out = a.shares > 1 ? sums : out;
  const dim3 grid(ceil_div(a.len, kOuterCols), a.shares, count);
  if (a.rank <= 16) outer_kernel<1><<<grid, 256, 0, st>>>(a, vec);
  else if (a.rank <= 32) outer_kernel<2><<<grid, 256, 0, st>>>(a, vec);
  else if (a.rank <= 64) outer_kernel<4><<<grid, 256, 0, st>>>(a, vec);
  else outer_kernel<8><<<grid, 256, 0, st>>>(a, vec);
  GPTQ_CHECK_LAUNCH();
  if (a.shares > 1) {
    const int64_t per = int64_t(a.rank) * a.len, total = per * count;
    outer_sum_kernel<<<ceil_div(total, 256), 256, 0, st>>>(sums, a.shares, per, total,
                                                           a.accumulate, out);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

// Rows that a 16-byte copy can take as they lie: aligned, whole 64-blocks, and
// a tile's rows within 32-bit offsets.
bool as_is(const uint16_t* V, int64_t ldv, int64_t len) {
  return ldv % 8 == 0 && reinterpret_cast<uintptr_t>(V) % 16 == 0 && len % 64 == 0 &&
         ldv < (int64_t(1) << 22);
}

// Rank as the padded layouts and kernels take it (a shrink of rank > 64 uses
// eight fragments, its parts 128 wide).
int parts_rank(int rank) { return rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// ---- workspaces
struct LoraWs {
  float* hidden;
  uint16_t* parts;
  float* sums;
  int32_t* plan;
  uint16_t* M;
  float* scale_t;
  uint16_t* V2;
};

// How the shared product is laid out: by groups that fold, by the row's one
// step, or (groups narrower than a matrix step) as parts of the weights.
enum { kByGroups, kByRow, kByParts };
int layout_of(int64_t group) { return group == -1 ? kByRow : group >= 32 ? kByGroups : kByParts; }

LoraWs carve_lora(Carver& c, int64_t n, int64_t m, int64_t d, int64_t group, int rank) {
  const int64_t nc = std::min<int64_t>(n, kRowChunk);
  const int64_t ng = group > 0 ? (d + group - 1) / group : 1;
  LoraWs w{};
  if (decode_takes(n, ng)) {
    w.hidden = c.take<float>(size_t(n) * rank);
    return w;
  }
  w.parts = c.take<uint16_t>(size_t(nc) * 3 * parts_rank(rank));
  const int shares = shrink_shares(nc, d);
  w.sums = c.take<float>(shares > 1 ? size_t(shares) * nc * rank : 0);
  const int64_t mpad = round_up(m, 256) + 64, ldp = round_up(d, 64);
  const int lay = layout_of(group);
  const int64_t cols = lay == kByGroups ? plan_cols(d, ng, group) : ldp;
  if (lay == kByGroups) w.plan = c.take<int32_t>(plan_words(d, ng, group));
  if (lay != kByParts) w.scale_t = c.take<float>(size_t(ng) * mpad);
  w.M = c.take<uint16_t>(size_t(m) * (lay == kByParts ? 3 * ldp : cols));
  w.V2 = c.take<uint16_t>(size_t(nc) * cols);
  return w;
}

struct BackWs {
  uint16_t* parts;
  float* sums;
  uint16_t* At;      // [count][d][rank]
  uint16_t* Bt;      // [count][rank][mp]
  uint16_t* Wt;      // [d][mp]
  uint16_t* V2;      // [rows][mp]
  float* outer;
};

BackWs carve_back(Carver& c, int64_t n, int64_t m, int64_t d, int rank, int count) {
  const int64_t nc = std::min<int64_t>(n, kRowChunk), mp = round_up(m, 64);
  BackWs w{};
  if (n == 0) return w;
  w.Wt = c.take<uint16_t>(size_t(d) * mp);
  w.V2 = c.take<uint16_t>(size_t(nc) * mp);
  if (count == 0) return w;
  w.parts = c.take<uint16_t>(size_t(n) * 3 * parts_rank(rank));
  const int shares = shrink_shares(n, m);
  w.sums = c.take<float>(shares > 1 ? size_t(shares) * n * rank : 0);
  w.At = c.take<uint16_t>(size_t(count) * d * rank);
  w.Bt = c.take<uint16_t>(size_t(count) * rank * mp);
  w.outer = c.take<float>(std::max(outer_floats(n, d, rank, count), outer_floats(n, m, rank, count)));
  return w;
}

}  // namespace

size_t lora_ws_bytes(int64_t n, int64_t m, int64_t d, int64_t group, int rank) {
  if (n == 0) return 0;
  Carver c(nullptr);
  carve_lora(c, n, m, d, group, rank);
  return c.bytes();
}

gptq_status launch_lora(const uint16_t* X, int64_t ldx, int64_t n, const Packed& w,
                        const gptq_adapters& ad, float* H, void* Y, int out_bf16, int64_t ldy,
                        void* ws, hipStream_t st) {
  Carver c(ws);
  const LoraWs b = carve_lora(c, n, w.m, w.d, w.group, ad.rank);
  if (decode_takes(n, w.ng))
    return launch_lora_decode(X, ldx, n, w, ad, H ? H : b.hidden, Y, out_bf16, ldy, st);
  const int lay = layout_of(w.group);
  const bool direct = as_is(X, ldx, w.d);
  const int rp = parts_rank(ad.rank);
  const int64_t ldp = round_up(w.d, 64);
  GemmArgs g{};
  g.m = w.m;
  g.M = b.M;
  g.L = static_cast<const uint16_t*>(ad.B);
  g.n_adapters = ad.n_adapters;
  g.rank = ad.rank;
  g.rp = rp;
  g.parts = b.parts;
  g.ldy = ldy;
  g.out_bf16 = out_bf16;
  g.mpad = round_up(w.m, 256) + 64;
  g.scale_t = b.scale_t;
  g.kwrap = int(ldp / 64);
  gptq_status s;
  if (lay == kByGroups) {
    g.plan = b.plan;
    g.ldm = g.ldv2 = plan_cols(w.d, w.ng, w.group);
    g.V2 = b.V2;
    if ((s = launch_plan(w, b.plan, st)) != GPTQ_OK) return s;
  } else if (lay == kByRow) {
    g.ldm = ldp;
    g.kblocks = g.kwrap;
    if ((s = launch_expand_row(w, b.M, ldp, b.scale_t, st)) != GPTQ_OK) return s;
  } else {
    g.ldm = 3 * ldp;
    g.kblocks = 3 * g.kwrap;
    if ((s = launch_expand_parts(w, b.M, ldp, st)) != GPTQ_OK) return s;
  }
  for (int64_t t0 = 0; t0 < n; t0 += kRowChunk) {
    const int64_t nc = std::min<int64_t>(kRowChunk, n - t0);
    const uint16_t* Xc = X + t0 * ldx;
    ShrinkArgs h{Xc, ldx, nc, w.d, static_cast<const uint16_t*>(ad.A), w.d, ad.row + t0,
                 ad.n_adapters, ad.rank, rp, ad.alpha, 0, H ? H + t0 * ad.rank : nullptr, b.parts,
                 b.sums};
    if ((s = launch_shrink(h, st)) != GPTQ_OK) return s;
    g.V = direct ? Xc : nullptr;
    g.ldv = ldx;
    if (lay == kByGroups) {
      if ((s = launch_layout(w, b.plan, t0 ? nullptr : b.M, g.ldm, b.scale_t, g.mpad, Xc, ldx, nc,
                             !direct, b.V2, g.ldv2, st)) != GPTQ_OK)
        return s;
    } else if (!direct) {
      if ((s = launch_pad_rows(Xc, ldx, nc, w.d, b.V2, ldp, st)) != GPTQ_OK) return s;
      g.V = b.V2;
      g.ldv = ldp;
    }
    g.n = nc;
    g.row = ad.row + t0;
    g.Y = out_bf16 ? static_cast<void*>(static_cast<uint16_t*>(Y) + t0 * ldy)
                   : static_cast<void*>(static_cast<float*>(Y) + t0 * ldy);
    if ((s = launch_gemm(g, lay == kByGroups ? fold_unit(w.group) : 0, st)) != GPTQ_OK) return s;
  }
  return GPTQ_OK;
}

size_t lora_backward_ws_bytes(int64_t n, int64_t m, int64_t d, int rank, int n_adapters) {
  if (n == 0) return 0;
  Carver c(nullptr);
  carve_back(c, n, m, d, rank, n_adapters);
  return c.bytes();
}

gptq_status launch_lora_backward(const uint16_t* dY, int64_t lddy, int64_t n, const uint16_t* X,
                                 int64_t ldx, const float* H, const Packed& w,
                                 const gptq_adapters* adp, uint16_t* dX, int64_t lddx, float* dA,
                                 float* dB, int accumulate, void* ws, hipStream_t st) {
  const gptq_adapters ad = adp ? *adp : gptq_adapters{};
  gptq_status s;
  if (n == 0) {
    if (accumulate || !adp || (!dA && !dB)) return GPTQ_OK;
    const int64_t na = int64_t(ad.n_adapters) * ad.rank * w.d, nb = int64_t(ad.n_adapters) * ad.rank * w.m;
    if (dA) zero_kernel<<<ceil_div(na, 256), 256, 0, st>>>(dA, na);
    if (dB) zero_kernel<<<ceil_div(nb, 256), 256, 0, st>>>(dB, nb);
    GPTQ_CHECK_LAUNCH();
    return GPTQ_OK;
  }
  Carver c(ws);
  const BackWs b = carve_back(c, n, w.m, w.d, ad.rank, ad.n_adapters);
  const int64_t mp = round_up(w.m, 64);
  const int rp = parts_rank(ad.rank);
  ShrinkArgs h{dY, lddy, n, w.m, b.Bt, mp, ad.row, ad.n_adapters, ad.rank, rp, ad.alpha, 1,
               nullptr, b.parts, b.sums};
  if (dB) {
    // alpha H as parts, then the sums over rows
    split_kernel<<<ceil_div(n * rp, 256), 256, 0, st>>>(h, H);
    GPTQ_CHECK_LAUNCH();
    OuterArgs o{dY, lddy, n, w.m, b.parts, ad.row, ad.rank, rp,
                outer_shares(n, w.m, ad.rank, ad.n_adapters), 1, accumulate, nullptr};
    if ((s = launch_outer(o, ad.n_adapters, b.outer, dB, st)) != GPTQ_OK) return s;
  }
  if (adp && (dX || dA)) {
    // G as parts (over those of H)
    turn_kernel<<<dim3(ceil_div(ad.rank, 64), ceil_div(mp, 64), ad.n_adapters), 256, 0, st>>>(
        static_cast<const uint16_t*>(ad.B), w.m, ad.rank, b.Bt, mp);
    GPTQ_CHECK_LAUNCH();
    if ((s = launch_shrink(h, st)) != GPTQ_OK) return s;
  }
  if (dA) {
    OuterArgs o{X, ldx, n, w.d, b.parts, ad.row, ad.rank, rp,
                outer_shares(n, w.d, ad.rank, ad.n_adapters), 0, accumulate, nullptr};
    if ((s = launch_outer(o, ad.n_adapters, b.outer, dA, st)) != GPTQ_OK) return s;
  }
  if (!dX) return GPTQ_OK;
  if (adp) {
    turn_kernel<<<dim3(ceil_div(w.d, 64), ceil_div(ad.rank, 64), ad.n_adapters), 256, 0, st>>>(
        static_cast<const uint16_t*>(ad.A), ad.rank, w.d, b.At, ad.rank);
    GPTQ_CHECK_LAUNCH();
  }
  if ((s = launch_expand_transposed(w, b.Wt, mp, st)) != GPTQ_OK) return s;
  const bool direct = as_is(dY, lddy, w.m);
  GemmArgs g{};
  g.m = w.d;
  g.M = b.Wt;
  g.ldm = mp;
  g.kblocks = g.kwrap = int(mp / 64);
  g.L = adp ? b.At : nullptr;
  g.n_adapters = ad.n_adapters;
  g.rank = ad.rank;
  g.rp = rp;
  g.ldy = lddx;
  g.out_bf16 = 1;
  for (int64_t t0 = 0; t0 < n; t0 += kRowChunk) {
    const int64_t nc = std::min<int64_t>(kRowChunk, n - t0);
    const uint16_t* Vc = dY + t0 * lddy;
    g.V = Vc;
    g.ldv = lddy;
    if (!direct) {
      if ((s = launch_pad_rows(Vc, lddy, nc, w.m, b.V2, mp, st)) != GPTQ_OK) return s;
      g.V = b.V2;
      g.ldv = mp;
    }
    g.n = nc;
    g.row = adp ? ad.row + t0 : nullptr;
    g.parts = adp ? b.parts + t0 * 3 * rp : nullptr;
    g.Y = dX + t0 * lddx;
    if ((s = launch_gemm(g, 0, st)) != GPTQ_OK) return s;
  }
  return GPTQ_OK;
}

}  // namespace gptq
