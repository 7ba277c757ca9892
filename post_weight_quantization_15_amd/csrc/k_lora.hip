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
// A workgroup owns 32 rows; its eight waves take every eighth 32-step of k
// (and grid.y a share of the steps where there are few rows), and their
// sums meet in LDS.  Rows are independent in the product, so a tile with
// several adapters runs once per adapter and keeps each adapter's rows.
// Read once per adapter of the tile: 32 rows of V from HBM, rank rows of
// M from L2.  Bound by memory: 8192 rows of 4096, rank 16, 32 us (2.1 TB/s);
// 16384 rows, rank 64, 72 us.
// ---------------------------------------------------------------------------
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
  size_t sums_floats;       // kept for them
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

template <int NF, int NW>
__global__ __launch_bounds__(NW * 64) void shrink_kernel(ShrinkArgs a, bool vec_v, bool vec_m) {
  __shared__ float red[NW][kShrinkRows][16 * NF + 4];
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
      for (; s < whole; s += NW) {
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
    for (; s < s1; s += NW) {
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
    for (int e = tid; e < kShrinkRows * a.rp; e += NW * 64) {
      const int tl = e / a.rp, p = e % a.rp;
      if (!((in >> tl) & 1u)) continue;
      const int64_t t = t0 + tl;
      float v = 0.0f;
      if (p < a.rank) {
#pragma unroll
        for (int w = 0; w < NW; ++w) v += red[w][tl][p];
      }
      if (gridDim.y > 1) {
        if (p < a.rank) a.sums[(int64_t(blockIdx.y) * a.n + t) * a.rank + p] = v;
      } else {
        put_hidden(a, t, p, v, a.alpha[ad]);
      }
    }
  }
  // rows without an adapter
  if (blockIdx.y == 0 && a.H)
    for (int e = tid; e < kShrinkRows * a.rank; e += NW * 64) {
      const int tl = e / a.rank;
      if (((none >> tl) & 1u) && t0 + tl < a.n) a.H[(t0 + tl) * a.rank + e % a.rank] = 0.0f;
    }
}

// Few values: one wave per value, fp32 sums of exact products in pairs.  Where a
// tile's rows have an adapter each, the tiles above would run once per row.
__global__ __launch_bounds__(256) void values_kernel(ShrinkArgs a, bool vec) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.y;
  const int p = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int id = a.row[t];
  const bool on = id >= 0 && id < a.n_adapters;
  float s = 0.0f;
  if (on && p < a.rank) {
    const uint16_t* v = a.V + t * a.ldv;
    const uint16_t* m = a.M + (int64_t(id) * a.rank + p) * a.ldm;
    s = dot_wave(v, m, a.len, vec, lane);
  }
  if (lane != 0) return;
  if (on) put_hidden(a, t, p, s, a.alpha[id]);
  else if (a.H && p < a.rank) a.H[t * a.rank + p] = 0.0f;
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

gptq_status launch_shrink(const ShrinkArgs& a, hipStream_t st) {
  const bool vv = a.ldv % 8 == 0 && reinterpret_cast<uintptr_t>(a.V) % 16 == 0;
  const bool vm = a.ldm % 8 == 0 && reinterpret_cast<uintptr_t>(a.M) % 16 == 0;
  // one wave a value (some 700 elements' time besides the sum's own) while that
  // takes no longer than the tiles' 12 us; elements loaded one by one take four
  // times as long: 4096 rows of 512, rank 16: 25 us and 7 by tiles; 203 rows of
  // 11008, rank 8: 12 us and 24
  if (a.n <= 65535 && a.n * a.rank * (a.len + 700) * (vv && vm ? 1 : 4) <= (int64_t(40) << 20)) {
    values_kernel<<<dim3(a.rp / 4, unsigned(a.n)), 256, 0, st>>>(a, vv && vm);
    GPTQ_CHECK_LAUNCH();
    return GPTQ_OK;
  }
  const int shares = shrink_shares(a.n, a.len, a.rank, a.sums_floats);
  const dim3 grid(ceil_div(a.n, kShrinkRows), shares);
  if (a.rank <= 16) shrink_kernel<1, 8><<<grid, 512, 0, st>>>(a, vv, vm);
  else if (a.rank <= 32) shrink_kernel<2, 8><<<grid, 512, 0, st>>>(a, vv, vm);
  else if (a.rank <= 64) shrink_kernel<4, 8><<<grid, 512, 0, st>>>(a, vv, vm);
  else shrink_kernel<8, 4><<<grid, 256, 0, st>>>(a, vv, vm);
  GPTQ_CHECK_LAUNCH();
  if (shares > 1) {
    shrink_sum_kernel<<<ceil_div(a.n * a.rp, 256), 256, 0, st>>>(a, shares);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
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

struct OuterSide {
  const uint16_t* V;         // NULL: not asked for
  int64_t ldv, len;
  const uint16_t* parts;     // [n][3 rp]
  int by_column;             // 1: out_a [len][rank] (dB), 0: [rank][len] (dA)
  int shares;
  float* sums;               // [a][share] where shares > 1
  float* out;
  int vec;
  unsigned blocks;
};
struct OuterArgs {           // both gradients in one launch, a range of blocks each
  OuterSide side[2];
  int64_t n;
  const int32_t* row;
  int rank, rp;
  int accumulate;
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
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs args) {
  constexpr int kRp = NF <= 2 ? 32 : 16 * NF;               // padded rank
  constexpr int kPartRow = kRp * 2 + 16;                    // bytes of a row of one part in LDS
  constexpr int kChunks = (3 * kRp / 8 + 7) / 8;            // 16-byte chunks of parts a thread moves
  __shared__ __attribute__((aligned(16))) char lv[32 * kOuterCols * 2];
  __shared__ __attribute__((aligned(16))) char lp[3][32 * kPartRow];
  __shared__ int32_t list[kOuterList];
  __shared__ int wcount[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int kg = lane >> 4, c16 = lane & 15;
  const unsigned block = flat_block();
  const bool second = block >= args.side[0].blocks;
  const OuterSide& a = args.side[second ? 1 : 0];
  const unsigned bx = block - (second ? args.side[0].blocks : 0);
  if (bx >= a.blocks) return;
  const unsigned tiles = static_cast<unsigned>((a.len + kOuterCols - 1) / kOuterCols);
  const int64_t c0 = int64_t(bx % tiles) * kOuterCols;
  const int share = bx / tiles % a.shares, ad = bx / tiles / a.shares;
  const int64_t r0 = args.n * share / a.shares, r1 = args.n * (share + 1) / a.shares;
  const bool vec_v = a.vec;
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
      const bool mine = e < piece && args.row[p0 + e] == ad;
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
    // ---- a step: thread t holds the two 16-byte chunks 2 (t % 8), + 1 of row t / 8
    //      of V and every eighth chunk of its parts, loaded a step ahead
    const int rl = tid >> 3;
    const bool fast = vec_v && c0 + kOuterCols <= a.len;
    u32x4 nv[2], np[kChunks];
    auto load_step = [&](int s) {
      const bool have = s + rl < count;
      const int64_t t = p0 + list[have ? s + rl : 0];
      const uint16_t* src = a.V + t * a.ldv + c0 + 16 * (tid & 7);
      if (fast) {
#pragma unroll
        for (int h = 0; h < 2; ++h) nv[h] = *reinterpret_cast<const u32x4*>(src + 8 * h);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          nv[h] = load8(a.V + t * a.ldv, c0 + 16 * (tid & 7) + 8 * h, a.len, vec_v);
      }
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int ch = min((tid & 7) + 8 * u, 3 * kRp / 8 - 1);
        np[u] = *reinterpret_cast<const u32x4*>(a.parts + t * 3 * args.rp + 8 * ch);
      }
      if (!have) {
        nv[0] = nv[1] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int u = 0; u < kChunks; ++u) np[u] = u32x4{0u, 0u, 0u, 0u};
      }
    };
    if (count) load_step(0);
    for (int s = 0; s < count; s += 32) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4*>(lv + rl * (kOuterCols * 2) + 16 * ((2 * (tid & 7) + h) ^ swz(rl))) = nv[h];
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int ch = (tid & 7) + 8 * u;
        if (ch < 3 * kRp / 8)
          *reinterpret_cast<u32x4*>(lp[ch / (kRp / 8)] + rl * kPartRow + 16 * (ch % (kRp / 8))) = np[u];
      }
      __syncthreads();
      if (s + 32 < count) load_step(s + 32);
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
  float* out = (a.shares > 1 ? a.sums : a.out) + (int64_t(ad) * a.shares + share) * args.rank * a.len;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int p = 16 * f + (a.by_column ? c16 : 4 * kg + v);
        const int64_t c = c0 + 32 * wv + 16 * j + (a.by_column ? 4 * kg + v : c16);
        if (p >= args.rank || c >= a.len) continue;
        float* o = out + (a.by_column ? c * args.rank + p : p * a.len + c);
        *o = args.accumulate && a.shares == 1 ? *o + acc[f][j][v] : acc[f][j][v];
      }
}

// The shares' sums in their order, four neighbouring values a thread (16-byte
// loads where a result's length is a multiple of four).
__global__ __launch_bounds__(256) void outer_sum_kernel(OuterArgs args, int count, unsigned blocks0) {
  const bool second = blockIdx.x >= blocks0;
  const OuterSide& a = args.side[second ? 1 : 0];
  const int64_t e = (int64_t(blockIdx.x - (second ? blocks0 : 0)) * 256 + threadIdx.x) * 4;
  const int64_t per = int64_t(args.rank) * a.len;
  if (e >= per * count) return;
  if (per % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0) {
    const float* s = a.sums + e / per * a.shares * per + e % per;
    f32x4 v = *reinterpret_cast<const f32x4*>(s);
#pragma unroll 8
    for (int i = 1; i < a.shares; ++i) v += *reinterpret_cast<const f32x4*>(s + i * per);
    f32x4* o = reinterpret_cast<f32x4*>(a.out + e);
    *o = args.accumulate ? *o + v : v;
    return;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (e + u >= per * count) break;
    const float* s = a.sums + (e + u) / per * a.shares * per + (e + u) % per;
    float v = s[0];
    for (int i = 1; i < a.shares; ++i) v += s[i * per];
    a.out[e + u] = args.accumulate ? a.out[e + u] + v : v;
  }
}

__global__ void zero_kernel(float* __restrict__ p, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
    p[i] = 0.0f;
}

// Shares of the rows per adapter: enough workgroups, more than 128 rows each,
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

gptq_status launch_outer(OuterArgs a, int count, hipStream_t st) {
  unsigned sum_blocks[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    OuterSide& o = a.side[i];
    o.blocks = 0;
    if (!o.out) continue;
    o.vec = o.ldv % 8 == 0 && reinterpret_cast<uintptr_t>(o.V) % 16 == 0;
    o.shares = outer_shares(a.n, o.len, a.rank, count);
    o.blocks = ceil_div(o.len, kOuterCols) * o.shares * count;
    if (o.shares > 1) sum_blocks[i] = ceil_div(int64_t(a.rank) * o.len * count, 1024);
  }
  if (!(a.side[0].blocks + a.side[1].blocks)) return GPTQ_OK;
  const dim3 grid = flat_grid(int64_t(a.side[0].blocks) + a.side[1].blocks);
  if (a.rank <= 16) outer_kernel<1><<<grid, 256, 0, st>>>(a);
  else if (a.rank <= 32) outer_kernel<2><<<grid, 256, 0, st>>>(a);
  else if (a.rank <= 64) outer_kernel<4><<<grid, 256, 0, st>>>(a);
  else outer_kernel<8><<<grid, 256, 0, st>>>(a);
  GPTQ_CHECK_LAUNCH();
  if (sum_blocks[0] + sum_blocks[1]) {
    outer_sum_kernel<<<sum_blocks[0] + sum_blocks[1], 256, 0, st>>>(a, count, sum_blocks[0]);
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
  size_t sums_floats;
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
  w.sums_floats = shrink_floats_chunked(n, d, rank);
  w.sums = c.take<float>(w.sums_floats);
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
  uint16_t* parts;   // of G
  uint16_t* hparts;  // of alpha H
  float* sums;
  size_t sums_floats;
  uint16_t* At;      // [count][d][rank]
  uint16_t* Bt;      // [count][rank][mp]
  uint16_t* Wt;      // [d][mp]
  uint16_t* V2;      // [rows][mp]
  float* outer[2];
};

BackWs carve_back(Carver& c, int64_t n, int64_t m, int64_t d, int rank, int count) {
  const int64_t nc = std::min<int64_t>(n, kRowChunk), mp = round_up(m, 64);
  BackWs w{};
  if (n == 0) return w;
  w.Wt = c.take<uint16_t>(size_t(d) * mp);
  w.V2 = c.take<uint16_t>(size_t(nc) * mp);
  if (count == 0) return w;
  w.parts = c.take<uint16_t>(size_t(n) * 3 * parts_rank(rank));
  w.hparts = c.take<uint16_t>(size_t(n) * 3 * parts_rank(rank));
  w.sums_floats = shrink_floats(n, m, rank);
  w.sums = c.take<float>(w.sums_floats);
  w.At = c.take<uint16_t>(size_t(count) * d * rank);
  w.Bt = c.take<uint16_t>(size_t(count) * rank * mp);
  w.outer[0] = c.take<float>(outer_floats(n, d, rank, count));
  w.outer[1] = c.take<float>(outer_floats(n, m, rank, count));
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
                 b.sums, b.sums_floats};
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
    auto blocks = [](int64_t v) { return unsigned(std::min<int64_t>((v + 255) / 256, 4096)); };
    if (dA) zero_kernel<<<blocks(na), 256, 0, st>>>(dA, na);
    if (dB) zero_kernel<<<blocks(nb), 256, 0, st>>>(dB, nb);
    GPTQ_CHECK_LAUNCH();
    return GPTQ_OK;
  }
  Carver c(ws);
  const BackWs b = carve_back(c, n, w.m, w.d, ad.rank, ad.n_adapters);
  const int64_t mp = round_up(w.m, 64);
  const int rp = parts_rank(ad.rank);
  const bool need_g = adp && (dX || dA);
  PrepareArgs pa{w, mp, dX ? b.Wt : nullptr, ad, rp, need_g ? b.Bt : nullptr,
                 adp && dX ? b.At : nullptr, H, n, dB ? b.hparts : nullptr};
  if ((s = launch_prepare(pa, st)) != GPTQ_OK) return s;
  if (need_g) {
    const ShrinkArgs h{dY, lddy, n, w.m, b.Bt, mp, ad.row, ad.n_adapters, ad.rank, rp, ad.alpha, 1,
                       nullptr, b.parts, b.sums, b.sums_floats};
    if ((s = launch_shrink(h, st)) != GPTQ_OK) return s;
  }
  if (dA || dB) {
    OuterArgs o{{OuterSide{X, ldx, w.d, b.parts, 0, 1, b.outer[0], dA, 0, 0},
                 OuterSide{dY, lddy, w.m, b.hparts, 1, 1, b.outer[1], dB, 0, 0}},
                n, ad.row, ad.rank, rp, accumulate};
    if ((s = launch_outer(o, ad.n_adapters, st)) != GPTQ_OK) return s;
  }
  if (!dX) return GPTQ_OK;
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
