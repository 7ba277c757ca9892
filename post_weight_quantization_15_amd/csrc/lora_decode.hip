// The adapter product for few activation rows (single tokens of up to 128
// requests): the packed weights are read once per 64 rows, straight into
// matrix-core operands, and nothing is laid out first.
//
// hidden_kernel: H[t][p] = X[t] . A_a[p], one wave per value (fp32, exact
//   bf16 products in pairs); the rows of A are the traffic.
// decode_kernel: a workgroup of 4 to 16 waves owns 16, 32 or 64 output rows;
//   the waves share the input dimension in chunks of 128 columns.  In a chunk lane
//   (j, q) loads the 32 codes of row j, columns 32 q .. 32 q + 31, in one
//   load (16 rows x 64 bytes at 4 bits), four register swaps turn them so that
//   the lane holds columns 32 s + 8 q .. + 7 of each 32-step s, and each
//   8-code run becomes a matrix operand in about ten instructions.
//
// A 32-step whose columns share one group enters as exact small numbers -- 16
// + k for 2 to 4 bits (the code in the mantissa under the exponent of 16), k
// for 8 -- and the group's grid comes out of the sums: acc += Delta (P - zz
// Xs) with Xs = sum x from one more product with ones and zz the zero point
// (plus 16).  A step that mixes groups (act-order, groups under 32) forms
// Delta (code - zero) per column in fp32 and multiplies its three bf16 parts.
// The grids of the rows lie in LDS for both.
//
// One token through 4096 x 4096 in 4 bits takes 11.0 us on the card (9.3 MB,
// bound by the chain load - product - sum of one workgroup and its launch), 16
// tokens through 11008 x 4096 20.0 us (33 MB with the adapters' factors, 1.7
// TB/s: bound by the activations' operands, which every workgroup reads from
// L2, and the loads' latency).  Beyond 128 rows, or 768 groups a row, the
// laid-out product takes over.
#include "lora.h"

namespace gptq {
namespace {

constexpr int kWideFrom = 400;             // workgroups of 16 rows from which 32 are taken
constexpr int kWiderFrom = 512;            // ... and 64, up to 32 activation rows
constexpr int kDecodeMaxGroups = 768;      // 96 KB of grids in LDS

// ---------------------------------------------------------------------------
struct HiddenArgs {
  const uint16_t* X;
  int64_t ldx, d;
  const uint16_t* A;
  const int32_t* row;
  int n_adapters, rank;
  float* H;
};

__global__ __launch_bounds__(256) void hidden_kernel(HiddenArgs a, bool vec_x, bool vec_a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.y;
  const int p = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (p >= a.rank) return;
  const int id = a.row[t];
  float s = 0.0f;
  if (id >= 0 && id < a.n_adapters) {
    const uint16_t* x = a.X + t * a.ldx;
    const uint16_t* w = a.A + (int64_t(id) * a.rank + p) * a.d;
    s = dot_wave(x, w, a.d, vec_x && vec_a, lane);
  }
  if (lane == 0) a.H[t * a.rank + p] = s;
}

// ---------------------------------------------------------------------------
struct DecodeArgs {
  const uint16_t* X;
  int64_t ldx, n;
  Packed w;
  int64_t words;
  float* H;
  const uint16_t* A;
  const uint16_t* B;
  const float* alpha;
  const int32_t* row;
  int n_adapters, rank;
  void* Y;
  int64_t ldy;
  int out_bf16, fused;
};

// Eight codes in nibbles as four bf16 pairs 16 + k, in order.
__device__ inline u32x4 nibbles_to_bf16(uint32_t w) {
  const uint32_t even = ((w << 3) & 0x78787878u) | 0x80808080u;
  const uint32_t odd = ((w >> 1) & 0x78787878u) | 0x80808080u;
  return u32x4{__builtin_amdgcn_perm(odd, even, 0x0C040C00u) | 0x41004100u,
               __builtin_amdgcn_perm(odd, even, 0x0C050C01u) | 0x41004100u,
               __builtin_amdgcn_perm(odd, even, 0x0C060C02u) | 0x41004100u,
               __builtin_amdgcn_perm(odd, even, 0x0C070C03u) | 0x41004100u};
}

template <int BITS>
struct Run {                               // the codes of an 8-column run
  uint32_t w[BITS == 8 ? 2 : 1];
};

// Run `s` of the 32 codes in w[0 .. BITS).
template <int BITS>
__device__ inline Run<BITS> run_of(const uint32_t* w, int s) {
  Run<BITS> r;
  if constexpr (BITS == 4) {
    r.w[0] = w[s];
  } else if constexpr (BITS == 2) {
    r.w[0] = (w[s >> 1] >> (16 * (s & 1))) & 0xFFFFu;
  } else if constexpr (BITS == 3) {
    const uint32_t v = s == 0 ? w[0] : s == 3 ? w[2] >> 8
                     : __builtin_amdgcn_alignbit(w[s], w[s - 1], s == 1 ? 24 : 16);
    r.w[0] = v & 0xFFFFFFu;
  } else {
    r.w[0] = w[2 * s];
    r.w[1] = w[2 * s + 1];
  }
  return r;
}

// Spreads 3- and 2-bit fields to nibbles (4: as they are).
template <int BITS>
__device__ inline uint32_t to_nibbles(uint32_t w) {
  if (BITS == 3) {
    uint32_t u = (w & 0xFFFu) | ((w & 0xFFF000u) << 4);
    u = (u & 0x003F003Fu) | ((u & 0x0FC00FC0u) << 2);
    return (u & 0x07070707u) | ((u & 0x38383838u) << 1);
  }
  if (BITS == 2) {
    uint32_t u = (w & 0xFFu) | ((w & 0xFF00u) << 8);
    u = (u & 0x000F000Fu) | ((u & 0x00F000F0u) << 4);
    return (u & 0x03030303u) | ((u & 0x0C0C0C0Cu) << 2);
  }
  return w;
}

// Unsigned code i of a run (signed codes arrive with their top bit flipped).
template <int BITS>
__device__ inline uint32_t run_code(const Run<BITS>& r, int i) {
  if (BITS == 8) return (r.w[(i >> 2) % (BITS == 8 ? 2 : 1)] >> (8 * (i & 3))) & 0xFFu;
  return (r.w[0] >> (BITS * i)) & ((1u << BITS) - 1u);
}

template <int BITS>
__device__ inline u32x4 run_operand(const Run<BITS>& r) {
  if constexpr (BITS == 8) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = r.w[i >> 1] >> (16 * (i & 1));
      o[i] = __builtin_amdgcn_perm(__float_as_uint(static_cast<float>((v >> 8) & 0xFFu)),
                                   __float_as_uint(static_cast<float>(v & 0xFFu)), 0x07060302u);
    }
    return o;
  } else {
    return nibbles_to_bf16(to_nibbles<BITS>(r.w[0]));
  }
}

// Every code's top bit, for the runs' word layouts.
template <int BITS>
constexpr uint32_t top_bits() {
  return BITS == 8 ? 0x80808080u : BITS == 4 ? 0x88888888u : BITS == 3 ? 0x00924924u : 0x0000AAAAu;
}

// Turns the 4 x 4 block that lanes q = 0 .. 3 (16 lanes each) hold in r[0 .. 3]:
// lane q's r[s] becomes lane s's r[q].
__device__ inline void turn4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  auto x = __builtin_amdgcn_permlane32_swap(a, c, false, false);
  auto y = __builtin_amdgcn_permlane32_swap(b, d, false, false);
  auto u = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
  auto v = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
  a = u[0];
  b = u[1];
  c = v[0];
  d = v[1];
}

// NJ x 16 output rows a workgroup (the activations' operands serve all of them),
// NW waves share the input dimension; grid.y: passes of 64 rows.  FUSED (one
// row): every workgroup forms the hidden values itself, from L2.
template <int BITS, int NT, int NW, int NJ>
__global__ __launch_bounds__(NW * 64, NT == 4 || NJ > 1 ? 2 : 4) void decode_kernel(DecodeArgs a, bool vec_x,
                                                                   bool vec_w, bool vec_a) {
  constexpr int kW = BITS == 8 ? 8 : BITS;      // words of 32 codes
  constexpr int kRows = NJ * 16;
  extern __shared__ __attribute__((aligned(16))) float grid[];   // [ng][kRows] (Delta, zz)
  __shared__ float red[NW][NT][16][17];
  __shared__ float hid[kMaxRank];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, c16 = lane & 15;
  const Packed& w = a.w;
  const int64_t tb = int64_t(blockIdx.y) * 64;
  const int64_t j0 = int64_t(blockIdx.x) * kRows;
  const int ng = static_cast<int>(w.ng);
  const int chunks = static_cast<int>((w.d + 127) / 128);
  const uint32_t* wrow[NJ];
#pragma unroll
  for (int f = 0; f < NJ; ++f) wrow[f] = w.qw + min<int64_t>(j0 + 16 * f + c16, w.m - 1) * a.words;

  // A chunk's codes, activations and group ids.  Chunks are loaded kAhead
  // ahead of their use; whole ones (of aligned rows) in wide loads without
  // a condition among them, the last one of the row piece by piece.
  // Activation rows past n read row n - 1: their sums are not stored.
  constexpr int kAhead = NT == 1 ? 2 : 1;
  uint32_t codes[kAhead][NJ][kW];
  u32x4 x[kAhead][NT][4];
  int ga[kAhead], gb[kAhead];              // group ids of columns 2 lane, 2 lane + 1
  const uint16_t* xr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xr[i] = a.X + min<int64_t>(tb + 16 * i + c16, a.n - 1) * a.ldx;
  const int whole = vec_x && vec_w ? static_cast<int>(w.d / 128) : 0;
  auto load_chunk = [&](int ch, uint32_t (*cv)[kW], u32x4 (*xv)[4], int& g0, int& g1) {
    const int64_t k0 = int64_t(ch) * 128;
    const int64_t at = int64_t(ch) * (4 * kW) + q * kW;     // first word of the lane's 32 codes
    if (ch < whole) {
#pragma unroll
      for (int f = 0; f < NJ; ++f) {
        const uint32_t* src = wrow[f] + at;
        if constexpr (BITS == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(src);
          cv[f][0] = u.x;
          cv[f][1] = u.y;
        } else if constexpr (BITS == 3) {
#pragma unroll
          for (int i = 0; i < 3; ++i) cv[f][i] = src[i];
        } else {
#pragma unroll
          for (int h = 0; h < kW / 4; ++h) {
            const u32x4 u = *reinterpret_cast<const u32x4*>(src + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) cv[f][4 * h + i] = u[i];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          xv[i][s] = *reinterpret_cast<const u32x4*>(xr[i] + k0 + 32 * s + 8 * q);
      g0 = w.g_idx[k0 + 2 * lane];
      g1 = w.g_idx[k0 + 2 * lane + 1];
    } else {
#pragma unroll
      for (int f = 0; f < NJ; ++f)
#pragma unroll
        for (int i = 0; i < kW; ++i) cv[f][i] = at + i < a.words ? wrow[f][at + i] : 0u;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) xv[i][s] = load8(xr[i], k0 + 32 * s + 8 * q, w.d, vec_x);
      g0 = w.g_idx[min<int64_t>(k0 + 2 * lane, w.d - 1)];
      g1 = w.g_idx[min<int64_t>(k0 + 2 * lane + 1, w.d - 1)];
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (wv + NW * u < chunks)
      load_chunk(wv + NW * u, codes[u], x[u], ga[u], gb[u]);

  if (NT == 1 && a.fused) {
    const int id = a.row[0];
    const bool some = id >= 0 && id < a.n_adapters;
    for (int p = wv; p < a.rank; p += NW) {
      float s = 0.0f;
      if (some) s = dot_wave(a.X, a.A + (int64_t(id) * a.rank + p) * w.d, w.d, vec_x && vec_a, lane);
      if (lane == 0) {
        hid[p] = s;
        if (a.H && blockIdx.x == 0) a.H[p] = s;
      }
    }
    __syncthreads();
  }
  // The adapter's part of the outputs this thread will write (element e: column
  // e % 16 of fragment e / (256 NT), row e / 16 % (16 NT)): its loads ride along with those above.
  constexpr int kOuts = (NT * NJ * 256 + NW * 64 - 1) / (NW * 64);
  float part_y[kOuts];
#pragma unroll
  for (int o = 0; o < kOuts; ++o) {
    const int e = tid + o * NW * 64;
    const int64_t t = tb + (e >> 4) % (16 * NT), j = j0 + 16 * (e / (256 * NT)) + (e & 15);
    part_y[o] = 0.0f;
    if (e >= NT * NJ * 256 || t >= a.n || j >= w.m) continue;
    const int id = a.row[t];
    if (id < 0 || id >= a.n_adapters) continue;
    const uint16_t* b = a.B + (int64_t(id) * w.m + j) * a.rank;
    const float* h = a.fused ? hid : a.H + t * a.rank;
    float s = 0.0f;
    int p = 0;
    if (a.rank % 8 == 0 && reinterpret_cast<uintptr_t>(a.B) % 16 == 0)
      for (; p < a.rank; p += 8) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(b + p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          s = fmaf(h[p + i], bf16_f32((v[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), s);
      }
    for (; p < a.rank; ++p) s = fmaf(h[p], bf16_f32(b[p]), s);
    part_y[o] = a.alpha[id] * s;
  }
  constexpr bool kMagic = BITS != 8;
  for (int e = tid; e < ng * kRows; e += NW * 64) {
    const int r = e / ng, g = e % ng;
    const int64_t at = min<int64_t>(j0 + r, w.m - 1) * ng + g;
    grid[(g * kRows + r) * 2] = step_at(w, at);
    grid[(g * kRows + r) * 2 + 1] =
        w.sgn ? static_cast<float>(1 << (BITS - 1)) : static_cast<float>(w.zeros[at]);
  }
  __syncthreads();

  f32x4 acc[NJ][NT];
#pragma unroll
  for (int f = 0; f < NJ; ++f)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  for (int cb = wv; cb < chunks; cb += NW * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int ch = cb + NW * u;
      if (ch >= chunks) break;
      const int64_t k0 = int64_t(ch) * 128;
      Run<BITS> run[NJ][4];
#pragma unroll
      for (int f = 0; f < NJ; ++f) {
#pragma unroll
        for (int s = 0; s < 4; ++s) run[f][s] = run_of<BITS>(codes[u][f], s);
#pragma unroll
        for (int h = 0; h < (BITS == 8 ? 2 : 1); ++h)
          turn4(run[f][0].w[h], run[f][1].w[h], run[f][2].w[h], run[f][3].w[h]);
        if (w.sgn) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int h = 0; h < (BITS == 8 ? 2 : 1); ++h) run[f][s].w[h] ^= top_bits<BITS>();
        }
      }
      // The chunk's groups: one, one per step, or steps that mix them.  Decided
      // once a chunk, so that its four steps' chains run side by side.
      // (Ids outside the row's groups count as the nearest; seen to here, not
      // at their load, which nothing waits for.)
      const int ia = min(max(ga[u], 0), ng - 1), ib = min(max(gb[u], 0), ng - 1);
      const int G0 = __builtin_amdgcn_readlane(ia, 0), G1 = __builtin_amdgcn_readlane(ia, 16),
                G2 = __builtin_amdgcn_readlane(ia, 32), G3 = __builtin_amdgcn_readlane(ia, 48);
      const int own = q == 0 ? G0 : q == 1 ? G1 : q == 2 ? G2 : G3;
      const uint64_t diff = __ballot(ia != own || ib != own);
      if (!diff && G0 == G1 && G1 == G2 && G2 == G3) {
        // sums of the activations: the same for every fragment of rows
        f32x4 Xs[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          Xs[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < 4; ++s) Xs[i] = mfma16(x[u][i][s], ones, Xs[i]);
        }
#pragma unroll
        for (int f = 0; f < NJ; ++f) {
          const float2 gr = *reinterpret_cast<const float2*>(&grid[(G0 * kRows + 16 * f + c16) * 2]);
          const float zz = gr.y + (kMagic ? 16.0f : 0.0f);
          u32x4 m[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) m[s] = run_operand<BITS>(run[f][s]);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            f32x4 P = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 4; ++s) P = mfma16(x[u][i][s], m[s], P);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              acc[f][i][v] = fmaf(gr.x, fmaf(-zz, Xs[i][v], P[v]), acc[f][i][v]);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if (k0 + 32 * s >= w.d) break;
          const int G = s == 0 ? G0 : s == 1 ? G1 : s == 2 ? G2 : G3;
          const f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
          if (!((diff >> (16 * s)) & 0xFFFFu)) {
            f32x4 Xs[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) Xs[i] = mfma16(x[u][i][s], ones, z);
#pragma unroll
            for (int f = 0; f < NJ; ++f) {
              const u32x4 m = run_operand<BITS>(run[f][s]);
              const float2 gr = *reinterpret_cast<const float2*>(&grid[(G * kRows + 16 * f + c16) * 2]);
              const float zz = gr.y + (kMagic ? 16.0f : 0.0f);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const f32x4 P = mfma16(x[u][i][s], m, z);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  acc[f][i][v] = fmaf(gr.x, fmaf(-zz, Xs[i][v], P[v]), acc[f][i][v]);
              }
            }
          } else {
            int g8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int src = 16 * s + 4 * q + (i >> 1);
              g8[i] = __shfl(i & 1 ? ib : ia, src);
            }
#pragma unroll
            for (int f = 0; f < NJ; ++f) {
              u32x4 part[3] = {};
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 gr =
                    *reinterpret_cast<const float2*>(&grid[(g8[i] * kRows + 16 * f + c16) * 2]);
                uint16_t p[3];
                split3(gr.x * (static_cast<float>(run_code<BITS>(run[f][s], i)) - gr.y), p);
#pragma unroll
                for (int h = 0; h < 3; ++h) part[h][i >> 1] |= uint32_t(p[h]) << (16 * (i & 1));
              }
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < 3; ++h) acc[f][i] = mfma16(x[u][i][s], part[h], acc[f][i]);
            }
          }
        }
      }
      const int next = ch + NW * kAhead;
      if (next < chunks) load_chunk(next, codes[u], x[u], ga[u], gb[u]);
    }
  }
  // ---- the waves' shares, in their order, and the adapter's part; one
  //      fragment of rows at a time
#pragma unroll
  for (int f = 0; f < NJ; ++f) {
    if (f) __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wv][i][4 * q + v][c16] = acc[f][i][v];
    __syncthreads();
#pragma unroll
    for (int o = 0; o < kOuts; ++o) {
      const int e = tid + o * NW * 64;
      if (e / (256 * NT) != f) continue;
      const int64_t t = tb + (e >> 4) % (16 * NT), j = j0 + 16 * f + (e & 15);
      if (t >= a.n || j >= w.m) continue;
      float y = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) y += red[v][(e >> 8) % NT][(e >> 4) & 15][e & 15];
      y += part_y[o];
      if (a.out_bf16) static_cast<uint16_t*>(a.Y)[t * a.ldy + j] = f32_bf16(y);
      else static_cast<float*>(a.Y)[t * a.ldy + j] = y;
    }
  }
}

template <int BITS, int NT, int NW, int NJ>
void launch_waves(const DecodeArgs& a, bool vx, bool vw, bool va, hipStream_t st) {
  const dim3 grid(ceil_div(a.w.m, 16 * NJ), ceil_div(a.n, 64));
  const size_t lds = size_t(a.w.ng) * NJ * 16 * 8;
  decode_kernel<BITS, NT, NW, NJ><<<grid, NW * 64, lds, st>>>(a, vx, vw, va);
}

// Workgroups and their waves: about 16 waves a CU, so that their loads keep
// memory busy.  The activations are read once a workgroup, and from some 9
// rows on that stream is the larger one, so where there are enough output rows
// a workgroup takes 64 of them (32 from 33 activation rows on, whose operands
// fill the registers): 14336 x 4096, 16 tokens 28.1 -> 22.5 us, 32 tokens 44.6
// -> 29.6; 28672 x 8192, 16 tokens 81 -> 54; 4096 x 4096, 128 tokens 48 -> 33.
// With fewer rows the registers cost more than it saves (14336 x 4096, 4
// tokens 20.4 by 16 output rows, 19.8 by 64; 11008 x 4096 16.7 and 19.4).
template <int BITS, int NT>
void launch_rows(const DecodeArgs& a, bool vx, bool vw, bool va, hipStream_t st) {
  const int64_t wgs = int64_t(ceil_div(a.w.m, 16)) * ceil_div(a.n, 64);
  const int64_t chunks = (a.w.d + 127) / 128;
  if constexpr (NT == 4) {
    if (wgs >= kWideFrom && a.w.ng <= kDecodeMaxGroups / 2) {
      if (chunks >= 8) return launch_waves<BITS, NT, 8, 2>(a, vx, vw, va, st);
      return launch_waves<BITS, NT, 4, 2>(a, vx, vw, va, st);
    }
  }
  if constexpr (NT <= 2 && BITS != 8)        // 8-bit codes' registers would spill
    if (a.n > 8 && wgs >= kWiderFrom && a.w.ng <= kDecodeMaxGroups / 4) {
      if (chunks >= 8 && wgs <= 1024) return launch_waves<BITS, NT, 8, 4>(a, vx, vw, va, st);
      return launch_waves<BITS, NT, 4, 4>(a, vx, vw, va, st);
    }
  if constexpr (NT < 4)
    if (wgs <= 256 && chunks >= 16) return launch_waves<BITS, NT, 16, 1>(a, vx, vw, va, st);
  if (wgs <= 512 && chunks >= 8) return launch_waves<BITS, NT, 8, 1>(a, vx, vw, va, st);
  launch_waves<BITS, NT, 4, 1>(a, vx, vw, va, st);
}

template <int BITS>
void launch_bits(const DecodeArgs& a, bool vx, bool vw, bool va, hipStream_t st) {
  if (a.n <= 16) launch_rows<BITS, 1>(a, vx, vw, va, st);
  else if (a.n <= 32) launch_rows<BITS, 2>(a, vx, vw, va, st);
  else launch_rows<BITS, 4>(a, vx, vw, va, st);
}

}  // namespace

bool decode_takes(int64_t n, int64_t ng) { return n <= kDecodeMaxRows && ng <= kDecodeMaxGroups; }

gptq_status launch_lora_decode(const uint16_t* X, int64_t ldx, int64_t n, const Packed& w,
                               const gptq_adapters& ad, float* H, void* Y, int out_bf16,
                               int64_t ldy, hipStream_t st) {
  const bool vx = ldx % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0;
  const bool va = w.d % 8 == 0 && reinterpret_cast<uintptr_t>(ad.A) % 16 == 0;
  // One row of a small adapter: a second launch costs more than forming the
  // hidden values in every workgroup, unless there are many (rank 16, 4096 x
  // 4096: 14.5 us and 15.8; 14336 x 4096: 24 and 17; 28672 x 8192: 79 and 50).
  const int fused = n == 1 && w.m <= 8192 && ad.rank * w.d <= (int64_t(1) << 17);
  if (!fused) {
    const HiddenArgs h{X, ldx, w.d, static_cast<const uint16_t*>(ad.A), ad.row, ad.n_adapters,
                       ad.rank, H};
    hidden_kernel<<<dim3(ceil_div(ad.rank, 4), unsigned(n)), 256, 0, st>>>(h, vx, va);
    GPTQ_CHECK_LAUNCH();
  }
  const int64_t words = (w.d * w.bits + 31) / 32;
  const int bytes = w.bits == 2 ? 8 : w.bits == 3 ? 4 : 16;
  const bool vw = words * 4 % bytes == 0 && reinterpret_cast<uintptr_t>(w.qw) % bytes == 0;
  const DecodeArgs a{X, ldx, n, w, words, H, static_cast<const uint16_t*>(ad.A),
                     static_cast<const uint16_t*>(ad.B), ad.alpha, ad.row, ad.n_adapters, ad.rank,
                     Y, ldy, out_bf16, fused};
  switch (w.bits) {
    case 2: launch_bits<2>(a, vx, vw, va, st); break;
    case 3: launch_bits<3>(a, vx, vw, va, st); break;
    case 4: launch_bits<4>(a, vx, vw, va, st); break;
    default: launch_bits<8>(a, vx, vw, va, st); break;
  }
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace gptq
