// The 4-bit floating-point products on matrix-core tiles, for many activation
// rows: both operands in 4 bits (scaled matrix instructions, a block's scale a
// lane), or bf16 activations against weights that leave LDS in 4 bits and
// become bf16, exactly, in registers on their way into the instruction.
#include <algorithm>

#include "mx.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------
// Layout, one launch: every operand's scale bytes as [block of 256 columns][row]
// [8], so that a tile's for one step are contiguous; and the activations in 4
// bits, rounded or copied, with zeros up to whole 256 columns.
// ---------------------------------------------------------------------------
struct LayArgs {
  MxInput x;
  Mx w, up;
  int64_t nbp;               // blocks of 32 padded to 8
  int64_t npad, mpad;        // rows of the scales' layout
  uint8_t* xcodes;           // [n][16 nbp], or NULL (bf16; codes used as they lie)
  uint8_t* xscale;           // [nbp / 8][npad][8], or NULL
  uint8_t* wscale;           // [nbp / 8][mpad][8], then the other layer's
  uint32_t runs;             // runs of 512 columns of a row
  unsigned blocks_x, blocks_xs, blocks_w;
  bool vec;
};

// Thread e: the eight scale bytes of one row and step; 127 (1) past the row's blocks.
__device__ inline void lay_scales(const uint8_t* __restrict__ scales, int64_t rows, int64_t nb,
                                  int64_t pad, int64_t steps, uint8_t* __restrict__ out, int64_t e) {
  const int64_t step = e / pad, row = e % pad;
  if (step >= steps || row >= rows) return;
  uint32_t v[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t b = 8 * step + i;
    v[i >> 2] |= (b < nb ? uint32_t(scales[row * nb + b]) : 127u) << (8 * (i & 3));
  }
  reinterpret_cast<uint2*>(out)[step * pad + row] = make_uint2(v[0], v[1]);
}

__global__ __launch_bounds__(256) void mx_lay_kernel(LayArgs a) {
  const int tid = threadIdx.x;
  unsigned b = blockIdx.x;
  if (b < a.blocks_x) {
    const int lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(b * 4 + (tid >> 6));
    const uint32_t row = wave / a.runs, run = wave % a.runs;
    if (row >= a.x.n) return;
    const int64_t c = int64_t(run) * 512 + 8 * lane, blk = c / kMxBlock;
    if (blk >= a.nbp) return;                // whole blocks leave
    uint32_t* out = reinterpret_cast<uint32_t*>(a.xcodes) + (row * a.nbp + blk) * 4 + (lane & 3);
    if (a.x.form == GPTQ_MX_CODES) {
      const uint32_t* in = static_cast<const uint32_t*>(a.x.X) + (row * a.w.nb + blk) * 4 + (lane & 3);
      *out = blk < a.w.nb ? *in : 0u;
      return;
    }
    const u32x4 v = load8(static_cast<const uint16_t*>(a.x.X) + row * a.x.ldx, c, a.x.d, a.vec);
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = mx_amax2(m, v[i]);
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2)));
    const uint32_t byte = mx_scale_byte(m << 16);
    *out = byte == 255u ? 0u : mx_round8(v, mx_scale_f32(byte));
    if ((lane & 3) == 0)
      a.xscale[((blk >> 3) * a.npad + row) * 8 + (blk & 7)] = static_cast<uint8_t>(byte);
    return;
  }
  b -= a.blocks_x;
  if (b < a.blocks_xs) {
    lay_scales(a.x.scales, a.x.n, a.w.nb, a.npad, a.nbp / 8, a.xscale, int64_t(b) * 256 + tid);
    return;
  }
  b -= a.blocks_xs;
  const bool second = b >= a.blocks_w;
  const Mx& w = second ? a.up : a.w;
  lay_scales(w.scales, w.rows, w.nb, a.mpad, a.nbp / 8,
             a.wscale + (second ? a.nbp * a.mpad : 0), int64_t(b - (second ? a.blocks_w : 0)) * 256 + tid);
}

// ---------------------------------------------------------------------------
// The product.  A workgroup of WM x WN waves owns TM activation rows x TN weight
// rows; k goes by in blocks of 128 bytes of an activation row (256 4-bit or 64
// bf16 values) through a ring of S stages in LDS, copied by global_load_lds (no
// registers), one barrier per block.  KS shares of k, each with its own waves
// and ring, where tiles are few and small.
// In LDS a row of 128 bytes has its eight 16-byte units at c ^ ((r / 2) % 8):
// copies (8 rows of 8 units) and fragment reads (16 rows, one unit each) pass
// without bank conflicts.  Lane 16 q + r reads unit 2 q + s of its row in half s of
// a block: 32 4-bit values, or 8 bf16 ones.  For bf16 a block of a weight
// row is 32 bytes, of which the lane takes bytes 8 q .. + 7 (values 16 q .. + 15, those
// of its activation units); rows with bit 3 set have their halves swapped, which
// spreads a read over the banks.  Weights are the matrix instruction's first
// operand: a lane then holds four consecutive columns of one activation row.
// GATED: 16 rows of the gate's layer and 16 of the other in turn, so that a lane
// holds both factors of a result.
// ---------------------------------------------------------------------------
struct GemmMx {
  const char* X;             // rows of ldx bytes: bf16, or padded codes
  int64_t ldx, n;
  const uint8_t* xs;         // scales' layout (4-bit)
  int64_t npad;
  const uint8_t* W[2];       // codes [m][16 nb]
  const uint8_t* ws;         // scales' layout, the second layer's behind
  int64_t mpad, m;
  int nb, kblocks;
  MxOutput y;
};

enum { kBf16 = 0, kFour = 1 };

__device__ inline uint32_t unit_at(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
}

template <int FORM, int TM, int TN, int WM, int WN, int KS, int S, bool GATED>
__global__ __launch_bounds__(WM* WN* KS * 64) void mx_gemm_kernel(GemmMx a, unsigned tiles_j,
                                                                  unsigned tiles, int vec_y) {
  constexpr int kWaves = WM * WN;                        // of one share of k
  constexpr int kFi = TM / WM / 16, kFj = TN / WN / 16;  // fragments of a wave
  constexpr int kWRow = FORM == kFour ? 128 : 32;        // bytes of a weight row and block
  constexpr int kLoadsX = TM / 8 / kWaves;               // copies of a wave and block
  constexpr int kLoadsW = FORM == kFour ? TN / 8 / kWaves : 1;
  constexpr int kLanesW = FORM == kFour ? 64 : TN * 2 / kWaves;
  constexpr int kSRows = FORM == kFour ? TM + TN : TN;   // rows with scales
  constexpr int kLanesS = kSRows / 2 / kWaves;
  static_assert(TM % (8 * kWaves) == 0 && kLanesS >= 1 && kLanesS <= 64 && kLanesW <= 64 &&
                (FORM != kFour || TN % (8 * kWaves) == 0), "copies divide evenly");
  static_assert(!GATED || (TN / WN) % 32 == 0, "a wave has both factors");
  constexpr int kCopies = kLoadsX + kLoadsW + 1;
  constexpr int kOffW = TM * 128, kOffS = kOffW + TN * kWRow;
  constexpr int kStage = kOffS + kSRows * 8;
  constexpr int kRing = S * kStage;
  extern __shared__ __attribute__((aligned(16))) char lds_all[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int kg = __builtin_amdgcn_readfirstlane((tid >> 6) / kWaves);
  const int wv = __builtin_amdgcn_readfirstlane((tid >> 6) % kWaves);
  char* lds = lds_all + kg * kRing;
  const int q = lane >> 4, c16 = lane & 15;
  // Each XCD (workgroups b, b + 8, ...) walks a contiguous range of tiles, in bands of
  // kBand activation tiles, so that its L2 takes in the fewest rows per step.
  constexpr unsigned kBand = 4;
  unsigned tile = blockIdx.x;
  const unsigned per = tiles / 8;
  if (tile < 8 * per) tile = (tile % 8) * per + tile / 8;
  const unsigned tiles_t = tiles / tiles_j, band = tile / (kBand * tiles_j);
  const unsigned high = min(kBand, tiles_t - band * kBand), rest = tile - band * kBand * tiles_j;
  const int64_t tb = int64_t(__builtin_amdgcn_readfirstlane(band * kBand + rest % high)) * TM;
  // first result column: a gated tile has TN / 2 of them
  const int64_t jb = int64_t(__builtin_amdgcn_readfirstlane(rest / high)) * (GATED ? TN / 2 : TN);
  const int wi = (wv % WM) * (TM / WM), wj = (wv / WM) * (TN / WN);

  // this share's blocks; all shares turn as often as the longest
  const int kb0 = a.kblocks * kg / KS, kb1 = a.kblocks * (kg + 1) / KS;
  const int turns = (a.kblocks + KS - 1) / KS;
  // tile row r of the weights: its layer and row
  auto w_layer = [&](int r) { return GATED ? (r >> 4) & 1 : 0; };
  auto w_row = [&](int r) { return GATED ? (r >> 5) * 16 + (r & 15) : r; };
  const int64_t ldw = int64_t(a.nb) * 16;
  const char* xbase = a.X + tb * a.ldx;
  uint32_t offx[kLoadsX];
#pragma unroll
  for (int i = 0; i < kLoadsX; ++i) {
    const int r = 8 * (kLoadsX * wv + i) + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    offx[i] = static_cast<uint32_t>((min<int64_t>(tb + r, a.n - 1) - tb) * a.ldx + 16 * c);
  }
  // weights: 4-bit as the activations; bf16: 32 rows of two units a copy
  const char* pw[kLoadsW];
  int cw[kLoadsW];                           // the lane's unit of a block
#pragma unroll
  for (int i = 0; i < kLoadsW; ++i) {
    const int r = FORM == kFour ? 8 * (kLoadsW * wv + i) + (lane >> 3)
                                : (kLanesW * wv + min(lane, kLanesW - 1)) >> 1;
    cw[i] = FORM == kFour ? (lane & 7) ^ ((r >> 1) & 7) : (lane & 1) ^ ((r >> 3) & 1);
    pw[i] = reinterpret_cast<const char*>(a.W[w_layer(r)]) + min<int64_t>(jb + w_row(r), a.m - 1) * ldw +
            16 * cw[i];
  }
  // scales: 16 bytes are two rows'
  const char* ps;
  int64_t step_s;
  {
    int r = 2 * (kLanesS * wv + min(lane, kLanesS - 1));
    if (FORM == kFour && r < TM) {
      ps = reinterpret_cast<const char*>(a.xs) + (tb + r) * 8;
      step_s = a.npad * 8;
    } else {
      if (FORM == kFour) r -= TM;
      step_s = a.mpad * 8;
      ps = reinterpret_cast<const char*>(a.ws) + (jb + w_row(r)) * 8 +
           (w_layer(r) ? step_s * ((a.nb + 7) / 8) : 0);
    }
  }
  // copies of block kb into its stage (past the end: the last block again, into a
  // stage nobody reads any more, so that every block counts alike)
  auto fetch = [&](int kb) {
    char* st = lds + (kb % S) * kStage;
    const int k = __builtin_amdgcn_readfirstlane(max(min(kb0 + kb, kb1 - 1), 0));
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i) {
      const char* base = xbase + int64_t(k) * 128;
      uint32_t o = offx[i];                  // opaque: a scalar base and a 32-bit offset
      asm volatile("" : "+s"(base), "+v"(o));
      __builtin_amdgcn_global_load_lds((gvoid)(base + o), (lvoid)(st + 8 * (kLoadsX * wv + i) * 128),
                                       16, 0, 0);
    }
    constexpr int kUnits = kWRow / 16;
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) {
      // units past the row's last: that one again (the activations are 0 there)
      const int over = max(kUnits * k + cw[i] - (a.nb - 1), 0);
      const char* p = pw[i] + int64_t(k) * kWRow - 16 * over;
      char* to = st + kOffW + (FORM == kFour ? 8 * (kLoadsW * wv + i) * 128 : kLanesW * wv * 16);
      if (kLanesW == 64 || lane < kLanesW)
        __builtin_amdgcn_global_load_lds((gvoid)p, (lvoid)to, 16, 0, 0);
    }
    const char* p = ps + (FORM == kFour ? k : k >> 2) * step_s;
    if (kLanesS == 64 || lane < kLanesS)
      __builtin_amdgcn_global_load_lds((gvoid)p, (lvoid)(st + kOffS + kLanesS * wv * 16), 16, 0, 0);
  };
  const uint32_t ox = unit_at(wi + c16, 2 * q);
  const uint32_t ow = kOffW + (FORM == kFour ? unit_at(wj + c16, 2 * q)
                                             : uint32_t((wj + c16) * 32 + ((8 * q) ^ ((c16 & 8) << 1))));
  const uint32_t osx = kOffS + (wi + c16) * 8 + 2 * q;
  const uint32_t osw = kOffS + ((FORM == kFour ? TM : 0) + wj + c16) * 8 + (FORM == kFour ? 2 * q : q >> 1);
  f32x4 acc[kFi][kFj];
#pragma unroll
  for (int i = 0; i < kFi; ++i)
#pragma unroll
    for (int j = 0; j < kFj; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  for (int kb = 0; kb < turns; ++kb) {
    wait_vmcnt<(S - 2) * kCopies>();
    // LDS reads of the stage that is filled next are done as well
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fetch(kb + S - 1);
    if (KS > 1 && kb >= kb1 - kb0) continue;
    const char* st = lds + (kb % S) * kStage;
    if constexpr (FORM == kFour) {
      uint32_t sx[kFi], sw[kFj];             // both halves' scales
#pragma unroll
      for (int i = 0; i < kFi; ++i) sx[i] = *reinterpret_cast<const uint16_t*>(st + osx + 128 * i);
#pragma unroll
      for (int j = 0; j < kFj; ++j) sw[j] = *reinterpret_cast<const uint16_t*>(st + osw + 128 * j);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        i32x8 fx[kFi], fw[kFj];
#pragma unroll
        for (int i = 0; i < kFi; ++i) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(st + (ox ^ (16 * s)) + 2048 * i);
          fx[i] = i32x8{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < kFj; ++j) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(st + (ow ^ (16 * s)) + 2048 * j);
          fw[j] = i32x8{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < kFj; ++j)
#pragma unroll
          for (int i = 0; i < kFi; ++i) {
            if (s == 0)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  fw[j], fx[i], acc[i][j], 4, 4, 0, int(sw[j]), 0, int(sx[i]));
            else
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  fw[j], fx[i], acc[i][j], 4, 4, 1, int(sw[j]), 1, int(sx[i]));
          }
      }
    } else {
      uint2 raw[kFj];
      float sc[kFj];
      const int sb = 2 * ((kb0 + kb) & 3);   // the block's place in its 256 columns
#pragma unroll
      for (int j = 0; j < kFj; ++j) {
        raw[j] = *reinterpret_cast<const uint2*>(st + ow + 512 * j);
        sc[j] = mx_scale_f32(*reinterpret_cast<const uint8_t*>(st + osw + sb + 128 * j));
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4 fx[kFi];
#pragma unroll
        for (int i = 0; i < kFi; ++i)
          fx[i] = *reinterpret_cast<const u32x4*>(st + (ox ^ (16 * s)) + 2048 * i);
#pragma unroll
        for (int j = 0; j < kFj; ++j) {
          const u32x4 fw = mx_expand8(s ? raw[j].y : raw[j].x, sc[j]);
#pragma unroll
          for (int i = 0; i < kFi; ++i) acc[i][j] = mfma16(fw, fx[i], acc[i][j]);
        }
      }
    }
  }
  wait_vmcnt<0>();

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
        for (int j = 0; j < kFj; ++j) acc[i][j] += sums[g * kAll + (i * kFj + j) * 64];
  }

  // ---- results, turned through LDS 16 rows at a time into whole lines
  constexpr int kCols = GATED ? TN / WN / 2 : TN / WN, kPitch = kCols + 4;
  constexpr int kTurn = KS > 1 ? (KS - 1) * kWaves * kFi * kFj * 1024 : 0;   // behind the sums
  static_assert(kTurn + kWaves * 16 * kPitch * 4 <= KS * kRing, "the turned rows fit the rings");
  if (KS == 1) __syncthreads();              // the last stage is read
  float* out = reinterpret_cast<float*>(lds_all + kTurn) + wv * (16 * kPitch);
  const int64_t r0 = jb + (GATED ? wj / 2 : wj);
  const bool wide = vec_y && r0 + kCols <= a.m;
  // 16 rows from t0 on, of which `value` gives the lane's four columns of fragment j
  auto store = [&](int64_t t0, void* Y, int64_t ldy, bool bf16, auto value) {
#pragma unroll
    for (int j = 0; j < kCols / 16; ++j)
      *reinterpret_cast<f32x4*>(out + c16 * kPitch + 16 * j + 4 * q) = value(j);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (wide && bf16) {
      constexpr int kPer = kCols / 8;        // lanes a row
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
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(Y) + (t0 + r) * ldy + r0 + c) = v;
      }
    } else if (wide) {
      constexpr int kPer = kCols / 4;
#pragma unroll
      for (int r = lane / kPer; r < 16; r += 64 / kPer) {
        const int c = 4 * (lane % kPer);
        const f32x4 v = *reinterpret_cast<const f32x4*>(out + r * kPitch + c);
        if (t0 + r < a.n)
          *reinterpret_cast<f32x4*>(static_cast<float*>(Y) + (t0 + r) * ldy + r0 + c) = v;
      }
    } else {
      const int c = lane % kCols;
      if (r0 + c < a.m)
        for (int r = lane / kCols; r < 16 && t0 + r < a.n; r += 64 / kCols) {
          const float v = out[r * kPitch + c];
          const int64_t at = (t0 + r) * ldy + r0 + c;
          if (bf16) static_cast<uint16_t*>(Y)[at] = f32_bf16(v);
          else static_cast<float*>(Y)[at] = v;
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next rows' writes
  };
#pragma unroll
  for (int i = 0; i < kFi; ++i) {
    int row = wi + 16 * i;                   // opaque: these rows' addresses only now
    asm volatile("" : "+s"(row));
    const int64_t t0 = tb + row;
    if constexpr (GATED) {
      store(t0, a.y.Y, a.y.ldy, true, [&](int j) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mx_act(acc[i][2 * j][e], a.y.act) * acc[i][2 * j + 1][e];
        return v;
      });
      if (a.y.G) {
        store(t0, a.y.G, a.y.ldg, true, [&](int j) { return acc[i][2 * j]; });
        store(t0, a.y.U, a.y.ldg, true, [&](int j) { return acc[i][2 * j + 1]; });
      }
    } else {
      store(t0, a.y.Y, a.y.ldy, a.y.out_bf16, [&](int j) { return acc[i][j]; });
    }
  }
}

template <int FORM, int TM, int TN, int WM, int WN, int KS, int S, bool GATED>
gptq_status launch_tile(const GemmMx& a, hipStream_t st) {
  constexpr int lds = KS * S * (TM * 128 + TN * (FORM == kFour ? 128 : 32) +
                                (FORM == kFour ? TM + TN : TN) * 8);
  static_assert(lds <= 160 * 1024, "the ring fits the LDS");
  const unsigned tj = ceil_div(a.m, GATED ? TN / 2 : TN);
  const unsigned tiles = tj * ceil_div(a.n, TM);
  auto lines = [](const void* p, int64_t bytes) {
    return bytes % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  const int vec_y = lines(a.y.Y, a.y.ldy * (a.y.out_bf16 ? 2 : 4)) &&
                    (!a.y.G || (lines(a.y.G, a.y.ldg * 2) && lines(a.y.U, a.y.ldg * 2)));
  mx_gemm_kernel<FORM, TM, TN, WM, WN, KS, S, GATED><<<tiles, WM * WN * KS * 64, lds, st>>>(a, tj, tiles, vec_y);
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

// Tiles by the time they take on 256 CUs: rounds of workgroups times a tile's
// area over the rate measured for its shape (relative).
template <int FORM, bool GATED>
gptq_status launch_form(const GemmMx& a, hipStream_t st) {
  const int64_t rows = GATED ? 2 * a.m : a.m;
  auto cost = [&](int tm, int tn, int per_cu, double rate) {
    const int64_t tiles = int64_t(ceil_div(a.n, tm)) * ceil_div(rows, tn);
    const int64_t rounds = (tiles + 256 * per_cu - 1) / (256 * per_cu);
    const int64_t left = tiles - (rounds - 1) * 256 * per_cu;
    return double((rounds - 1) * per_cu + (left + 255) / 256) * tm * tn / rate;
  };
  const double c256 = cost(256, 256, 1, 1.2), c128 = cost(128, 128, 1, 0.75), c64 = cost(64, 64, 2, 0.40);
  const double best = std::min(c256, std::min(c128, c64));
  constexpr int S = FORM == kFour ? 2 : 3;
  if (best == c256) return launch_tile<FORM, 256, 256, 2, 4, 1, S, GATED>(a, st);
  if (best == c128) return launch_tile<FORM, 128, 128, 2, 2, 2, 2, GATED>(a, st);
  return launch_tile<FORM, 64, 64, 2, 2, 4, 2, GATED>(a, st);
}

bool as_is(const void* X, int64_t ldx, int64_t d) {
  return ldx % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0 && d % 64 == 0 &&
         ldx < (int64_t(1) << 22);
}

struct GemmWs {
  uint8_t* xcodes;           // a chunk of rows
  uint8_t* xscale;
  uint8_t* wscale;
  uint16_t* V2;              // bf16 rows, padded
};

GemmWs carve(Carver& c, int64_t n, int64_t m, int64_t d, int form, bool gated) {
  const int64_t nc = std::min<int64_t>(n, kRowChunk), nbp = round_up(mx_blocks(d), 8);
  GemmWs w{};
  w.wscale = c.take<uint8_t>(size_t(gated ? 2 : 1) * nbp * round_up(m, 256));
  if (form == GPTQ_MX_BF16) {
    w.V2 = c.take<uint16_t>(size_t(nc) * round_up(d, 64));
  } else {
    w.xcodes = c.take<uint8_t>(size_t(nc) * nbp * 16);
    w.xscale = c.take<uint8_t>(size_t(nbp) * round_up(nc, 256));
  }
  return w;
}

}  // namespace

size_t mx_gemm_ws_bytes(int64_t n, int64_t m, int64_t d, int form, bool gated) {
  Carver c(nullptr);
  carve(c, n, m, d, form, gated);
  return c.bytes();
}

gptq_status launch_mx_gemm(const MxInput& x, const Mx& w, const Mx& up, const MxOutput& y, void* ws,
                           hipStream_t st) {
  const bool gated = up.codes;
  Carver c(ws);
  const GemmWs b = carve(c, x.n, w.rows, x.d, x.form, gated);
  const int64_t m = w.rows, nb = w.nb, nbp = round_up(nb, 8), mpad = round_up(m, 256);
  for (int64_t t0 = 0; t0 < x.n; t0 += kRowChunk) {
    const int64_t nc = std::min<int64_t>(kRowChunk, x.n - t0), npad = round_up(nc, 256);
    GemmMx g{};
    g.n = nc;
    g.W[0] = w.codes;
    g.W[1] = up.codes;
    g.ws = b.wscale;
    g.mpad = mpad;
    g.m = m;
    g.nb = int(nb);
    g.y = y;
    g.y.Y = static_cast<char*>(y.Y) + t0 * y.ldy * (y.out_bf16 ? 2 : 4);
    if (y.G) {
      g.y.G = y.G + t0 * y.ldg;
      g.y.U = y.U + t0 * y.ldg;
    }
    LayArgs l{x, w, up, nbp, npad, mpad, nullptr, nullptr, b.wscale, uint32_t((nbp + 15) / 16),
              0, 0, 0, false};
    l.x.n = nc;
    gptq_status s;
    if (x.form == GPTQ_MX_BF16) {
      const uint16_t* Xc = static_cast<const uint16_t*>(x.X) + t0 * x.ldx;
      g.X = reinterpret_cast<const char*>(Xc);
      g.ldx = x.ldx * 2;
      if (!as_is(Xc, x.ldx, x.d)) {
        const int64_t ldp = round_up(x.d, 64);
        if ((s = launch_pad_rows(Xc, x.ldx, nc, x.d, b.V2, ldp, st)) != GPTQ_OK) return s;
        g.X = reinterpret_cast<const char*>(b.V2);
        g.ldx = ldp * 2;
      }
      g.kblocks = int((x.d + 63) / 64);
    } else {
      g.xs = b.xscale;
      g.npad = npad;
      g.ldx = nbp * 16;
      g.kblocks = int(nbp / 8);
      l.xscale = b.xscale;
      g.X = reinterpret_cast<const char*>(b.xcodes);
      l.xcodes = b.xcodes;
      if (x.form == GPTQ_MX_CODES) {
        l.x.X = static_cast<const uint8_t*>(x.X) + t0 * nb * 16;
        l.x.scales = x.scales + t0 * nb;
        l.blocks_xs = ceil_div(npad * (nbp / 8), 256);
        if (nb == nbp) {                     // whole blocks: used as they lie
          g.X = static_cast<const char*>(l.x.X);
          l.xcodes = nullptr;
        }
      } else {
        l.x.X = static_cast<const uint16_t*>(x.X) + t0 * x.ldx;
        l.vec = x.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(l.x.X) % 16 == 0;
      }
      if (l.xcodes) l.blocks_x = ceil_div(nc * l.runs, 4);
    }
    if (t0 == 0) l.blocks_w = ceil_div(mpad * (nbp / 8), 256);
    const unsigned grid = l.blocks_x + l.blocks_xs + l.blocks_w * (gated ? 2 : 1);
    if (grid) {
      mx_lay_kernel<<<grid, 256, 0, st>>>(l);
      GPTQ_CHECK_LAUNCH();
    }
    if (x.form == GPTQ_MX_BF16)
      s = gated ? launch_form<kBf16, true>(g, st) : launch_form<kBf16, false>(g, st);
    else
      s = gated ? launch_form<kFour, true>(g, st) : launch_form<kFour, false>(g, st);
    if (s != GPTQ_OK) return s;
  }
  return GPTQ_OK;
}

}  // namespace gptq
