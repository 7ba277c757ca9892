// The 4-bit floating-point products on matrix-core tiles, for many activation
// rows: both operands in 4 bits (scaled matrix instructions, a block's scale a
// lane), or bf16 activations against weights that leave LDS in 4 bits and
// become bf16, exactly, in registers on their way into the instruction.
#include <algorithm>

#include "mx.h"

namespace gptq {
namespace {

// ---------------------------------------------------------------------------
// Layout, one launch: every operand's scale bytes as [step][row][kPer], kPer blocks of
// 32 columns a step, so that a tile's for one step are contiguous; and the
// activations in 4 bits, rounded or copied, with zeros up to whole steps.
// ---------------------------------------------------------------------------
constexpr int kPer = 8;
constexpr int kLayRows = 4;

struct LayArgs {
  MxInput x;
  Mx w, up;
  int64_t nbp;               // blocks of 32 padded to whole steps
  int64_t npad, mpad;        // rows of the scales' layout
  uint8_t* xcodes;           // [n][16 nbp], or NULL (bf16; codes used as they lie)
  uint8_t* xscale;           // [nbp / kPer][npad][kPer], or NULL
  uint8_t* wscale;           // [nbp / kPer][mpad][kPer], then the other layer's
  uint32_t runs;             // runs of 512 columns of a row
  unsigned blocks_x, blocks_xs, blocks_w;
  bool vec;
};

// Thread e: the scale bytes of one row and step; 127 (1) past the row's blocks.
__device__ inline void lay_scales(const uint8_t* __restrict__ scales, int64_t rows, int64_t nb,
                                  int64_t pad, int64_t steps, uint8_t* __restrict__ out, int64_t e) {
  const int64_t step = e / pad, row = e % pad;
  if (step >= steps || row >= rows) return;
  uint32_t v[kPer / 4] = {};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t b = kPer * step + i;
    v[i >> 2] |= (b < nb ? uint32_t(scales[row * nb + b]) : 127u) << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i)
    reinterpret_cast<uint32_t*>(out)[(step * pad + row) * (kPer / 4) + i] = v[i];
}

__global__ __launch_bounds__(256) void mx_lay_kernel(LayArgs a) {
  const int tid = threadIdx.x;
  unsigned b = blockIdx.x;
  if (b < a.blocks_x) {
    // a wave takes 512 columns of four rows, all loads first (8192 x 4096 in 25 us, 31 with a row
    // a wave); each of a block's four lanes writes one row's scale
    const int lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(b * 4 + (tid >> 6));
    const uint32_t row0 = wave / a.runs * kLayRows, run = wave % a.runs;
    const int64_t c = int64_t(run) * 512 + 8 * lane, blk = c / kMxBlock;
    if (row0 >= a.x.n || blk >= a.nbp) return;             // whole blocks leave
    uint32_t* out = reinterpret_cast<uint32_t*>(a.xcodes) + (row0 * a.nbp + blk) * 4 + (lane & 3);
    if (a.x.form == GPTQ_MX_CODES) {
      const uint32_t* in = static_cast<const uint32_t*>(a.x.X) + (row0 * a.w.nb + blk) * 4 + (lane & 3);
#pragma unroll
      for (int i = 0; i < kLayRows; ++i)
        if (row0 + i < a.x.n) out[i * a.nbp * 4] = blk < a.w.nb ? in[i * a.w.nb * 4] : 0u;
      return;
    }
    u32x4 v[kLayRows];
    uint32_t own = 0u;
    static_assert(kLayRows == kMxBlock / 8, "a row a lane of the block");
#pragma unroll
    for (int i = 0; i < kLayRows; ++i)
      v[i] = load8(static_cast<const uint16_t*>(a.x.X) + min<int64_t>(row0 + i, a.x.n - 1) * a.x.ldx, c,
                   a.x.d, a.vec);
#pragma unroll
    for (int i = 0; i < kLayRows; ++i) {
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = mx_amax2(m, v[i][e]);
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1)));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2)));
      const uint32_t byte = mx_scale_byte(m << 16);
      own = (lane & 3) == i ? byte : own;
      if (row0 + i < a.x.n)
        out[i * a.nbp * 4] = byte == 255u ? 0u : mx_round8(v[i], mx_scale_f32(byte));
    }
    const uint32_t row = row0 + (lane & 3);
    if (row < a.x.n) a.xscale[(blk / kPer * a.npad + row) * kPer + blk % kPer] = static_cast<uint8_t>(own);
    return;
  }
  b -= a.blocks_x;
  if (b < a.blocks_xs) {
    lay_scales(a.x.scales, a.x.n, a.w.nb, a.npad, a.nbp / kPer, a.xscale, int64_t(b) * 256 + tid);
    return;
  }
  b -= a.blocks_xs;
  const bool second = b >= a.blocks_w;
  const Mx& w = second ? a.up : a.w;
  lay_scales(w.scales, w.rows, w.nb, a.mpad, a.nbp / kPer,
             a.wscale + (second ? a.nbp * a.mpad : 0), int64_t(b - (second ? a.blocks_w : 0)) * 256 + tid);
}

// ---------------------------------------------------------------------------
// The product.  A workgroup of WM x WN waves owns TM activation rows x TN weight
// rows; k goes by in blocks of 128 bytes of an activation row (256 4-bit or 64 bf16
// values) through a ring of S stages in LDS, copied by global_load_lds (no
// registers), one barrier per block.  KS shares of k, each with its own waves and
// ring, where tiles are few and small; `splits` more by workgroups of their own, whose sums a
// second launch adds in their order.
//   kFour    both operands in 4 bits: a lane reads 16 bytes of each and a scale byte a
//            block, and the scaled matrix instruction takes them as they are
//   kBf16    bf16 activations; weights pass through LDS in 4 bits (a quarter of the
//            copies and reads) and become bf16, exactly, in registers
//   kDense   both operands bf16, for the gradient through a turned layer
// In LDS a row has its 16-byte units at c ^ unit_swap(r): copies and fragment reads (16
// rows, one unit each) pass without bank conflicts.  In half s of a block lane 16 q + r reads
// unit 2 q + s of its row with kFour (so that its two scale bytes are neighbours), unit q + 4 s
// otherwise.  With kBf16 a block of a weight row is 32 bytes, of which the lane takes word q + 4 s;
// rows with bit 3 set have their halves swapped, which spreads a read over the banks.  Weights
// are the matrix instruction's first operand: a lane then holds four consecutive columns of one
// activation row.
// GATED: 16 rows of the gate's layer and 16 of the other in turn, so that a lane
// holds both factors of a result.
//
// What bounds it.  kBf16: the matrix unit (8192 rows of 4096 into 11008: 600 us, 1230 TFLOP/s,
// four fifths of what a large library product in bf16 reaches on the card).  With three stages block kb
// + 1 has landed at the barrier of block kb, and a wave reads the operands of its next half block
// into the registers that the products of this one have freed, so no product waits behind a
// barrier for LDS; the conversions run beside the matrix unit.  kFour: LDS and the barrier: a
// block's products take a third of the bf16 ones' time and its reads as long as theirs (212 us on
// codes, 3480 TFLOP/s, where the instruction alone runs at 7700).  Two stages, as three do not fit beside
// tiles of 256 x 256; stages of half the length, of which three fit, were no faster with twice
// the barriers, and waves in two groups that take turns at LDS and the matrix unit were slower.
// ---------------------------------------------------------------------------
struct GemmMx {
  const char* X;             // rows of ldx bytes: bf16, or padded codes
  int64_t ldx, n;
  const uint8_t* xs;         // scales' layout (4-bit)
  int64_t npad;
  const uint8_t* W[2];       // codes [m][16 nb], or (kDense) bf16 rows of ldw bytes
  int64_t ldw;
  const uint8_t* S[2];       // their scales, as stored (s_rows) or in the layout
  int64_t mpad, m;
  int nb, kblocks, s_rows;
  // the sum over k in `splits` parts by workgroups of their own: fp32 [splits][n][ldp], the second
  // factor's columns from ldp / 2 on
  int splits;
  float* part;
  int64_t ldp;
  MxOutput y;
};

enum { kBf16 = 0, kFour = 1, kDense = 2 };

constexpr int kRow = 128;    // bytes of an activation row and block
// A 16-byte read passes in four parts of 16 lanes, of which the first takes
// rows 0 .. 3 and 12 .. 15 of one quarter of the wave with rows 4 .. 11 of the next.  Where the
// next quarter's unit differs in bit 0 any turn by row pairs will do; where it differs in bit 1
// (PAIR) row pairs 2 .. 5 have to lie in one half of the units, the others in the other one.
template <bool PAIR>
__device__ inline int unit_swap(int r) {
  const int p = (r >> 1) & 7;
  return PAIR ? (0x76321054 >> (4 * p)) & 7 : p;
}
template <bool PAIR>
__device__ inline uint32_t unit_at(int r, int c) {
  return static_cast<uint32_t>(r * kRow + ((c ^ unit_swap<PAIR>(r)) << 4));
}

template <int FORM, int TM, int TN, int WM, int WN, int KS, int S, bool GATED>
__global__ __launch_bounds__(WM* WN* KS * 64, TM * TN >= 128 * 128 ? 2 : 4) void mx_gemm_kernel(GemmMx a, unsigned tiles_j,
                                                                  unsigned tiles, int vec_y) {
  constexpr int kWaves = WM * WN;                        // of one share of k
  constexpr bool kPair = FORM == kFour;                  // a lane's units: 2 q + s, else q + 4 s
  constexpr int kFlip = kPair ? 16 : 64;                 // bytes that the other half's differ in
  constexpr int kFi = TM / WM / 16, kFj = TN / WN / 16;  // fragments of a wave
  constexpr int kWRow = FORM == kBf16 ? 32 : kRow;       // bytes of a weight row and block
  constexpr int kCopyRows = 1024 / kRow;                 // rows of a wave's copy
  constexpr int kLoadsX = TM / kCopyRows / kWaves;       // copies of a wave and block
  constexpr int kLanesX = TM * kRow / 16 / kWaves >= 64 ? 64 : TM * kRow / 16 / kWaves;
  constexpr int kUnitsW = TN * kWRow / 16 / kWaves;      // 16-byte units of a wave and block
  constexpr int kLoadsW = kUnitsW > 64 ? kUnitsW / 64 : 1, kLanesW = kUnitsW > 64 ? 64 : kUnitsW;
  constexpr int kSRows = FORM == kFour ? TM + TN : FORM == kBf16 ? TN : 0;   // rows with scales
  // copied 16 bytes a lane (two rows), bf16: 4 (half a row), which the stored scales' alignment allows
  constexpr int kBytesS = FORM == kFour ? 16 : 4;
  constexpr int kLanesS = kSRows * kPer / kBytesS / kWaves;
  static_assert(TM % (kCopyRows * kWaves) == 0 && kLanesX == 64 && kLanesS <= 64 &&
                    kUnitsW % kLanesW == 0 && kSRows * kPer % (kBytesS * kWaves) == 0,
                "copies divide evenly");
  static_assert(!GATED || (TN / WN) % 32 == 0, "a wave has both factors");
  // copies one at a time behind the products of the first half block (two waves a SIMD: 423 us
  // where all at once take 443, 8192 x 4096 -> 8192; smaller tiles need them earlier)
  constexpr bool kSpread = FORM == kBf16 && TM * TN == 256 * 256;
  constexpr bool kEarly = FORM == kBf16;                 // the next block has landed at a barrier, too
  static_assert(S >= (kEarly ? 3 : 2), "stages");
  constexpr int kCopies = kLoadsX + kLoadsW + (kSRows ? 1 : 0);
  constexpr int kOffW = TM * kRow, kOffS = kOffW + TN * kWRow;
  constexpr int kStage = kOffS + kSRows * kPer;
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
  const unsigned split = blockIdx.x / tiles;
  unsigned tile = blockIdx.x % tiles;
  const unsigned per = tiles / 8;
  if (tile < 8 * per) tile = (tile % 8) * per + tile / 8;
  const unsigned tiles_t = tiles / tiles_j, band = tile / (kBand * tiles_j);
  const unsigned high = min(kBand, tiles_t - band * kBand), rest = tile - band * kBand * tiles_j;
  const int64_t tb = int64_t(__builtin_amdgcn_readfirstlane(band * kBand + rest % high)) * TM;
  // first result column: a gated tile has TN / 2 of them
  const int64_t jb = int64_t(__builtin_amdgcn_readfirstlane(rest / high)) * (GATED ? TN / 2 : TN);
  const int wi = (wv % WM) * (TM / WM), wj = (wv / WM) * (TN / WN);

  // this share's blocks; all shares turn as often as the longest
  const int share = split * KS + kg, shares = a.splits * KS;
  const int kb0 = a.kblocks * share / shares, kb1 = a.kblocks * (share + 1) / shares;
  const int turns = (a.kblocks + shares - 1) / shares;
  // tile row r of the weights: its layer and row
  auto w_layer = [&](int r) { return GATED ? (r >> 4) & 1 : 0; };
  auto w_row = [&](int r) { return GATED ? (r >> 5) * 16 + (r & 15) : r; };
  const int64_t ldw = FORM == kDense ? a.ldw : int64_t(a.nb) * 16;
  const char* xbase = a.X + tb * a.ldx;
  uint32_t offx[kLoadsX];
#pragma unroll
  for (int i = 0; i < kLoadsX; ++i) {
    const int r = kCopyRows * (kLoadsX * wv + i) + lane / (kRow / 16);
    const int c = (lane % (kRow / 16)) ^ unit_swap<kPair>(r);
    offx[i] = static_cast<uint32_t>((min<int64_t>(tb + r, a.n - 1) - tb) * a.ldx + 16 * c);
  }
  // weights: units in the order of the stage.  4-bit: a copy's rows are of one layer; bf16: a
  // lane's own pointer
  constexpr int kUnits = kWRow / 16;
  const char* pw = nullptr;
  uint32_t offw[kLoadsW];
  // the lane's unit of a block in copy i
  auto unit_w = [&](int i) {
    const int u = kUnitsW * wv + 64 * i + min(lane, kLanesW - 1), r = u / kUnits;
    return (u % kUnits) ^ (FORM == kBf16 ? (r >> 3) & 1 : unit_swap<kPair>(r));
  };
#pragma unroll
  for (int i = 0; i < kLoadsW; ++i) {
    const int u = kUnitsW * wv + 64 * i + min(lane, kLanesW - 1), r = u / kUnits;
    offw[i] = static_cast<uint32_t>((min<int64_t>(jb + w_row(r), a.m - 1) - jb) * ldw + 16 * unit_w(i));
    if (FORM == kBf16) pw = reinterpret_cast<const char*>(a.W[w_layer(r)]) + jb * ldw + offw[i];
  }
  const char* wbase[2] = {reinterpret_cast<const char*>(a.W[0]) + jb * ldw,
                          reinterpret_cast<const char*>(a.W[1]) + jb * ldw};
  const char* ps = nullptr;
  int64_t step_s = 0;
  const int half_s = lane & 1;               // bf16: the lane's half of a row
  if (FORM != kDense) {
    const int u = kLanesS * wv + min(lane, kLanesS - 1);
    int r = FORM == kFour ? 2 * u : u >> 1;
    if (FORM == kFour && r < TM) {
      ps = reinterpret_cast<const char*>(a.xs) + (tb + r) * kPer;
      step_s = a.npad * kPer;
    } else {
      if (FORM == kFour) r -= TM;
      const int64_t row = jb + w_row(r);
      if (a.s_rows) {                        // as stored
        ps = reinterpret_cast<const char*>(a.S[w_layer(r)]) + min<int64_t>(row, a.m - 1) * a.nb;
        step_s = kPer;
      } else {
        ps = reinterpret_cast<const char*>(a.S[w_layer(r)]) + row * kPer;
        step_s = a.mpad * kPer;
      }
      if (FORM == kBf16) ps += 4 * half_s;
    }
  }
  // copy p (of kCopies) of block kb into its stage (past the end: of the last block again,
  // into a stage nobody reads any more, so that every block counts alike)
  auto copy = [&](int kb, int p) {
    char* st = lds + (kb % S) * kStage;
    const int k = __builtin_amdgcn_readfirstlane(max(min(kb0 + kb, kb1 - 1), 0));
    if (p < kLoadsX) {
      const int i = p;
      const char* base = xbase + int64_t(k) * kRow;
      uint32_t o = offx[i];                  // opaque: a scalar base and a 32-bit offset
      asm volatile("" : "+s"(base), "+v"(o));
      __builtin_amdgcn_global_load_lds((gvoid)(base + o), (lvoid)(st + 1024 * (kLoadsX * wv + i)),
                                       16, 0, 0);
    } else if (p < kLoadsX + kLoadsW) {
      const int i = p - kLoadsX;
      // units past the row's last: that one again (the activations are 0 there)
      int over = 0;
      if (FORM != kDense && kUnits * (k + 1) > a.nb) over = 16 * max(kUnits * k + unit_w(i) - (a.nb - 1), 0);
      const char* from;
      if (FORM != kBf16) {
        const char* base = wbase[w_layer((kUnitsW * wv + 64 * i) / kUnits)] + int64_t(k) * kWRow;
        uint32_t o = offw[i] - over;
        asm volatile("" : "+s"(base), "+v"(o));
        from = base + o;
      } else {
        from = pw + (k * kWRow - over);
      }
      if (kLanesW == 64 || lane < kLanesW)
        __builtin_amdgcn_global_load_lds((gvoid)from, (lvoid)(st + kOffW + 16 * (kUnitsW * wv + 64 * i)),
                                         16, 0, 0);
    } else if (FORM != kDense) {
      const int step = FORM == kFour ? k : k >> 2;
      const char* from = ps + step * step_s;
      // past the stored row's last four: those again (the activations are 0 there)
      if (FORM == kBf16 && a.s_rows && kPer * (step + 1) > a.nb && half_s) from -= 4;
      char* to = st + kOffS + kLanesS * wv * kBytesS;
      if (kLanesS == 64 || lane < kLanesS) {
        if constexpr (FORM == kFour) __builtin_amdgcn_global_load_lds((gvoid)from, (lvoid)to, 16, 0, 0);
        else __builtin_amdgcn_global_load_lds((gvoid)from, (lvoid)to, 4, 0, 0);
      }
    }
  };
  auto fetch = [&](int kb) {
#pragma unroll
    for (int p = 0; p < kCopies; ++p) copy(kb, p);
  };
  const uint32_t ox = unit_at<kPair>(wi + c16, kPair ? 2 * q : q);
  const uint32_t ow = kOffW + (FORM == kBf16 ? uint32_t((wj + c16) * 32 + 4 * q + ((c16 & 8) << 1))
                                             : unit_at<kPair>(wj + c16, kPair ? 2 * q : q));
  const uint32_t osx = kOffS + (wi + c16) * kPer + 2 * q;  // both halves' scales
  const uint32_t osw = kOffS + ((FORM == kFour ? TM : 0) + wj + c16) * kPer + (FORM == kFour ? 2 * q : 0);
  f32x4 acc[kFi][kFj];
#pragma unroll
  for (int i = 0; i < kFi; ++i)
#pragma unroll
    for (int j = 0; j < kFj; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the operands in work, and the weights of the step behind it
  u32x4 fx[kFi], fw[kFj], nw[kFj];
  uint32_t sx[kFi], sw[kFj], tw[kFj];        // 4-bit: scales
  auto read_x = [&](int kb, int s, int i) {
    const char* st = lds + (kb % S) * kStage;
    fx[i] = *reinterpret_cast<const u32x4*>(st + (ox ^ (kFlip * s)) + 16 * kRow * i);
    if (FORM == kFour && s == 0) sx[i] = *reinterpret_cast<const uint16_t*>(st + osx + 16 * kPer * i);
  };
  uint32_t raw[kFj];                         // bf16: the next step's weights as stored, and scales
  auto read_w = [&](int kb, int s) {
    const char* st = lds + (kb % S) * kStage;
#pragma unroll
    for (int j = 0; j < kFj; ++j) {
      if (FORM != kBf16) {
        nw[j] = *reinterpret_cast<const u32x4*>(st + (ow ^ (kFlip * s)) + 16 * kRow * j);
        if (FORM == kFour && s == 0) tw[j] = *reinterpret_cast<const uint16_t*>(st + osw + 16 * kPer * j);
      } else {
        raw[j] = *reinterpret_cast<const uint32_t*>(st + (ow ^ (16 * s)) + 512 * j);
        // the block's place in its 256 columns
        tw[j] = *reinterpret_cast<const uint8_t*>(st + osw + 2 * ((kb0 + kb) & 3) + s + 128 * j);
      }
    }
  };
  auto expand_w = [&](int j) {
    if (FORM == kBf16) nw[j] = mx_expand8(raw[j], mx_scale_f32(tw[j]));
  };
  auto next_w = [&]() {
#pragma unroll
    for (int j = 0; j < kFj; ++j) {
      fw[j] = nw[j];
      if (FORM == kFour) sw[j] = tw[j];
    }
  };
  auto read_first = [&](int kb) {
    read_w(kb, 0);
#pragma unroll
    for (int i = 0; i < kFi; ++i) read_x(kb, 0, i);
#pragma unroll
    for (int j = 0; j < kFj; ++j) expand_w(j);
    next_w();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  if (kEarly) {
    wait_vmcnt<(S - 2) * kCopies>();
    asm volatile("s_barrier" ::: "memory");
    read_first(0);
  }
  for (int kb = 0; kb < turns; ++kb) {
    // block kb (kEarly: kb + 1) has landed for all; the stage of block kb - 1 is read (its last
    // reads were waited for before their products)
    wait_vmcnt<(kEarly ? S - 3 : 0) * kCopies>();
    asm volatile("s_barrier" ::: "memory");
    const bool done = kb >= kb1 - kb0;
    if (done) {
      fetch(kb + S - 1);
      continue;
    }
    if (!kSpread) fetch(kb + S - 1);
    if constexpr (kEarly) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int kn = s ? kb + 1 : kb, sn = 1 - s;
        read_w(kn, sn);
        // in this order: left to itself the compiler puts the reads right before their use
#pragma unroll
        for (int i = 0; i < kFi; ++i) {
#pragma unroll
          for (int j = 0; j < kFj; ++j)
            if (i == (kFi > 1 ? 1 + j * (kFi - 1) / kFj : 0)) expand_w(j);
#pragma unroll
          for (int j = 0; j < kFj; ++j) acc[i][j] = mfma16(fw[j], fx[i], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
          read_x(kn, sn, i);
          if (kSpread && s == 0) {
#pragma unroll
            for (int p = 0; p < kCopies; ++p)
              if (p * kFi / kCopies == i) copy(kb + S - 1, p);
          }
        }
        next_w();
      }
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        read_w(kb, s);
        next_w();
#pragma unroll
        for (int i = 0; i < kFi; ++i) read_x(kb, s, i);
#pragma unroll
        for (int j = 0; j < kFj; ++j)
#pragma unroll
          for (int i = 0; i < kFi; ++i) {
            if (FORM != kFour) acc[i][j] = mfma16(fw[j], fx[i], acc[i][j]);
            else if (s == 0) acc[i][j] = mx_mfma<0>(fw[j], sw[j], fx[i], sx[i], acc[i][j]);
            else acc[i][j] = mx_mfma<1>(fw[j], sw[j], fx[i], sx[i], acc[i][j]);
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
    if (a.part) {
      float* part = a.part + split * a.n * a.ldp;
      store(t0, part, a.ldp, false, [&](int j) { return acc[i][GATED ? 2 * j : j]; });
      if constexpr (GATED)
        store(t0, part + a.ldp / 2, a.ldp, false, [&](int j) { return acc[i][2 * j + 1]; });
      continue;
    }
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

// The parts of a sum added in their order, and what is made of them: four columns a thread.
// (A row's columns in blockIdx.x, rows in blockIdx.y: at most kRowChunk.)
__global__ __launch_bounds__(256) void mx_join_kernel(GemmMx a, int vec_y) {
  const int64_t t = blockIdx.y;
  const int64_t c = 4 * (int64_t(blockIdx.x) * 256 + threadIdx.x);
  if (c >= a.m) return;
  const bool gated = a.W[1];
  const float* p = a.part + t * a.ldp + c;
  f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f}, u = v;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    v += *reinterpret_cast<const f32x4*>(p + s * a.n * a.ldp);
    if (gated) u += *reinterpret_cast<const f32x4*>(p + s * a.n * a.ldp + a.ldp / 2);
  }
  auto bf16 = [&](void* Y, int64_t ld, const f32x4& x) {
    uint16_t* y = static_cast<uint16_t*>(Y) + t * ld + c;
    if (vec_y && c + 4 <= a.m) {
      *reinterpret_cast<uint2*>(y) =
          make_uint2(uint32_t(f32_bf16(x[0])) | uint32_t(f32_bf16(x[1])) << 16,
                     uint32_t(f32_bf16(x[2])) | uint32_t(f32_bf16(x[3])) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < a.m) y[i] = f32_bf16(x[i]);
    }
  };
  if (gated) {
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mx_act(v[i], a.y.act) * u[i];
    bf16(a.y.Y, a.y.ldy, y);
    if (a.y.G) {
      bf16(a.y.G, a.y.ldg, v);
      bf16(a.y.U, a.y.ldg, u);
    }
  } else if (a.y.out_bf16) {
    bf16(a.y.Y, a.y.ldy, v);
  } else {
    float* y = static_cast<float*>(a.y.Y) + t * a.y.ldy + c;
    if (vec_y && c + 4 <= a.m) {
      *reinterpret_cast<f32x4*>(y) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < a.m) y[i] = v[i];
    }
  }
}

template <int FORM, int TM, int TN, int WM, int WN, int KS, int S, bool GATED>
gptq_status launch_tile(GemmMx a, int splits, hipStream_t st) {
  constexpr int lds = KS * S * (FORM == kFour   ? (TM + TN) * (kRow + kPer)
                                : FORM == kBf16 ? TM * kRow + TN * (32 + kPer)
                                                : (TM + TN) * kRow);
  static_assert(lds <= 160 * 1024, "the ring fits the LDS");
  const unsigned tj = ceil_div(a.m, GATED ? TN / 2 : TN);
  const unsigned tiles = tj * ceil_div(a.n, TM);
  auto lines = [](const void* p, int64_t bytes) {
    return bytes % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  const int vec_y = lines(a.y.Y, a.y.ldy * (a.y.out_bf16 ? 2 : 4)) &&
                    (!a.y.G || (lines(a.y.G, a.y.ldg * 2) && lines(a.y.U, a.y.ldg * 2)));
  a.splits = splits;
  if (splits == 1) a.part = nullptr;
  mx_gemm_kernel<FORM, TM, TN, WM, WN, KS, S, GATED>
      <<<tiles * splits, WM * WN * KS * 64, lds, st>>>(a, tj, tiles, a.part ? 1 : vec_y);
  GPTQ_CHECK_LAUNCH();
  if (splits > 1) {
    mx_join_kernel<<<dim3(ceil_div(a.m, 1024), unsigned(a.n)), 256, 0, st>>>(a, vec_y);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

// Tile and parts of the sum by the time they take (us): a CU's workgroups, at most `resident` at a
// time, turn once per block of k and share, in turn[c - 1] where c of them are there (measured for
// each form and tile, with products whose tiles fill the card evenly); parts of the sum cost
// their bytes, written and read at 4 TB/s, and a second launch.  Bf16 rows of 4096 into 4096, us:
//   100 rows   21 in 64 x 64 with 4 shares and 2 parts (24 without parts), 24 in 128 x 128 with 4
//              parts, 32 in 256 x 256 with 8
//   1024 rows  49 in 128 x 128 with 2 shares, 53 with one, 57 in 256 x 256 with 4 parts, 69 in 64 x 64
//   8192 rows  227 in 256 x 256, 289 in 128 x 128, 467 in 64 x 64
struct Shape {
  int tm, tn, ks, resident;
  double turn[4];
};
constexpr int kTiles = 5;
constexpr Shape kShapes[3][kTiles] = {{{256, 256, 1, 1, {1.52}},
                                       {128, 128, 2, 1, {1.13}},
                                       {128, 128, 1, 2, {0.66, 1.08}},
                                       {64, 64, 4, 1, {1.05}},
                                       {64, 64, 1, 4, {0.42, 0.57, 0.73, 0.92}}},
                                      {{256, 256, 1, 1, {1.8}},
                                       {128, 128, 2, 1, {1.4}},
                                       {128, 128, 1, 2, {0.9, 1.3}},
                                       {64, 64, 4, 1, {1.3}},
                                       {64, 64, 1, 4, {0.57, 0.69, 0.88, 1.08}}},
                                      {{256, 256, 1, 1, {1.5}},
                                       {128, 128, 2, 1, {1.25}},
                                       {128, 128, 1, 2, {0.75, 1.1}},
                                       {64, 64, 4, 1, {1.2}},
                                       {64, 64, 1, 4, {0.5, 0.6, 0.8, 1.0}}}};
constexpr int kMaxSplits = 16;
constexpr int64_t kPartFloats = int64_t(16) << 20;       // of all parts

inline double time_of(const Shape& s, int64_t n, int64_t rows, int64_t kblocks, int splits) {
  const int64_t wgs = int64_t(ceil_div(n, s.tm)) * ceil_div(rows, s.tn) * splits;
  const double turns = double(ceil_div(kblocks, s.ks * splits)) + 2.0;
  const int64_t most = (wgs + 255) / 256;    // of the fullest CU
  const int64_t last = most % s.resident;
  double time = turns * double(most / s.resident) * s.turn[s.resident - 1];
  if (last) time += turns * s.turn[last - 1];
  if (splits > 1) time += 3.0 + double(splits) * double(n * rows) * 8.0 / 4e6;
  return time;
}

struct Choice {
  int tile, splits;
  double time;
};
inline Choice choose(int form, int64_t n, int64_t m, int64_t kblocks, bool gated) {
  const int64_t rows = (gated ? 2 : 1) * round_up(m, 4);
  const int64_t most = std::min<int64_t>(kMaxSplits, kPartFloats / (n * rows));
  Choice c{0, 1, 1e30};
  for (int i = 0; i < kTiles; ++i)
    for (int p = 1; p == 1 || (p <= most && p * kShapes[form][i].ks * 2 <= kblocks); ++p) {
      const double t = time_of(kShapes[form][i], n, rows, kblocks, p);
      if (t < c.time) c = Choice{i, p, t};
    }
  return c;
}

template <int FORM, bool GATED>
gptq_status launch_form(const GemmMx& a, hipStream_t st) {
  const Choice c = choose(FORM, a.n, a.m, a.kblocks, GATED);
  constexpr int S = FORM == kBf16 ? 3 : 2;
  switch (c.tile) {
    case 0: return launch_tile<FORM, 256, 256, 2, 4, 1, S, GATED>(a, c.splits, st);
    case 1: return launch_tile<FORM, 128, 128, 2, 2, 2, S, GATED>(a, c.splits, st);
    case 2: return launch_tile<FORM, 128, 128, 2, 2, 1, S, GATED>(a, c.splits, st);
    case 3: return launch_tile<FORM, 64, 64, 2, 2, 4, S, GATED>(a, c.splits, st);
    default: return launch_tile<FORM, 64, 64, 2, 2, 1, S, GATED>(a, c.splits, st);
  }
}

bool as_is(const void* X, int64_t ldx, int64_t d) {
  return ldx % 8 == 0 && reinterpret_cast<uintptr_t>(X) % 16 == 0 && d % 64 == 0 &&
         ldx < (int64_t(1) << 22);
}

// Scales that 4-byte copies can take as they are stored.
bool stored_scales(const Mx& w) {
  return w.nb % 4 == 0 && reinterpret_cast<uintptr_t>(w.scales) % 4 == 0;
}

struct GemmWs {
  float* part;               // of the sums over k
  uint8_t* xcodes;           // a chunk of rows
  uint8_t* xscale;
  uint8_t* wscale;
  uint16_t* V2;              // bf16 rows, padded
};

GemmWs carve(Carver& c, int64_t n, int64_t m, int64_t d, int form, bool gated) {
  const int64_t nc = std::min<int64_t>(n, kRowChunk), nbp = round_up(mx_blocks(d), kPer);
  GemmWs w{};
  // a last, shorter chunk of rows may want more parts than a whole one
  size_t floats = 0;
  for (int64_t rows : {nc, n % kRowChunk}) {
    if (rows == 0) continue;
    const bool four = form != GPTQ_MX_BF16;
    const int64_t kblocks = four ? nbp / kPer : (d + 63) / 64;
    const int p = choose(four ? kFour : kBf16, rows, m, kblocks, gated).splits;
    if (p > 1) floats = std::max(floats, size_t(p) * rows * (gated ? 2 : 1) * round_up(m, 4));
  }
  w.part = c.take<float>(floats);
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

double mx_gemm_time(int64_t n, int64_t m, int64_t d, int form, bool gated) {
  if (form == GPTQ_MX_BF16) return choose(kBf16, n, m, (d + 63) / 64, gated).time;
  return choose(kFour, n, m, ceil_div(mx_blocks(d), kPer), gated).time + 4.0;   // and the layout
}

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
  const int64_t m = w.rows, nb = w.nb, nbp = round_up(nb, kPer), mpad = round_up(m, 256);
  for (int64_t t0 = 0; t0 < x.n; t0 += kRowChunk) {
    const int64_t nc = std::min<int64_t>(kRowChunk, x.n - t0), npad = round_up(nc, 256);
    GemmMx g{};
    g.n = nc;
    g.W[0] = w.codes;
    g.W[1] = up.codes;
    g.part = b.part;
    g.ldp = (gated ? 2 : 1) * round_up(m, 4);
    g.s_rows = x.form == GPTQ_MX_BF16 && stored_scales(w) && (!gated || stored_scales(up));
    g.S[0] = g.s_rows ? w.scales : b.wscale;
    g.S[1] = g.s_rows ? up.scales : b.wscale + nbp * mpad;
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
      g.kblocks = int(nbp / kPer);
      l.xscale = b.xscale;
      g.X = reinterpret_cast<const char*>(b.xcodes);
      l.xcodes = b.xcodes;
      if (x.form == GPTQ_MX_CODES) {
        l.x.X = static_cast<const uint8_t*>(x.X) + t0 * nb * 16;
        l.x.scales = x.scales + t0 * nb;
        l.blocks_xs = ceil_div(npad * (nbp / kPer), 256);
        if (nb == nbp) {                     // whole blocks: used as they lie
          g.X = static_cast<const char*>(l.x.X);
          l.xcodes = nullptr;
        }
      } else {
        l.x.X = static_cast<const uint16_t*>(x.X) + t0 * x.ldx;
        l.vec = x.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(l.x.X) % 16 == 0;
      }
      if (l.xcodes) l.blocks_x = ceil_div(int64_t(ceil_div(nc, kLayRows)) * l.runs, 4);
    }
    if (t0 == 0 && !g.s_rows) l.blocks_w = ceil_div(mpad * (nbp / kPer), 256);
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

// Y = V M^T, both bf16: rows 16-byte aligned, k in blocks of 64, n at most kRowChunk.
size_t mx_dense_floats(int64_t n, int64_t m, int64_t k) {
  const int p = choose(kDense, n, m, k / 64, false).splits;
  return p > 1 ? size_t(p) * n * round_up(m, 4) : 0;
}

gptq_status launch_mx_dense(const uint16_t* V, int64_t ldv, int64_t n, const uint16_t* M,
                            int64_t ldm, int64_t m, int64_t k, const MxOutput& y, float* part,
                            hipStream_t st) {
  GemmMx g{};
  g.X = reinterpret_cast<const char*>(V);
  g.ldx = ldv * 2;
  g.n = n;
  g.W[0] = reinterpret_cast<const uint8_t*>(M);
  g.ldw = ldm * 2;
  g.m = m;
  g.kblocks = int(k / 64);
  g.part = part;
  g.ldp = round_up(m, 4);
  g.y = y;
  return launch_form<kDense, false>(g, st);
}

}  // namespace gptq
