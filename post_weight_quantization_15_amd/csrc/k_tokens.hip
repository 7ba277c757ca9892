// What a row of logits says about a token: its log probability, the entropy of
// the row's distribution, its log-sum-exp, and the row's largest logits with
// their ids; and the gradient of the first two.
//
// With z = x / T, one pass over the row: s = sum 2^(c (x - r)) and t = sum c (x
// - r) 2^(c (x - r)), c = log2(e) / T, r the largest cell that the wave has seen,
// in the end the row's; then
//   lse = r / T + ln s,  log p = (x_v - r) / T - ln s,
//   entropy = ln s - ln2 t / s.
// No term is positive in t, none negative in s, and the largest cell is 1 in s, so nothing
// cancels.  Cells are exponentiated in fp32 and summed in fp32 for 32 cells of a thread,
// in fp64 beyond; a cell that becomes the largest is counted apart, as its 1 would leave
// a confident row's other cells no bits in an fp32 sum.  In a row without order a wave's largest
// rises in some ln(vocab / 2048) steps (all moves together take 1 to 3 % of the time).
//
// The largest k: cells pass a bar that only rises.  The first bar comes from the
// lanes' maxima over the cells at hand (a step's and those whose loads are ahead of it):
// the highest bound that 1, 2 or 4 waves give, each of which at least k cells
// reach.  What passes is kept in LDS as (value, lower id first) in one 64-bit number, all
// different; where many are there, the k-th of them, found digit by digit, is
// the new bar.  A cell later in the row has to exceed it: an equal one has the higher
// id (so the cells behind the last whole vector become candidates with the last step, though
// they are read first).  In a row without order some k ln(vocab) cells pass, so the selection
// is a comparison per 16 bytes; a row that rises all along selects at each look (k = 64, 1024
// rows of 128000 fp32 values: 1460 us, in disorder 117; 4096 of bf16: 6260 and 285).  Measured,
// bf16 rows: 4096 of 128000 take 197 us without alternatives (5.3 TB/s of one reading, part of it
// from the last cache), 285 with k = 64, 443 with 256, 638 with 512; one row of 128000, in 63
// parts of its own workgroups and joined by a second launch, 17 to 19 us with k = 20, of which the
// launches' kernels are 9 and 8: two readings' latency, a selection and the joining one.
#include <type_traits>

#include "lora.h"

namespace gptq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kLook = 4;                     // steps between two looks at the candidates
constexpr int kAhead = 3;                    // steps whose loads are under way
constexpr int kCap = 2048;                   // candidates in LDS (twice as many for k > kThreads)
constexpr int kByRank = 512;                 // as many are sorted by counting
constexpr int kBars = 3;                     // 1, 2, 4 waves
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.693147180559945309417;
constexpr float kLowest = -3.402823466e38f;

template <int DT>
struct Cells {
  using type = std::conditional_t<DT == GPTQ_F32, float, uint16_t>;
  static constexpr int kPer = DT == GPTQ_F32 ? 4 : 8;    // cells per 16 bytes
  static constexpr int kVec = 8 / kPer;                  // 16-byte loads of a thread's step
};

template <int DT>
__device__ inline float to_f32(typename Cells<DT>::type v) {
  if constexpr (DT == GPTQ_F32) return v;
  else if constexpr (DT == GPTQ_BF16) return __uint_as_float(uint32_t(v) << 16);
  else return static_cast<float>(__builtin_bit_cast(_Float16, v));
}
// Cell i of 16 bytes.
template <int DT>
__device__ inline float cell_of(const u32x4& v, int i) {
  if (DT == GPTQ_F32) return __uint_as_float(v[i % 4]);
  const uint32_t w = v[(i >> 1) % 4];
  if (DT == GPTQ_BF16) return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> (16 * (i & 1)))));
}

// The larger of three, numbers before quiet NaN (a signalling NaN may make the result NaN).
__device__ inline float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// fp32 numbers as integers that order alike: -inf above 0, NaN 0 (never among
// the largest), -0 as 0.
__device__ inline uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// A candidate: value, then lower id first (ids have 18 bits).
static_assert(kDistillMaxVocab == 1 << 18, "ids have 18 bits");
__device__ inline uint64_t entry_of(float x, int id) {
  return uint64_t(order_of(x)) << 18 | (0x3FFFFu - static_cast<uint32_t>(id));
}
__device__ inline uint32_t order_in(uint64_t e) { return static_cast<uint32_t>(e >> 18); }

template <class T, class F>
__device__ inline T wave_all(T v, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
  return v;
}

// What the selections share beside the candidates.
struct Scratch {
  int hist[256];
  uint32_t totals[kWaves];
  uint64_t prefix;
  int need, cnt;
};

// An entry that exactly k of buf[0 .. count) reach, k < count: digit by digit from
// the top, the digit where the k-th largest lies; done where all of it belong to the k.
__device__ inline uint64_t kth_entry(const uint64_t* buf, int count, int k, Scratch& sc) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  uint64_t prefix = 0u;
  int need = k;
#pragma unroll 1
  for (int known = 50; ;) {                  // the bits from here up are decided
    const int shift = max(known - 8, 0);
    const uint32_t digits = (1u << (known - shift)) - 1u;
    static_assert(kThreads == 256, "a thread a bin");
    sc.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < count; i += kThreads) {
      const uint64_t e = buf[i];
      if (e >> known == prefix >> known)
        atomicAdd(&sc.hist[static_cast<uint32_t>(e >> shift) & digits], 1);
    }
    __syncthreads();
    const int own = sc.hist[tid];
    int from = own;                          // entries in this bin and above
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_down(from, o);
      if (lane + o < 64) from += u;
    }
    if (lane == 0) sc.totals[wv] = from;
    __syncthreads();
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
      if (w > wv) from += sc.totals[w];
    if (from >= need && from - own < need) {
      sc.prefix = prefix | uint64_t(tid) << shift;
      // the whole bin: no digit below it matters
      sc.need = from == need ? 0 : need - (from - own);
    }
    __syncthreads();
    prefix = sc.prefix;
    need = sc.need;
    if (need == 0 || shift == 0) return prefix;
    known = shift;
  }
}

// The entries of buf[0 .. count) from `least` up, to its front; all threads call it.
__device__ inline void keep_from(uint64_t* buf, int count, uint64_t least, Scratch& sc) {
  const int tid = threadIdx.x;
  if (tid == 0) sc.cnt = 0;
  for (int b = 0; b < count; b += kThreads) {
    const uint64_t e = b + tid < count ? buf[b + tid] : 0u;
    __syncthreads();                         // these are read: as many places are free
    if (e >= least && b + tid < count) buf[atomicAdd(&sc.cnt, 1)] = e;
  }
  __syncthreads();
}

// buf[0 .. count), count <= kByRank, in descending order.
__device__ inline void sort_by_rank(uint64_t* buf, int count) {
  constexpr int kOwn = kByRank / kThreads;
  const int tid = threadIdx.x;
  uint64_t own[kOwn];
  int rank[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    own[j] = tid + j * kThreads < count ? buf[tid + j * kThreads] : 0u;
    rank[j] = 0;
  }
  if ((tid & ~63) < count) {                 // waves without an entry wait below
    if (count <= kThreads) {
#pragma unroll 4
      for (int i = 0; i < count; ++i) rank[0] += buf[i] > own[0];
    } else {
#pragma unroll 2
      for (int i = 0; i < count; ++i) {
        const uint64_t v = buf[i];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) rank[j] += v > own[j];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kOwn; ++j)
    if (tid + j * kThreads < count) buf[rank[j]] = own[j];
  __syncthreads();
}

// The wave's order numbers ranked.  The last six bits make way for the lane's number, which makes
// lanes different, and come back as zeros (a lower bound).
struct Ranked {
  uint32_t key;
  int rank;                                  // lanes above
};
__device__ inline Ranked rank_lanes(uint32_t order) {
  Ranked r{(order & ~63u) | (threadIdx.x & 63u), 0};
#pragma unroll 8
  for (int l = 0; l < 64; ++l)
    r.rank += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(r.key), l)) > r.key;
  return r;
}
// What p lanes reach: the p-th largest lane's, 1 <= p <= 64.  Where a lane has the (k / p)-th
// largest (rounded up) of its own list, k numbers of all lists reach it.
__device__ inline uint32_t reached_by(const Ranked& r, int p) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(
             static_cast<int>(r.key), __builtin_ctzll(__ballot(r.rank == p - 1)))) & ~63u;
}

struct TokenArgs {
  const void* logits;
  int64_t ldl;
  int vocab, k, parts, span;                 // a part: span cells of a row
  int cap;                                   // candidates that the LDS holds
  double inv_temp;
  const int32_t* token;
  float* logp;
  float* entropy;
  float* lse;
  float* stats;
  float* top;
  int32_t* idx;
  double* part_sums;                         // [n][parts][3]
  uint64_t* part_top;                        // [n][parts][k]
};

// The row's token's logit (0 without a token); asked for at the start, for two
// loads one behind the other.
template <int DT>
__device__ inline float token_logit(const TokenArgs& a, int64_t row, bool& given) {
  const int id = a.token ? a.token[row] : -1;
  given = id >= 0 && id < a.vocab;
  if (!given) return 0.0f;
  return to_f32<DT>(static_cast<const typename Cells<DT>::type*>(a.logits)[row * a.ldl + id]);
}

// What the row's sums say; one thread.
__device__ inline void finish_row(const TokenArgs& a, int64_t row, double ref, double s, double t,
                                  bool given, float x) {
  double lse, rest, h;
  if (s == 0.0) {                            // nothing but -inf
    lse = rest = -INFINITY;
    h = __longlong_as_double(0x7FF8000000000000ll);
  } else {
    rest = log(s);
    lse = ref * a.inv_temp + rest;
    h = rest - kLn2 * (t / s);
  }
  if (a.logp)
    a.logp[row] = given ? static_cast<float>(s == 0.0 ? h : (double(x) - ref) * a.inv_temp - rest) : 0.0f;
  if (a.entropy) a.entropy[row] = static_cast<float>(h);
  if (a.lse) a.lse[row] = static_cast<float>(lse);
  if (a.stats) {
    a.stats[3 * row] = static_cast<float>(ref);
    a.stats[3 * row + 1] = static_cast<float>(rest);
    a.stats[3 * row + 2] = static_cast<float>(h);
  }
}

__device__ inline void write_top(const TokenArgs& a, int64_t row, const uint64_t* buf, int have) {
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    const uint64_t e = i < have ? buf[i] : 0u;
    const bool some = order_in(e);
    a.top[row * a.k + i] = some ? value_of(order_in(e)) : -INFINITY;
    a.idx[row * a.k + i] = some ? static_cast<int32_t>(0x3FFFFu - (static_cast<uint32_t>(e) & 0x3FFFFu)) : -1;
  }
}

// Sums relative to a reference moved to one that is higher by `up` (in powers of
// two).  2^-up by the exponential's series for the fraction, |y| <= ln2 / 2, to 2e-10 (a row that
// rises all along moves its sums at every step); constant factors, not terms, as those
// would occupy registers throughout.
__device__ inline void move_sums(double& s, double& t, double up) {
  up = up < 1000.0 ? up : 1000.0;
  const int n = static_cast<int>(up + 0.5);
  const double y = (n - up) * kLn2;
  double f = 1.0;
#pragma unroll
  for (int k = 8; k > 0; --k) f = fma(y * (1.0 / k), f, 1.0);
  f = ldexp(f, -n);
  t = f * (t - up * s);
  s *= f;
}

// The lanes' sums, each relative to its own reference, as one of them all.
__device__ inline void join_sums(double& r, double& s, double& t, float c) {
  const double most = wave_all(r, [](double x, double y) { return x > y ? x : y; });
  if (r < most) move_sums(s, t, double(c) * (most - r));
  r = most;
  s = wave_all(s, [](double x, double y) { return x + y; });
  t = wave_all(t, [](double x, double y) { return x + y; });
}

template <int DT>
__global__ __launch_bounds__(kThreads, 6) void tokens_kernel(TokenArgs a) {
  using T = typename Cells<DT>::type;
  constexpr int E = Cells<DT>::kPer, NV = Cells<DT>::kVec;
  constexpr int kSteps = kThreads * NV;      // vectors of a step
  extern __shared__ __attribute__((aligned(16))) uint64_t buf[];
  __shared__ double red[3][kWaves];
  __shared__ uint32_t bars[kBars][kWaves];
  __shared__ Scratch sc;
  __shared__ int cnt;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t row = blockIdx.x;
  const int part = blockIdx.y, first = part * a.span;
  const int V = min(a.span, a.vocab - first);
  const T* src = static_cast<const T*>(a.logits) + row * a.ldl + first;
  const int head = min(V, static_cast<int>((E - (reinterpret_cast<uintptr_t>(src) / sizeof(T)) % E) % E));
  const int nvec = (V - head) / E, last = head + nvec * E;
  // the cells before and after the whole vectors, one a thread
  const int edge = tid < head ? tid : tid >= E && tid - E < V - last ? last + tid - E : -1;
  const float c = static_cast<float>(a.inv_temp) * kLog2e;
  const int steps = max(1, (nvec + kSteps - 1) / kSteps);
  const T* body = src + head;

  // loads run kAhead steps ahead, in registers that move up a step at a time (the loop is
  // not unrolled: a single row is bound by the fetch of its instructions)
  u32x4 ring[kAhead][NV];
  auto load = [&](u32x4 (&v)[NV], int step) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = step * kSteps + i * kThreads + tid;
      if (at < nvec) v[i] = *reinterpret_cast<const u32x4*>(body + int64_t(at) * E);
    }
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) load(ring[s], s);
  bool given = false;
  float token_x = 0.0f;
  if (tid == 0) {
    cnt = 0;
    if (a.parts == 1) token_x = token_logit<DT>(a, row, given);
  }
  float ez = -INFINITY;
  if (edge >= 0) ez = to_f32<DT>(src[edge]);
  __syncthreads();
  int have = 0;                              // candidates: the cells before the vectors, to begin with
  if (a.k) {
    const bool some = tid < head && ez == ez;
    if (some) buf[atomicAdd(&cnt, 1)] = entry_of(ez, first + edge);
    have = __syncthreads_count(some);
  }
  float bar = -INFINITY;                     // cells from here up are candidates
  float ref = kLowest;
  double s = 0.0, t = 0.0;                   // of this thread, relative to ref
  // candidates among the cells of one vector (past the buffer's end: counted only)
  auto push = [&](const u32x4& v, int at) {
    uint32_t hits = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e) hits |= cell_of<DT>(v, e) >= bar ? 1u << e : 0u;
    const u32x4 w = v;
    while (hits) {
      const int e = __builtin_ctz(hits);
      hits &= hits - 1u;
      const int i = DT == GPTQ_F32 ? e : e >> 1;
      uint32_t word = w[0];
      word = i == 1 ? w[1] : word;
      word = i == 2 ? w[2] : word;
      word = i == 3 ? w[3] : word;
      float x = __uint_as_float(word);
      if (DT == GPTQ_BF16) x = __uint_as_float(e & 1 ? word & 0xFFFF0000u : word << 16);
      if (DT == GPTQ_F16)
        x = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(word >> (16 * (e & 1)))));
      const int p = atomicAdd(&cnt, 1);
      if (p < a.cap) buf[p] = entry_of(x, first + head + at * E + e);
    }
  };
  // the cells behind the vectors: after all lower ids, so that a bar just above the k-th
  // candidate drops no cell of that value with a lower id
  auto push_tail = [&]() {
    if (edge >= last && ez >= bar) {
      const int p = atomicAdd(&cnt, 1);
      if (p < a.cap) buf[p] = entry_of(ez, first + edge);
    }
  };
  int from = 0;                              // first step since the last look
  float ps = 0.0f, pt = 0.0f;                // of kLook steps
  int ones = 0;                              // cells equal to a reference that is new
  auto add_cell = [&](float x, auto fresh) {
    float d = (x - ref) * c;
    float e = __builtin_amdgcn_exp2f(d);
    if constexpr (decltype(fresh)::value) {
      const bool one = d == 0.0f;            // (+inf: NaN, which goes into the sum)
      ones += one;
      e = one ? 0.0f : e;
    }
    d = max3(d, -1000.0f, -1000.0f);         // 0 times -inf
    ps += e;
    pt = fmaf(e, d, pt);
  };

#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    u32x4 cur[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cur[i] = ring[0][i];
#pragma unroll
      for (int u = 0; u + 1 < kAhead; ++u) ring[u][i] = ring[u + 1][i];
    }
    load(ring[kAhead - 1], step + kAhead);
    const int at0 = step * kSteps + tid;
    // ---- the largest cell of each vector
    float top[NV], gm = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float m = -INFINITY;
      if (at0 + i * kThreads < nvec) {
#pragma unroll
        for (int e = 0; e < E; e += 2) m = max3(m, cell_of<DT>(cur[i], e), cell_of<DT>(cur[i], e + 1));
      }
      top[i] = m;
      gm = max3(gm, m, step == 0 ? ez : m);
    }
    // ---- sums
    auto add_step = [&](auto fresh) {
      if (step == 0 && edge >= 0) add_cell(ez, fresh);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (at0 + i * kThreads < nvec) {
#pragma unroll
          for (int e = 0; e < E; ++e) add_cell(cell_of<DT>(cur[i], e), fresh);
        }
      }
    };
    uint64_t above = __ballot(gm > ref);
    if (above) {
      // the wave's largest, a lane that has more at a time (in a row that rises the last one has it)
      float up = ref;
      do {
        up = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gm), 63 - __builtin_clzll(above)));
        above = __ballot(gm > up);
      } while (above);
      s += ps;
      t += pt;
      ps = pt = 0.0f;
      if (step) move_sums(s, t, double(c) * (double(up) - double(ref)));
      ref = up;
      ones = 0;
      add_step(std::true_type{});
      s += ones;
    } else {
      add_step(std::false_type{});
    }
    // (without a first bar a step fills the candidates)
    const bool look = step % kLook == kLook - 1 || step + 1 == steps || (step == 0 && a.k > kThreads);
    if (look) {
      s += ps;
      t += pt;
      ps = pt = 0.0f;
    }
    // ---- candidates
    if (!a.k) continue;
    if (step == 0) {
      // A bar from the lanes' maxima over all cells at hand (this step's and those ahead).
      // For 1, 2, 4 waves: the (k / waves)-th of each wave, and of these the one that
      // as many waves reach: at least k cells are as large.  The highest of those
      // bars holds also where some waves see only masked cells.
      float most = gm;
#pragma unroll
      for (int u = 0; u + 1 < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (at0 + (u + 1) * kSteps + i * kThreads < nvec) {
#pragma unroll
            for (int e = 0; e < E; e += 2)
              most = max3(most, cell_of<DT>(ring[u][i], e), cell_of<DT>(ring[u][i], e + 1));
          }
      const Ranked lanes = rank_lanes(order_of(most));
#pragma unroll
      for (int g = 0; g < kBars; ++g) {
        const int want = (a.k + (1 << g) - 1) >> g;
        const uint32_t pick = want <= 64 ? reached_by(lanes, want) : 0u;
        if (lane == 0) bars[g][wv] = pick;
      }
      __syncthreads();
      // lane 8 g + w: wave w's for 2^g waves
      const bool one = lane < 8 * kBars && (lane & 7) < kWaves;
      const uint32_t mine = one ? bars[lane >> 3][lane & 7] : 0u;
      int above = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const uint32_t o = static_cast<uint32_t>(__shfl(static_cast<int>(mine), (lane & ~7) + w));
        above += o > mine || (o == mine && w < (lane & 7));
      }
      const uint32_t best = wave_all(one && above == (1 << (lane >> 3)) - 1 ? mine : 0u,
                                     [](uint32_t x, uint32_t y) { return x > y ? x : y; });
      bar = best > order_of(-INFINITY) ? value_of(best) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = at0 + i * kThreads;
      // (a signalling NaN makes the maximum NaN: its vector's cells are looked at one by one)
      bool in = !(top[i] < bar) && at < nvec;
      if (from == 0) {
        // many cells may equal the first bar (masked ones): those with k and more of them
        // before them in their wave are not among the k largest
        int same = 0;
        if (in && top[i] == bar) {
#pragma unroll
          for (int e = 0; e < E; ++e) same += cell_of<DT>(cur[i], e) == bar;
        }
        int before = same;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int u = __shfl_up(before, o);
          if (lane >= o) before += u;
        }
        if (top[i] == bar && before - same >= a.k) in = false;
      }
      if (in) push(cur[i], at);
    }
    if (!look) continue;
    if (step + 1 == steps) push_tail();
    __syncthreads();
    const int found = cnt;
    __syncthreads();
    const bool again = found > a.cap;
    if (found <= max(2 * a.k + 64, kByRank) && step + 1 < steps) {
      have = found;
      from = step + 1;
      continue;
    }
    // too many at once: these steps again in halves, each in room for all its cells
    int u = again ? 2 * from : 2 * step + 1, now = found;
#pragma unroll 1
    do {
      if (again) {
        if (tid == 0) cnt = have;
        __syncthreads();
        if (tid < kThreads / 2) {
#pragma unroll 1
          for (int i = 0; i < NV; ++i) {
            const int at = (u * NV + i) * (kThreads / 2) + tid;
            if (at < nvec) push(*reinterpret_cast<const u32x4*>(body + int64_t(at) * E), at);
          }
        }
        if (u == 2 * steps - 1) push_tail();
        __syncthreads();
        now = cnt;
        __syncthreads();
      }
      have = now;
      // (few are put in order as they are, below)
      if (now > (again || step + 1 < steps ? a.k : max(a.k, kThreads))) {
        const uint64_t least = kth_entry(buf, now, a.k, sc);
        keep_from(buf, now, least, sc);
        have = a.k;
        // where all of a bin belong to the k, `least` lies at or below the k-th
        bar = fmaxf(bar, value_of(order_in(least) + ((least & 0x3FFFFu) != 0u)));
      }
    } while (++u <= 2 * step + 1);
    from = step + 1;
    if (tid == 0) cnt = have;
    __syncthreads();
  }
  if (a.k) sort_by_rank(buf, have);
  // ---- the waves' sums, moved to the highest reference
  s = wave_all(s, [](double x, double y) { return x + y; });
  t = wave_all(t, [](double x, double y) { return x + y; });
  if (lane == 0) {
    red[0][wv] = ref;
    red[1][wv] = s;
    red[2][wv] = t;
  }
  __syncthreads();
  if (wv == 0) {
    double r = lane < kWaves ? red[0][lane] : double(kLowest);
    s = lane < kWaves ? red[1][lane] : 0.0;
    t = lane < kWaves ? red[2][lane] : 0.0;
    join_sums(r, s, t, c);
    if (lane == 0) {
      if (a.parts == 1) {
        finish_row(a, row, r, s, t, given, token_x);
      } else {
        double* o = a.part_sums + (row * a.parts + part) * 3;
        o[0] = r;
        o[1] = s;
        o[2] = t;
      }
    }
  }
  if (a.k) {
    if (a.parts == 1) {
      write_top(a, row, buf, have);
    } else {
      uint64_t* o = a.part_top + (row * a.parts + part) * a.k;
      for (int i = tid; i < a.k; i += kThreads) o[i] = i < have ? buf[i] : 0u;
    }
  }
}

// The parts of a row, joined: one workgroup a row.
template <int DT>
__global__ __launch_bounds__(kThreads) void tokens_join_kernel(TokenArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t buf[];
  __shared__ Scratch sc;
  __shared__ int cnt;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint64_t* in = a.part_top + row * a.parts * a.k;
  bool given = false;
  float token_x = 0.0f;
  double r = kLowest, s = 0.0, t = 0.0;      // a part's sums in a lane: at most 64 parts
  if (tid == 0) {
    cnt = 0;
    token_x = token_logit<DT>(a, row, given);
  }
  if (tid < a.parts) {
    const double* p = a.part_sums + (row * a.parts + tid) * 3;
    r = p[0];
    s = p[1];
    t = p[2];
  }
  uint64_t bar = 0u;
  if (a.k) {
    // as for a part's first cells: for all parts and for a quarter of them
    const int lane = tid & 63, few = max(a.parts / 4, 1);
    const uint64_t* mine = in + min(lane, a.parts - 1) * a.k;
    const uint32_t all = order_in(mine[(a.k + a.parts - 1) / a.parts - 1]);
    const uint32_t some = order_in(mine[(a.k + few - 1) / few - 1]);
    const uint32_t x = reached_by(rank_lanes(lane < a.parts ? all : 0u), a.parts);
    const uint32_t y = reached_by(rank_lanes(lane < a.parts ? some : 0u), few);
    bar = uint64_t(max(x, y)) << 18;
  }
  __syncthreads();
  if (a.k) {
    for (int i = tid; i < a.parts * a.k; i += kThreads) {
      const uint64_t e = in[i];
      if (e && e >= bar) buf[atomicAdd(&cnt, 1)] = e;
    }
    __syncthreads();
    int have = cnt;
    __syncthreads();
    if (have > max(a.k, kThreads)) {
      const uint64_t least = kth_entry(buf, have, a.k, sc);
      keep_from(buf, have, least, sc);
      have = a.k;
    }
    sort_by_rank(buf, have);
    write_top(a, row, buf, have);
  }
  if (tid < 64) {
    join_sums(r, s, t, static_cast<float>(a.inv_temp) * kLog2e);
    if (tid == 0) finish_row(a, row, r, s, t, given, token_x);
  }
}

// ---------------------------------------------------------------------------
// The gradient: dx_v = [g (1[v = token] - q_v) - h q_v (log q_v + entropy)] / T
// ---------------------------------------------------------------------------
struct TokenGradArgs {
  const void* logits;
  int64_t n, ldl;
  int vocab, pieces;
  double inv_temp;
  const float* stats;
  const int32_t* token;
  const float* grad_logp;
  const float* grad_entropy;
  void* dlogits;
  int64_t ldd;
};

constexpr int kGradThreads = 256, kGradVecs = 4;         // of 8 cells

template <int DT>
__global__ __launch_bounds__(kGradThreads) void tokens_grad_kernel(TokenGradArgs a) {
  using T = typename Cells<DT>::type;
  constexpr int E = Cells<DT>::kPer;
  constexpr int kVecs = kGradVecs * Cells<DT>::kVec;
  const int tid = threadIdx.x;
  const int64_t row = flat_block() / static_cast<unsigned>(a.pieces);
  const int piece = static_cast<int>(flat_block() % static_cast<unsigned>(a.pieces));
  if (row >= a.n) return;
  const T* src = static_cast<const T*>(a.logits) + row * a.ldl;
  T* dst = static_cast<T*>(a.dlogits) + row * a.ldd;
  const int V = a.vocab;
  auto head_of = [&](const T* p) {
    return min(V, static_cast<int>((E - (reinterpret_cast<uintptr_t>(p) / sizeof(T)) % E) % E));
  };
  const int head = head_of(src), nvec = (V - head) / E, last = head + nvec * E;
  const bool same = head_of(dst) == head;
  const int v0 = piece * kGradThreads * kVecs + tid;
  u32x4 x[kVecs];
  const int id = a.token ? a.token[row] : -1;
  const bool given = id >= 0 && id < V;
  const float g = given && a.grad_logp ? a.grad_logp[row] : 0.0f;
  const float h = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
  const bool none = g == 0.0f && h == 0.0f;  // a row that does not count: nothing of it is read
  if (!none) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = v0 + i * kGradThreads;
      if (v < nvec) x[i] = *reinterpret_cast<const u32x4*>(src + head + int64_t(v) * E);
    }
  }
  const float ref = a.stats[3 * row], rest = a.stats[3 * row + 1], H = a.stats[3 * row + 2];
  const float it = static_cast<float>(a.inv_temp), c = it * kLog2e, rest2 = rest * kLog2e;
  const float gt = g * it, ht = h * it;
  auto grad = [&](float v, int at) {
    if (none) return 0.0f;
    const float d = v - ref;
    const float q = __builtin_amdgcn_exp2f(fmaf(d, c, -rest2));
    const float lq = fmaxf(fmaf(d, it, -rest), -1e4f);
    float o = -q * fmaf(ht, lq + H, gt);
    if (at == id) o += gt;
    return o;
  };
  auto as_cell = [](float v) {
    if constexpr (DT == GPTQ_F32) return v;
    else if constexpr (DT == GPTQ_BF16) return f32_bf16(v);
    else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  };
  if (piece == 0) {
    const int edge = tid < head ? tid : tid >= E && tid - E < V - last ? last + tid - E : -1;
    if (edge >= 0) dst[edge] = as_cell(grad(none ? 0.0f : to_f32<DT>(src[edge]), edge));
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = v0 + i * kGradThreads;
    if (v >= nvec) break;
    const int at = head + v * E;
    T o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = as_cell(grad(cell_of<DT>(x[i], e), at + e));
    if (same) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (DT == GPTQ_F32) w[e] = __float_as_uint(o[e]);
        else w[e] = uint32_t(o[2 * e]) | uint32_t(o[2 * e + 1]) << 16;
      }
      *reinterpret_cast<u32x4*>(dst + at) = w;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) dst[at + e] = o[e];
    }
  }
}

// Parts of a row: enough workgroups for the chip where rows are few, of 2048
// cells (8 a thread) at least, their candidates within the join's LDS.
int parts_of(int64_t n, int64_t vocab, int64_t k) {
  int64_t p = std::min<int64_t>(1024 / std::max<int64_t>(n, 1), (vocab + 2047) / 2048);
  p = std::min<int64_t>(p, 64);
  if (k) p = std::min<int64_t>(p, kCap / k);
  return int(std::max<int64_t>(p, 1));
}

struct TokenWs {
  double* sums;
  uint64_t* top;
};
TokenWs carve_tokens(Carver& c, int64_t n, int64_t vocab, int64_t k) {
  TokenWs w{};
  const int parts = parts_of(n, vocab, k);
  if (n == 0 || parts == 1) return w;
  w.sums = c.take<double>(size_t(n) * parts * 3);
  if (k) w.top = c.take<uint64_t>(size_t(n) * parts * k);
  return w;
}

template <int DT>
gptq_status launch_forward(const TokenArgs& a, int64_t n, hipStream_t st) {
  const size_t lds = a.k ? size_t(a.cap) * 8 : 0;
  tokens_kernel<DT><<<dim3(unsigned(n), unsigned(a.parts)), kThreads, lds, st>>>(a);
  GPTQ_CHECK_LAUNCH();
  if (a.parts > 1) {
    tokens_join_kernel<DT><<<unsigned(n), kThreads, lds, st>>>(a);
    GPTQ_CHECK_LAUNCH();
  }
  return GPTQ_OK;
}

}  // namespace

size_t tokens_ws_bytes(int64_t n, int64_t vocab, int64_t k) {
  Carver c(nullptr);
  carve_tokens(c, n, vocab, k);
  return c.bytes();
}

gptq_status launch_tokens(const void* logits, gptq_dtype dt, int64_t n, int64_t vocab, int64_t ldl,
                          const int32_t* token, float temp, int64_t k, float* logp, float* entropy,
                          float* lse, float* stats, float* top, int32_t* idx, void* ws,
                          hipStream_t st) {
  Carver c(ws);
  const TokenWs w = carve_tokens(c, n, vocab, k);
  TokenArgs a{logits, ldl, int(vocab), int(k), parts_of(n, vocab, k), 0, k > kThreads ? 2 * kCap : kCap,
              1.0 / double(temp), token,
              logp, entropy, lse, stats, top, idx, w.sums, w.top};
  a.span = int(round_up((vocab + a.parts - 1) / a.parts, 8));
  a.parts = int((vocab + a.span - 1) / a.span);          // none is empty
  switch (dt) {
    case GPTQ_F32: return launch_forward<GPTQ_F32>(a, n, st);
    case GPTQ_F16: return launch_forward<GPTQ_F16>(a, n, st);
    default: return launch_forward<GPTQ_BF16>(a, n, st);
  }
}

gptq_status launch_tokens_grad(const void* logits, gptq_dtype dt, int64_t n, int64_t vocab,
                               int64_t ldl, const float* stats, const int32_t* token, float temp,
                               const float* grad_logp, const float* grad_entropy, void* dlogits,
                               int64_t ldd, hipStream_t st) {
  TokenGradArgs a{logits, n, ldl, int(vocab), int(ceil_div(vocab, 8 * kGradThreads * kGradVecs)),
                  1.0 / double(temp), stats, token, grad_logp, grad_entropy, dlogits, ldd};
  const dim3 grid = flat_grid(n * a.pieces);
  switch (dt) {
    case GPTQ_F32: tokens_grad_kernel<GPTQ_F32><<<grid, kGradThreads, 0, st>>>(a); break;
    case GPTQ_F16: tokens_grad_kernel<GPTQ_F16><<<grid, kGradThreads, 0, st>>>(a); break;
    default: tokens_grad_kernel<GPTQ_BF16><<<grid, kGradThreads, 0, st>>>(a); break;
  }
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

}  // namespace gptq
