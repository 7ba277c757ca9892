// Distillation from a teacher known by its top logits: the divergence of a
// student's logits from it, per row, and the gradient.
//
// With z = logits / T, q = softmax(z) over the vocabulary, S the row's known
// ids (those inside [0, V)) and p the teacher's probabilities on them,
//   loss = w T^2 sum_S p_i (log p_i - log q_i)
//   d loss / d logits_v = w T (q_v - p_v)           (p_v = 0 outside S),
// p renormalised over S (softmax of t / T), or, where the teacher's
// log-sum-exp is given, its true probabilities exp(t / T - t_lse) with what
// is left, p_r = 1 - sum p, as one more class against the student's
// q_r = 1 - sum_S q: the loss gains p_r (log p_r - log q_r) and the cells
// outside S get w T q_v (1 - p_r / q_r).  Where that class is left out (p_r =
// 0, or q_r = 0: every cell outside S at -inf) what the probabilities add up
// to, P = sum_S p, stands before q: w T (P q_v - p_v) on S, w T P q_v elsewhere.
//
// One workgroup per row.  The row's cells are read once, 16 bytes a load,
// and stay in registers as stored (a row of up to 131072 16-bit cells is
// 64 registers in each of 1024 threads) through the maximum, the sum of
// exponentials and the gradient's store, so the traffic is the floor: one
// read, and one write where a gradient is asked for.  Longer rows are read
// again for the gradient.  Cells of S are taken out of the registers through
// a bit mask of the row in LDS, so that q_r is a sum of its own and not the
// small difference of two large ones; everything per row or per known id
// (the teacher's probabilities, the two log-sum-exps, the loss, the
// gradient on S) is in fp64, because the loss's terms nearly cancel where
// student and teacher agree.  Cells are exponentiated in fp32 and summed in
// fp32 per thread (at most 128 and an edge cell; 16 bytes' worth in longer
// rows), in fp64 beyond that and across threads, in a fixed order: results
// are the same bits from run to run.
//
// Bound by memory where workgroups share a CU, so that one's loads and stores
// run beside another's exponentials: loss and gradient of 4096 bf16 rows of
// 64000 cells take 224 us, 4.7 TB/s of the 4.9 that a copy reaches (254 with a
// class for the rest).  A row of 128000 takes a CU's whole register file but
// for what the code needs, so its loads wait for the row before: 510 us, 4.1
// TB/s (545 to 570 with a class for the rest); with every wave at the known
// ids, a barrier per sum of theirs and a maximum in fp32 it took four tenths
// more.  Streamed rows move three lengths for the loss and the gradient: 1024
// rows of 262144 bf16 cells 316 us, of 128000 fp32 cells 320 (the loss alone
// 102 and 100, the gradient alone 218 and 226).  Few rows are bound by the
// chain of one row: 11 us for 24 rows of 32000.  Loading the next row into
// registers that the stores free was tried: its registers spill, four times
// the time.
#include <type_traits>

#include "common.h"

namespace gptq {
namespace {

constexpr int kMaxK = kDistillMaxK;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kFarLse = 1024.0f;       // from here fp32 stats are off by 2^-14 and more

template <int DT>
struct Cell;
template <>
struct Cell<GPTQ_F32> {
  using type = float;
  static constexpr int kPer = 4;                     // cells per 16 bytes
  static constexpr uint32_t kNegInf = 0xFF800000u;
};
template <>
struct Cell<GPTQ_BF16> {
  using type = uint16_t;
  static constexpr int kPer = 8;
  static constexpr uint32_t kNegInf = 0xFF80u;
};
template <>
struct Cell<GPTQ_F16> {
  using type = uint16_t;
  static constexpr int kPer = 8;
  static constexpr uint32_t kNegInf = 0xFC00u;
};

__device__ inline float cell_to_f32(float v, std::integral_constant<int, GPTQ_F32>) { return v; }
__device__ inline float cell_to_f32(uint16_t v, std::integral_constant<int, GPTQ_BF16>) {
  return __uint_as_float(uint32_t(v) << 16);
}
__device__ inline float cell_to_f32(uint16_t v, std::integral_constant<int, GPTQ_F16>) {
  return static_cast<float>(__builtin_bit_cast(_Float16, v));
}

// Cell i of a 16-byte vector.
template <int DT>
__device__ inline float get_cell(const u32x4& v, int i) {
  if (DT == GPTQ_F32) return __uint_as_float(v[i % 4]);
  const uint32_t h = (v[(i >> 1) % 4] >> (16 * (i & 1))) & 0xFFFFu;
  if (DT == GPTQ_BF16) return __uint_as_float(h << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}

template <int DT>
__device__ inline void set_bits(u32x4& v, int i, uint32_t bits) {
  if (DT == GPTQ_F32) {
    v[i % 4] = bits;
  } else {
    const int w = (i >> 1) % 4, s = 16 * (i & 1);
    v[w] = (v[w] & ~(0xFFFFu << s)) | (bits << s);
  }
}

// fp32 to the cell's type, rounded to nearest even, as bits.
template <int DT>
__device__ inline uint32_t to_bits(float v) {
  if (DT == GPTQ_F32) return __float_as_uint(v);
  if (DT == GPTQ_F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

struct DistillArgs {
  const void* logits;
  int64_t vocab, ldl;
  const int32_t* t_idx;
  const float* t_logits;
  int k;
  double inv_temp;
  float temp;
  const float* t_lse;
  const float* weight;
  const float* grad;      // backward: the loss's own gradient [n], else NULL
  float* loss;
  float* stats;           // [n][2]: read by backward, else written (may be NULL)
  void* dlogits;
  int64_t ldd;
};

// Sum (or maximum) over a wave / the workgroup, the same value in every thread.
template <class T, class F>
__device__ inline T wave_all(T v, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
  return v;
}
template <int THREADS, class T, class F>
__device__ inline T block_all(T v, T* red, F f) {
  v = wave_all(v, f);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) r = f(r, red[w]);
  return r;
}

template <class T>
__device__ inline T sum2(T a, T b) { return a + b; }
// NaN stays: a row with a NaN cell has a NaN loss
__device__ inline float fmax_nan(float a, float b) { return (a > b || a != a) ? a : b; }

typedef short s16x2 __attribute__((ext_vector_type(2)));

enum { kLoss = 0, kFused = 1, kBackward = 2 };

// fp64 exponential and logarithm, out of line: inlined, their constants are
// hoisted over the rows into registers that the row's cells need.
__device__ __attribute__((noinline)) double dexp(double x) { return exp(x); }
__device__ __attribute__((noinline)) double dlog(double x) { return log(x); }

// NV vectors of 16 bytes per thread held in registers; NV = 0: the row is
// streamed (and read again for the gradient).  The first wave alone sees to the
// known ids, the others wait for it at two barriers only.
template <int DT, int THREADS, int NV, int MODE>
__global__ __launch_bounds__(THREADS) void distill_kernel(DistillArgs a) {
  using T = typename Cell<DT>::type;
  using DTag = std::integral_constant<int, DT>;
  constexpr int E = Cell<DT>::kPer;
  constexpr double kLn2 = 0.693147180559945309417;
  extern __shared__ uint32_t mask[];     // one bit per cell, aligned as the vectors are
  __shared__ double p_s[kMaxK];          // teacher's probability of entry i (0: padding)
  __shared__ float z_s[kMaxK];           // student's logit of entry i
  __shared__ double redd[THREADS / 64];
  __shared__ float redf[THREADS / 64], redg[THREADS / 64];
  __shared__ int dup;
  __shared__ double sh_top, sh_lse, sh_factor, sh_mass;
  __shared__ float sh_coef, sh_refc;
  const int tid = threadIdx.x, lane = tid & 63;
  const bool first = tid < 64;           // the wave of the known ids
  const int V = static_cast<int>(a.vocab);
  const bool tail = a.t_lse != nullptr;
  const float cf = static_cast<float>(a.inv_temp) * kLog2e;

  // A row's body is its whole vectors, 16-byte aligned; the cells before and
  // after them (fewer than a vector each) are `edge`, one a thread.
  auto head_of = [&](const T* p) {
    const int h = static_cast<int>((E - (reinterpret_cast<uintptr_t>(p) / sizeof(T)) % E) % E);
    return min(h, V);
  };
  // the thread's edge cell, -1: none
  auto edge_of = [&](int head, int nvec) {
    const int last = head + nvec * E;
    return tid < head ? tid : tid >= E && tid - E < V - last ? last + tid - E : -1;
  };
  auto load_vec = [&](const T* body, int v) { return *reinterpret_cast<const u32x4*>(body + v * E); };
  const int64_t row = blockIdx.x;
  const T* src = static_cast<const T*>(a.logits) + row * a.ldl;
  T* dst = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  const int32_t* ids = a.t_idx + row * a.k;
  const float* tl = a.t_logits + row * a.k;
  const float w = a.weight ? a.weight[row] : 1.0f;
  if (w == 0.0f) {       // a row that does not count: nothing of it is read
    if (MODE != kBackward && tid == 0) {
      a.loss[row] = 0.0f;
      if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
    }
    if (MODE != kLoss)
      for (int c = tid; c < V; c += THREADS) dst[c] = T(0);
    return;
  }
  const int head = head_of(src), nvec = (V - head) / E;
  const int edge = edge_of(head, nvec);
  // the gradient's row has its vectors at the same places
  const bool same = dst && head_of(dst) == head;
  u32x4 cell[NV > 0 ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + THREADS * i < nvec) cell[i] = load_vec(src + head, tid + THREADS * i);
  // ---- the teacher's side (first wave)
  // mask bits: the body's cells in order, then from `ebase` on the edges'
  const int ebase = (nvec * E + 31) / 32 * 32;
  for (int i = tid; i <= ebase / 32; i += THREADS) mask[i] = 0u;
  if (tid == 0) dup = 0;
  __syncthreads();
  double t_norm = 0.0, p_sum = 0.0, p_rest = 0.0;
  if (first) {
    float tm = -INFINITY;
    for (int i = lane; i < a.k; i += 64) {
      const int32_t id = ids[i];
      if (id < 0 || id >= V) continue;
      const int in = id - head;
      const unsigned b = unsigned(in < 0 ? ebase + id : in < nvec * E ? in : ebase + E + in - nvec * E);
      if ((atomicOr(&mask[b >> 5], 1u << (b & 31)) >> (b & 31)) & 1u) dup = 1;
      z_s[i] = cell_to_f32(src[id], DTag());
      tm = fmax_nan(tm, tl[i]);
    }
    if (tail) {
      t_norm = static_cast<double>(a.t_lse[row]);
    } else {
      tm = wave_all(tm, fmax_nan);
      double ts = 0.0;
      if (tm != -INFINITY)
        for (int i = lane; i < a.k; i += 64) {
          const int32_t id = ids[i];
          if (id < 0 || id >= V) continue;
          ts += dexp((double(tl[i]) - double(tm)) * a.inv_temp);
        }
      ts = wave_all(ts, sum2<double>);
      t_norm = double(tm) * a.inv_temp + dlog(ts);     // -inf where nothing is known
    }
    for (int i = lane; i < a.k; i += 64) {
      const int32_t id = ids[i];
      double p = 0.0;
      if (id >= 0 && id < V && tl[i] != -INFINITY) p = dexp(double(tl[i]) * a.inv_temp - t_norm);
      p_s[i] = p;
      p_sum += p;
    }
    p_sum = wave_all(p_sum, sum2<double>);
    if (tail) p_rest = p_sum >= 1.0 ? 0.0 : 1.0 - p_sum;   // NaN stays
  }
  if (tail) __syncthreads();           // the mask is whole
  // with a class for the rest, the cells of S leave the registers here
  auto take_out = [&](u32x4& v, int vi) {
    const uint32_t byte = E == 8 ? reinterpret_cast<const uint8_t*>(mask)[vi]
                                 : (reinterpret_cast<const uint8_t*>(mask)[vi >> 1] >> (4 * (vi & 1))) & 15u;
    if (byte) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if ((byte >> i) & 1u) set_bits<DT>(v, i, Cell<DT>::kNegInf);
    }
  };
  float ez = edge >= 0 ? cell_to_f32(src[edge], DTag()) : -INFINITY;   // the edge cell
  if (tail && edge >= 0 && ((mask[ebase / 32] >> tid) & 1u)) ez = -INFINITY;
  // ---- the student's side: maximum, then sum of 2^(cf z - refc), refc = cf
  //      max as rounded (its rounding is put back per row, below)
  float mx = -INFINITY, refc = 0.0f, cr = cf;
  double sum = 0.0;
  // A log-sum-exp far from 0 keeps too little of its sum in the fp32 stats (that
  // of the cells outside S also where they are masked by a low value; there it
  // may lie beyond fp32): the backward pass then forms both again.
  const bool fresh = MODE != kBackward || !(fabsf(a.stats[2 * row]) < kFarLse &&
                                            fabsf(a.stats[2 * row + 1]) < kFarLse);
  // Where cf mx is so large that its rounding matters, cells are equal or so
  // far apart that only the maximum counts: a power of two near cf does, whose
  // product is exact (and finite).
  auto refer = [&]() {
    refc = mx * cf;
    if (!(fabsf(refc) < 0x1p30f) && mx == mx) {
      cr = ldexpf(1.0f, min(ilogbf(cf), 125 - ilogbf(mx)));
      refc = mx * cr;
    }
  };
  if (fresh) {
    double own = 0.0;                  // the thread's cells
    if (NV > 0) {
      float part = 0.0f;
      float m = -INFINITY;
      if (E == 8) {
        // 16-bit cells order like integers as long as one is positive
        s16x2 m2 = s16x2{short(0x8000), short(0x8000)};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (tid + THREADS * i >= nvec) break;
          if (tail) take_out(cell[i], tid + THREADS * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t word = cell[i][e];
            m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(s16x2, word));
          }
        }
        const short top = m2[0] > m2[1] ? m2[0] : m2[1];
        const short own = max(top, static_cast<short>(ez == -INFINITY ? short(0x8000) : short(to_bits<DT>(ez))));
        m = block_all<THREADS>(static_cast<float>(own), redf, [](float x, float y) { return x > y ? x : y; });
        if (m >= 0.0f) {
          mx = cell_to_f32(static_cast<T>(static_cast<int>(m)), DTag());
        } else {                       // no positive cell (log-probabilities)
          float neg = ez;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (tid + THREADS * i >= nvec) break;
#pragma unroll
            for (int e = 0; e < E; ++e) neg = fmax_nan(neg, get_cell<DT>(cell[i], e));
          }
          mx = block_all<THREADS>(neg, redg, fmax_nan);
        }
      } else {
        m = ez;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (tid + THREADS * i >= nvec) break;
          if (tail) take_out(cell[i], tid + THREADS * i);
#pragma unroll
          for (int e = 0; e < E; ++e) m = fmax_nan(m, get_cell<DT>(cell[i], e));
        }
        mx = block_all<THREADS>(m, redf, fmax_nan);
      }
      // all cells -inf: nothing to exponentiate (the sum stays 0)
      if (mx != -INFINITY) {
        refer();
        if (edge >= 0) part = __builtin_amdgcn_exp2f(fmaf(ez, cr, -refc));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (tid + THREADS * i >= nvec) break;
#pragma unroll
          for (int e = 0; e < E; ++e)
            part += __builtin_amdgcn_exp2f(fmaf(get_cell<DT>(cell[i], e), cr, -refc));
        }
      }
      own = double(part);
    } else {
      float run = ez;
      if (run != -INFINITY) own = 1.0;
      for (int v = tid; v < nvec; v += THREADS) {
        u32x4 c = load_vec(src + head, v);
        if (tail) take_out(c, v);
        float m8 = run;
#pragma unroll
        for (int e = 0; e < E; ++e) m8 = fmax_nan(m8, get_cell<DT>(c, e));
        if (m8 == -INFINITY) continue;
        if (m8 != run) own *= double(__builtin_amdgcn_exp2f((run - m8) * cf));
        run = m8;
        float part = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
          part += __builtin_amdgcn_exp2f((get_cell<DT>(c, e) - run) * cf);
        own += double(part);
      }
      mx = block_all<THREADS>(run, redf, fmax_nan);
      if (run != -INFINITY) own *= double(__builtin_amdgcn_exp2f((run - mx) * cf));
      if (mx != -INFINITY) refer();
    }
    sum = block_all<THREADS>(own, redd, sum2<double>);
    if (NV == 0 && cr == cf && mx != -INFINITY) sum *= exp2(double(mx) * double(cf) - double(refc));
  }
  // ---- per row, first wave: log-sum-exps, loss, the gradient's factors
  if (first) {
    // Log-sum-exps as a cell's (mx, or top) share and the rest: lse = top / T +
    // l_all over the row, mx / T + l_rest over the cells outside S, so that
    // differences from them are exact however large the logits are.
    double top = 0.0, l_all, l_rest, between = 0.0;       // between: lse_rest - lse
    bool rest = true;                                     // the cells outside S have mass
    if (!fresh) {
      l_all = double(a.stats[2 * row]);
      l_rest = double(a.stats[2 * row + 1]);
      between = l_rest - l_all;
    } else {
      rest = mx != -INFINITY;
      // refc stands for cf mx up to its rounding
      l_rest = rest ? dlog(sum) - (cr == cf ? (double(mx) * double(cf) - double(refc)) * kLn2 : 0.0)
                    : -INFINITY;
      if (!tail) {
        top = double(mx);
        l_all = rest ? l_rest : NAN;     // NaN for a row without a finite cell
        rest = true;
      } else {
        // the known ids' share, on the larger of the two maxima
        float ms = mx;
        for (int i = lane; i < a.k; i += 64) {
          const int32_t id = ids[i];
          if (id >= 0 && id < V) ms = fmax_nan(ms, z_s[i]);
        }
        top = double(wave_all(ms, fmax_nan));
        double ss = 0.0;
        for (int i = lane; i < a.k; i += 64) {
          const int32_t id = ids[i];
          if (id < 0 || id >= V) continue;
          bool one = true;               // an id named twice has its mass once
          if (dup)
            for (int j = 0; j < i; ++j) one = one && ids[j] != id;
          if (one) ss += dexp((double(z_s[i]) - top) * a.inv_temp);
        }
        ss = wave_all(ss, sum2<double>);
        const double lead = (double(mx) - top) * a.inv_temp + l_rest;
        if (rest) ss += dexp(lead);
        l_all = dlog(ss);
        between = rest ? lead - l_all : -INFINITY;
      }
    }
    const bool use_rest = tail && !(p_rest <= 0.0) && rest;
    if (MODE != kBackward) {
      double t = 0.0;
      for (int i = lane; i < a.k; i += 64) {
        const double p = p_s[i];
        if (p != 0.0)
          t += p * ((double(tl[i]) * a.inv_temp - t_norm) - ((double(z_s[i]) - top) * a.inv_temp - l_all));
      }
      t = wave_all(t, sum2<double>);
      if (use_rest) t += p_rest * (dlog(p_rest) - between);
      // a row that knows nothing of the teacher has no loss, whatever it holds
      if (!tail && p_sum == 0.0) t = 0.0;
      if (lane == 0) {
        a.loss[row] = static_cast<float>(double(w) * a.temp * a.temp * t);
        if (a.stats) {
          a.stats[2 * row] = static_cast<float>(top * a.inv_temp + l_all);
          a.stats[2 * row + 1] = static_cast<float>(tail ? (rest ? double(mx) * a.inv_temp + l_rest : -INFINITY)
                                                         : top * a.inv_temp + l_all);
        }
      }
    }
    if (MODE != kLoss && lane == 0) {
      // A cell outside S: q_v (1 - p_r / q_r) = exp(z_v - lse_rest) (q_r - p_r):
      // no factor overflows where q_r is tiny.  A row that knows nothing of
      // the teacher has no gradient, as no loss.
      const double factor = (!tail && p_sum == 0.0)
                                ? 0.0
                                : double(w) * a.temp * (MODE == kBackward ? double(a.grad[row]) : 1.0);
      const double mass = tail && !use_rest ? p_sum : 1.0;   // sum of the target's classes
      double coef = 0.0;
      float rc = refc;
      if (rest) {
        coef = factor * (mass * dexp(between) - (use_rest ? p_rest : 0.0));
        if (fresh) {
          coef /= sum;
        } else {
          const double base = l_rest / kLn2;
          rc = static_cast<float>(base);
          coef *= exp2(double(rc) - base);
        }
      }
      sh_coef = static_cast<float>(coef);
      sh_refc = rest ? rc : 0.0f;
      sh_top = top;
      sh_lse = l_all;
      sh_factor = factor;
      sh_mass = mass;
    }
  }
  if (MODE == kLoss) return;
  __syncthreads();
  // ---- the gradient: first every cell as one outside S ...
  const float coef = sh_coef, rc = sh_refc;
  auto grad_vec = [&](const u32x4& c) {
    u32x4 g;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (DT == GPTQ_F32) {
        g[e] = to_bits<DT>(coef * __builtin_amdgcn_exp2f(fmaf(get_cell<DT>(c, e), cr, -rc)));
      } else {
        const uint32_t lo = to_bits<DT>(
            coef * __builtin_amdgcn_exp2f(fmaf(get_cell<DT>(c, (2 * e) % E), cr, -rc)));
        const uint32_t hi = to_bits<DT>(
            coef * __builtin_amdgcn_exp2f(fmaf(get_cell<DT>(c, (2 * e + 1) % E), cr, -rc)));
        g[e] = lo | (hi << 16);
      }
    }
    return g;
  };
  if (edge >= 0) {
    const uint32_t b = to_bits<DT>(
        coef * __builtin_amdgcn_exp2f(fmaf(cell_to_f32(src[edge], DTag()), cr, -rc)));
    if (DT == GPTQ_F32) reinterpret_cast<uint32_t*>(dst)[edge] = b;
    else reinterpret_cast<uint16_t*>(dst)[edge] = static_cast<uint16_t>(b);
  }
  if (NV > 0 && same) {
    u32x4* out = reinterpret_cast<u32x4*>(dst + head);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + THREADS * i;
      if (v < nvec) out[v] = grad_vec(cell[i]);
    }
  } else {                             // streamed, or the gradient lies otherwise: read again
    for (int v = tid; v < nvec; v += THREADS) {
      const u32x4 g = grad_vec(load_vec(src + head, v));
      if (same) {
        *reinterpret_cast<u32x4*>(dst + head + v * E) = g;
      } else {
        for (int e = 0; e < E; ++e) {
          if (DT == GPTQ_F32)
            reinterpret_cast<uint32_t*>(dst)[head + v * E + e] = g[e % 4];
          else
            reinterpret_cast<uint16_t*>(dst)[head + v * E + e] =
                static_cast<uint16_t>(g[(e >> 1) % 4] >> (16 * (e & 1)));
        }
      }
    }
  }
  // ... then the cells of S over it (entries of one id write the same value)
  __syncthreads();
  const double top_z = sh_top, lse = sh_lse, factor = sh_factor, mass = sh_mass;
  for (int i = tid; i < a.k; i += THREADS) {
    const int32_t id = ids[i];
    if (id < 0 || id >= V) continue;
    double p = p_s[i];
    if (dup) {
      p = 0.0;
      for (int j = 0; j < a.k; ++j)
        if (ids[j] == id) p += p_s[j];
    }
    const double g = factor * (mass * dexp((double(z_s[i]) - top_z) * a.inv_temp - lse) - p);
    const uint32_t b = to_bits<DT>(static_cast<float>(g));
    if (DT == GPTQ_F32) reinterpret_cast<uint32_t*>(dst)[id] = b;
    else reinterpret_cast<uint16_t*>(dst)[id] = static_cast<uint16_t>(b);
  }
}

template <int DT, int MODE>
gptq_status launch_mode(const DistillArgs& a, int64_t n, hipStream_t st) {
  constexpr int E = Cell<DT>::kPer;
  const int64_t nvec = (a.vocab + 2 * (E - 1)) / E;            // the most a row can take
  const size_t lds = (size_t((nvec * E + 31) / 32) + 2) * 4;
  // A row takes the fewest threads that hold it, so that several rows share a
  // CU; where every row has a CU to itself it takes more of them.  32000 bf16
  // cells: 4096 rows 122 us by 256 threads, 211 by 1024; 256 rows 18.8 and 16.2.
#define GPTQ_DISTILL(TH, NVV) \
  distill_kernel<DT, TH, NVV, MODE><<<unsigned(n), TH, lds, st>>>(a)
  if (nvec <= 256 * 4)
    GPTQ_DISTILL(256, 4);
  else if (nvec <= 1024 * 4 && n <= 256)
    GPTQ_DISTILL(1024, 4);
  else if (nvec <= 256 * 16)
    GPTQ_DISTILL(256, 16);
  else if (nvec <= 1024 * 8)
    GPTQ_DISTILL(512, 16);
  else if (nvec <= 1024 * 16)
    GPTQ_DISTILL(1024, 16);
  else
    GPTQ_DISTILL(1024, 0);
#undef GPTQ_DISTILL
  GPTQ_CHECK_LAUNCH();
  return GPTQ_OK;
}

template <int DT>
gptq_status launch_dt(const DistillArgs& a, int64_t n, hipStream_t st) {
  if (a.grad) return launch_mode<DT, kBackward>(a, n, st);
  return a.dlogits ? launch_mode<DT, kFused>(a, n, st) : launch_mode<DT, kLoss>(a, n, st);
}

}  // namespace

gptq_status launch_distill(const void* logits, gptq_dtype dt, int64_t n, int64_t vocab,
                           int64_t ldl, const int32_t* t_idx, const float* t_logits, int64_t k,
                           float temp, const float* t_lse, const float* weight,
                           const float* grad, float* loss, float* stats, void* dlogits,
                           int64_t ldd, hipStream_t st) {
  if (n == 0) return GPTQ_OK;
  const DistillArgs a{logits, vocab, ldl, t_idx, t_logits, static_cast<int>(k), 1.0 / double(temp),
                      temp, t_lse, weight, grad, loss, stats, dlogits, ldd};
  switch (dt) {
    case GPTQ_F32: return launch_dt<GPTQ_F32>(a, n, st);
    case GPTQ_BF16: return launch_dt<GPTQ_BF16>(a, n, st);
    case GPTQ_F16: return launch_dt<GPTQ_F16>(a, n, st);
  }
  return GPTQ_ERR_INVALID_ARG;
}

}  // namespace gptq
