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
// outside S get w T q_v (1 - p_r / q_r).
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
// fp32 per thread (at most 128 terms), in fp64 across threads, in a fixed
// order: results are the same bits from run to run.
#include "common.h"

namespace gptq {
namespace {

constexpr int kMaxK = kDistillMaxK;
constexpr float kLog2e = 1.44269504088896340736f;

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

// Sum (or maximum) over the workgroup, the same value in every thread.
template <int THREADS, class T, class F>
__device__ inline T block_all(T v, T* red, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
  __syncthreads();                       // red is free
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

enum { kLoss = 0, kFused = 1, kBackward = 2 };

// NV vectors of 16 bytes per thread held in registers; NV = 0: the row is
// streamed (and read again for the gradient).
template <int DT, int THREADS, int NV, int MODE>
__global__ __launch_bounds__(THREADS) void distill_kernel(DistillArgs a) {
  using T = typename Cell<DT>::type;
  using DTag = std::integral_constant<int, DT>;
  constexpr int E = Cell<DT>::kPer;
  extern __shared__ uint32_t mask[];     // one bit per cell, aligned as the vectors are
  __shared__ double p_s[kMaxK];          // teacher's probability of entry i (0: padding)
  __shared__ float z_s[kMaxK];           // student's logit of entry i
  __shared__ double redd[THREADS / 64];
  __shared__ float redf[THREADS / 64];
  __shared__ int dup;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* src = static_cast<const T*>(a.logits) + row * a.ldl;
  T* dst = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
  const int V = static_cast<int>(a.vocab);
  const int32_t* ids = a.t_idx + row * a.k;
  const float* tl = a.t_logits + row * a.k;
  const float w = a.weight ? a.weight[row] : 1.0f;
  // vector v covers cells v E - off .. + E - 1, 16-byte aligned in logits
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(src) / sizeof(T)) % E);
  const int nvec = (V + off + E - 1) / E;
  // the gradient's row has its vectors at the same places
  const bool same = dst && (reinterpret_cast<uintptr_t>(dst) / sizeof(T)) % E == unsigned(off);

  auto store_vec = [&](int e0, const u32x4& v) {
    if (same && e0 >= 0 && e0 + E <= V) {
      *reinterpret_cast<u32x4*>(dst + e0) = v;
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (e0 + i < 0 || e0 + i >= V) continue;
        if (DT == GPTQ_F32)
          reinterpret_cast<uint32_t*>(dst)[e0 + i] = v[i % 4];
        else
          reinterpret_cast<uint16_t*>(dst)[e0 + i] =
              static_cast<uint16_t>(v[(i >> 1) % 4] >> (16 * (i & 1)));
      }
    }
  };
  if (w == 0.0f) {       // a row that does not count: nothing of it is read
    if (MODE != kBackward && tid == 0) {
      a.loss[row] = 0.0f;
      if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
    }
    if (MODE != kLoss)
      for (int v = tid; v < nvec; v += THREADS) store_vec(v * E - off, u32x4{0u, 0u, 0u, 0u});
    return;
  }
  const bool tail = a.t_lse != nullptr;
  // ---- the cells, a vector partly outside the row filled with -inf
  auto load_vec = [&](int e0) {
    u32x4 v;
    if (e0 >= 0 && e0 + E <= V) {
      v = *reinterpret_cast<const u32x4*>(src + e0);
    } else {
      constexpr uint32_t f = DT == GPTQ_F32 ? Cell<DT>::kNegInf
                                            : Cell<DT>::kNegInf | (Cell<DT>::kNegInf << 16);
      v = u32x4{f, f, f, f};
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e0 + i >= 0 && e0 + i < V) {
          const T c = src[e0 + i];
          uint32_t bits;
          if (DT == GPTQ_F32) bits = __builtin_bit_cast(uint32_t, static_cast<float>(c));
          else bits = static_cast<uint32_t>(c);
          set_bits<DT>(v, i, bits);
        }
    }
    return v;
  };
  u32x4 cell[NV > 0 ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + THREADS * i;
    if (v < nvec) cell[i] = load_vec(v * E - off);
  }
  // ---- the teacher's side
  for (int i = tid; i < (nvec * E + 31) / 32; i += THREADS) mask[i] = 0u;
  if (tid == 0) dup = 0;
  __syncthreads();
  float tm = -INFINITY;
  for (int i = tid; i < a.k; i += THREADS) {
    const int32_t id = ids[i];
    if (id < 0 || id >= V) continue;
    const unsigned b = unsigned(id + off);
    if ((atomicOr(&mask[b >> 5], 1u << (b & 31)) >> (b & 31)) & 1u) dup = 1;
    z_s[i] = cell_to_f32(src[id], DTag());
    tm = fmax_nan(tm, tl[i]);
  }
  double t_norm;
  if (tail) {
    t_norm = static_cast<double>(a.t_lse[row]);
    __syncthreads();
  } else {
    tm = block_all<THREADS>(tm, redf, fmax_nan);
    double ts = 0.0;
    if (tm != -INFINITY)
      for (int i = tid; i < a.k; i += THREADS) {
        const int32_t id = ids[i];
        if (id < 0 || id >= V) continue;
        ts += exp((double(tl[i]) - double(tm)) * a.inv_temp);
      }
    ts = block_all<THREADS>(ts, redd, sum2<double>);
    t_norm = double(tm) * a.inv_temp + log(ts);     // -inf where nothing is known
  }
  // probabilities; entries of one id more than once (dup) count each, and
  // the first of them stands for the id where the student's mass is summed
  auto first_of_id = [&](int i) {
    if (!dup) return true;
    for (int j = 0; j < i; ++j)
      if (ids[j] == ids[i]) return false;
    return true;
  };
  double p_sum = 0.0;
  for (int i = tid; i < a.k; i += THREADS) {
    const int32_t id = ids[i];
    double p = 0.0;
    if (id >= 0 && id < V && tl[i] != -INFINITY) p = exp(double(tl[i]) * a.inv_temp - t_norm);
    p_s[i] = p;
    p_sum += p;
  }
  p_sum = block_all<THREADS>(p_sum, redd, sum2<double>);
  double p_rest = 0.0;
  if (tail) p_rest = p_sum >= 1.0 ? 0.0 : 1.0 - p_sum;   // NaN stays
  // ---- the student's side
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
  const float cf = static_cast<float>(a.inv_temp) * kLog2e;
  double lse, lse_rest;
  float ref = 0.0f;                      // the gradient's exponentials are of (logit - ref) / T
  if (MODE == kBackward) {
    lse = double(a.stats[2 * row]);
    lse_rest = double(a.stats[2 * row + 1]);
  } else {
    float mx = -INFINITY;
    float sum = 0.0f;
    if (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + THREADS * i;
        if (v >= nvec) break;
        if (tail) take_out(cell[i], v);
#pragma unroll
        for (int e = 0; e < E; ++e) mx = fmax_nan(mx, get_cell<DT>(cell[i], e));
      }
      mx = block_all<THREADS>(mx, redf, fmax_nan);
      // all cells -inf: nothing to exponentiate (the sum stays 0)
      if (mx != -INFINITY) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (tid + THREADS * i >= nvec) break;
#pragma unroll
          for (int e = 0; e < E; ++e)
            sum += __builtin_amdgcn_exp2f((get_cell<DT>(cell[i], e) - mx) * cf);
        }
      }
    } else {
      float run = -INFINITY;
      for (int v = tid; v < nvec; v += THREADS) {
        u32x4 c = load_vec(v * E - off);
        if (tail) take_out(c, v);
        float m8 = run;
#pragma unroll
        for (int e = 0; e < E; ++e) m8 = fmax_nan(m8, get_cell<DT>(c, e));
        if (m8 == -INFINITY) continue;
        if (m8 != run) sum *= __builtin_amdgcn_exp2f((run - m8) * cf);
        run = m8;
#pragma unroll
        for (int e = 0; e < E; ++e)
          sum += __builtin_amdgcn_exp2f((get_cell<DT>(c, e) - run) * cf);
      }
      mx = block_all<THREADS>(run, redf, fmax_nan);
      if (run != -INFINITY) sum *= __builtin_amdgcn_exp2f((run - mx) * cf);
    }
    const double s = block_all<THREADS>(double(sum), redd, sum2<double>);
    if (!tail) {
      ref = mx;
      lse = double(mx) * a.inv_temp + log(s);       // NaN for a row without a finite cell
      lse_rest = lse;
    } else {
      lse_rest = mx == -INFINITY ? -INFINITY : double(mx) * a.inv_temp + log(s);
      ref = mx == -INFINITY ? 0.0f : mx;
      // the known ids' share, on the larger of the two maxima
      float ms = mx;
      for (int i = tid; i < a.k; i += THREADS) {
        const int32_t id = ids[i];
        if (id >= 0 && id < V) ms = fmax_nan(ms, z_s[i]);
      }
      const float top = block_all<THREADS>(ms, redf, fmax_nan);
      double ss = 0.0;
      for (int i = tid; i < a.k; i += THREADS) {
        const int32_t id = ids[i];
        if (id >= 0 && id < V && first_of_id(i)) ss += exp((double(z_s[i]) - double(top)) * a.inv_temp);
      }
      ss = block_all<THREADS>(ss, redd, sum2<double>);
      if (mx != -INFINITY) ss += s * exp((double(mx) - double(top)) * a.inv_temp);
      lse = double(top) * a.inv_temp + log(ss);
    }
  }
  const bool use_rest = tail && !(p_rest <= 0.0) && lse_rest != -INFINITY;
  if (MODE != kBackward) {
    double t = 0.0;
    for (int i = tid; i < a.k; i += THREADS) {
      const double p = p_s[i];
      if (p != 0.0)
        t += p * ((double(tl[i]) * a.inv_temp - t_norm) - (double(z_s[i]) * a.inv_temp - lse));
    }
    t = block_all<THREADS>(t, redd, sum2<double>);
    if (use_rest) t += p_rest * (log(p_rest) - (lse_rest - lse));
    if (tid == 0) {
      a.loss[row] = static_cast<float>(double(w) * a.temp * a.temp * t);
      if (a.stats) {
        a.stats[2 * row] = static_cast<float>(lse);
        a.stats[2 * row + 1] = static_cast<float>(lse_rest);
      }
    }
  }
  if (MODE == kLoss) return;
  // ---- the gradient: first every cell as one outside S, q_v (1 - p_r / q_r)
  // = exp(z_v - lse_rest) (q_r - p_r): no factor overflows where q_r is tiny.
  // A row that knows nothing of the teacher has no gradient, as no loss.
  const double factor = (!tail && !(p_sum > 0.0) && p_sum == p_sum)
                            ? 0.0
                            : double(w) * a.temp * (MODE == kBackward ? double(a.grad[row]) : 1.0);
  const double base = tail ? lse_rest : lse;      // the log-sum-exp that ref goes with
  double coef_d = 0.0;
  if (base != -INFINITY) {
    coef_d = factor * (exp(base - lse) - (use_rest ? p_rest : 0.0));
    if (MODE != kBackward) coef_d *= exp(double(ref) * a.inv_temp - base);
  }
  const float coef = static_cast<float>(coef_d);
  const float base_f = base == -INFINITY ? 0.0f : static_cast<float>(base);
  const float it = static_cast<float>(a.inv_temp);
  auto grad_vec = [&](const u32x4& c) {
    u32x4 g = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float z = get_cell<DT>(c, e);
      const float x = MODE == kBackward ? fmaf(z, it, -base_f) * kLog2e : (z - ref) * cf;
      const uint32_t b = to_bits<DT>(coef * __builtin_amdgcn_exp2f(x));
      if (DT == GPTQ_F32) g[e % 4] = b;
      else g[(e >> 1) % 4] |= b << (16 * (e & 1));
    }
    return g;
  };
  if (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + THREADS * i;
      if (v >= nvec) break;
      store_vec(v * E - off, grad_vec(cell[i]));
    }
  } else {
    for (int v = tid; v < nvec; v += THREADS) store_vec(v * E - off, grad_vec(load_vec(v * E - off)));
  }
  // ... then the cells of S over it (entries of one id write the same value)
  __syncthreads();
  for (int i = tid; i < a.k; i += THREADS) {
    const int32_t id = ids[i];
    if (id < 0 || id >= V) continue;
    double p = p_s[i];
    if (dup) {
      p = 0.0;
      for (int j = 0; j < a.k; ++j)
        if (ids[j] == id) p += p_s[j];
    }
    const double g = factor * (exp(double(z_s[i]) * a.inv_temp - lse) - p);
    const uint32_t b = to_bits<DT>(static_cast<float>(g));
    if (DT == GPTQ_F32) reinterpret_cast<uint32_t*>(dst)[id] = b;
    else reinterpret_cast<uint16_t*>(dst)[id] = static_cast<uint16_t>(b);
  }
}

template <int DT, int MODE>
gptq_status launch_mode(const DistillArgs& a, int64_t n, hipStream_t st) {
  constexpr int E = Cell<DT>::kPer;
  const int64_t nvec = (a.vocab + 2 * (E - 1)) / E;            // the most a row can take
  const size_t lds = size_t((nvec * E + 31) / 32) * 4;
  const unsigned grid = static_cast<unsigned>(n);
#define GPTQ_DISTILL(TH, NVV) \
  distill_kernel<DT, TH, NVV, MODE><<<grid, TH, lds, st>>>(a)
  if (nvec <= 256 * 4)
    GPTQ_DISTILL(256, 4);
  else if (nvec <= 1024 * 4)
    GPTQ_DISTILL(1024, 4);
  else if (nvec <= 1024 * 8)
    GPTQ_DISTILL(1024, 8);
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
