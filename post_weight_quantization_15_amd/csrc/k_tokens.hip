// What a row of logits says about a token: its log probability, the entropy of
// the row's distribution, its log-sum-exp, and the row's largest logits with
// their ids; and the gradient of the first two.
//
// With z = x / T, one pass over the row: s = sum 2^(c (x - r)) and t = sum c (x
// - r) 2^(c (x - r)), c = log2(e) / T, r a reference that a wave takes from its
// own first cells and moves only for a cell far above it; then
//   lse = r / T + ln s,  log p = (x_v - r) / T - ln s,
//   entropy = ln s - ln2 t / s
// (all terms of one sign, so nothing cancels).  Cells are exponentiated in fp32
// and summed in fp32 for 32 cells of a thread, in fp64 beyond.
//
// The largest k: cells pass a bar that only rises.  The first cells' bar is the
// smallest, over the waves, of the (k / waves)-th largest of the lanes' maxima
// (so at least k cells reach it); what passes is kept in LDS as (value, lower
// id first) in one 64-bit number, all different, and once more than k are there the
// k-th of them is the new bar.  A cell later in the row has to exceed it: an
// equal one has the higher id.  In a row without order some k ln(vocab) cells pass, so the selection
// is a comparison per 16 bytes; a row that rises all along fills the LDS
// again and again and is sorted there each time (correct, and slow).
#include <type_traits>

#include "lora.h"

namespace gptq {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kGroup = 4;                    // steps between two looks at the candidates
constexpr int kCap = 8192;                   // candidates in LDS
constexpr int kByRank = 1024;                // as many are ranked by counting, more sorted
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

// The larger of three, numbers before NaN.
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
__device__ inline uint64_t entry_of(float x, int id) {
  return uint64_t(order_of(x)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

template <class T, class F>
__device__ inline T wave_all(T v, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o));
  return v;
}

// The k largest of buf[0 .. count), in order, at its front; all threads call it,
// with buf written and a barrier behind that.  Returns how many there are.
__device__ __attribute__((noinline)) int select_top(uint64_t* buf, int count, int k) {
  const int tid = threadIdx.x;
  if (count <= kByRank) {
    const uint64_t a0 = tid < count ? buf[tid] : 0u;
    const uint64_t a1 = tid + kThreads < count ? buf[tid + kThreads] : 0u;
    int r0 = 0, r1 = 0;
    if ((tid & ~63) < count) {               // waves without a candidate wait below
      if (count <= kThreads) {
#pragma unroll 8
        for (int i = 0; i < count; ++i) r0 += buf[i] > a0;
      } else {
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
          const uint64_t v = buf[i];
          r0 += v > a0;
          r1 += v > a1;
        }
      }
    }
    __syncthreads();
    if (tid < count && r0 < k) buf[r0] = a0;
    if (tid + kThreads < count && r1 < k) buf[r1] = a1;
    __syncthreads();
    return min(count, k);
  }
  int size = 2 * kByRank;
  while (size < count) size *= 2;
  for (int i = count + tid; i < size; i += kThreads) buf[i] = 0u;
  __syncthreads();
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step > 0; step /= 2) {
      for (int p = tid; p < size / 2; p += kThreads) {
        const int i = 2 * p - (p & (step - 1)), j = i + step;
        const uint64_t a = buf[i], b = buf[j];
        if ((a < b) == ((i & run) == 0)) {
          buf[i] = b;
          buf[j] = a;
        }
      }
      __syncthreads();
    }
  return min(count, k);
}

struct TokenArgs {
  const void* logits;
  int64_t ldl;
  int vocab, k, parts, span;                 // a part: span cells of a row
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

// What the row's sums say; one thread.
template <int DT>
__device__ inline void finish_row(const TokenArgs& a, int64_t row, double ref, double s, double t) {
  double lse, rest, h;
  if (s == 0.0) {                            // nothing but -inf
    lse = rest = -INFINITY;
    h = __longlong_as_double(0x7FF8000000000000ll);
  } else {
    rest = log(s);
    lse = ref * a.inv_temp + rest;
    h = rest - kLn2 * (t / s);
  }
  if (a.logp) {
    const int id = a.token ? a.token[row] : -1;
    double lp = 0.0;
    if (id >= 0 && id < a.vocab) {
      const float x = to_f32<DT>(static_cast<const typename Cells<DT>::type*>(a.logits)[row * a.ldl + id]);
      lp = s == 0.0 ? h : (double(x) - ref) * a.inv_temp - rest;
    }
    a.logp[row] = static_cast<float>(lp);
  }
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
    const bool some = e >> 32;
    a.top[row * a.k + i] = some ? value_of(static_cast<uint32_t>(e >> 32)) : -INFINITY;
    a.idx[row * a.k + i] = some ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(e)) : -1;
  }
}

// Sums relative to reference r moved to a higher one.
__device__ inline void move_sums(double& s, double& t, double up) {
  up = up < 1000.0 ? up : 1000.0;
  const double f = exp2(-up);
  t = f * (t - up * s);
  s *= f;
}

template <int DT>
__global__ __launch_bounds__(kThreads, 4) void tokens_kernel(TokenArgs a) {
  using T = typename Cells<DT>::type;
  constexpr int E = Cells<DT>::kPer, NV = Cells<DT>::kVec;
  constexpr int kSteps = kThreads * NV;      // vectors of a step
  extern __shared__ __attribute__((aligned(16))) uint64_t buf[];
  __shared__ double red[3][kWaves];
  __shared__ float bars[kWaves];
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
  const float margin = 40.0f / c;
  const int steps = (nvec + kSteps - 1) / kSteps;
  const T* body = src + head;

  u32x4 cur[kGroup][NV], nxt[kGroup][NV];
  auto load = [&](u32x4 (&v)[kGroup][NV], int step) {
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (step + u) * kSteps + i * kThreads + tid;
        if (at < nvec) v[u][i] = *reinterpret_cast<const u32x4*>(body + int64_t(at) * E);
      }
  };
  load(cur, 0);
  if (tid == 0) cnt = 0;
  float ez = -INFINITY;
  if (edge >= 0) ez = to_f32<DT>(src[edge]);
  __syncthreads();
  int have = 0;                              // candidates: the edges, to begin with
  if (a.k) {
    const bool some = edge >= 0 && ez == ez;
    if (some) buf[atomicAdd(&cnt, 1)] = entry_of(ez, first + edge);
    have = __syncthreads_count(some);
  }
  float bar = -INFINITY;                     // cells from here up are candidates
  float ref = kLowest;
  double s = 0.0, t = 0.0;                   // of this thread, relative to ref
  // candidates among the vectors of one step (past the buffer's end: counted only)
  auto push = [&](const u32x4& v, int at) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = cell_of<DT>(v, e);
      if (x >= bar) {
        const int p = atomicAdd(&cnt, 1);
        if (p < kCap) buf[p] = entry_of(x, first + head + at * E + e);
      }
    }
  };
  // the bar after a selection
  auto raise = [&]() {
    if (have >= a.k) bar = value_of(static_cast<uint32_t>(buf[a.k - 1] >> 32) + 1u);
  };

  for (int step = 0; step == 0 || step < steps; step += kGroup) {
    if (step + kGroup < steps) load(nxt, step + kGroup);
    // ---- the largest cells of each vector
    float top[kGroup][NV], gm = step == 0 ? ez : -INFINITY;
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (step + u) * kSteps + i * kThreads + tid;
        float m = -INFINITY;
        if (at < nvec) {
#pragma unroll
          for (int e = 0; e < E; e += 2) m = max3(m, cell_of<DT>(cur[u][i], e), cell_of<DT>(cur[u][i], e + 1));
        }
        top[u][i] = m;
        gm = fmaxf(gm, m);
      }
    if (__any(gm > ref + margin)) {
      const float up = wave_all(gm, [](float x, float y) { return fmaxf(x, y); });
      move_sums(s, t, double(c) * (double(up) - double(ref)));
      ref = up;
    }
    // ---- sums
    float ps = 0.0f, pt = 0.0f;
    auto add_cell = [&](float x) {
      float d = (x - ref) * c;
      const float e = __builtin_amdgcn_exp2f(d);
      d = max3(d, -1000.0f, -1000.0f);       // 0 times -inf
      ps += e;
      pt = fmaf(e, d, pt);
    };
    if (step == 0 && edge >= 0) add_cell(ez);
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (step + u) * kSteps + i * kThreads + tid;
        if (at < nvec) {
#pragma unroll
          for (int e = 0; e < E; ++e) add_cell(cell_of<DT>(cur[u][i], e));
        }
      }
    s += ps;
    t += pt;
    // ---- candidates
    if (a.k) {
      if (step == 0) {
        // this wave's (k / waves)-th largest of the lanes' maxima
        const int want = (a.k + kWaves - 1) / kWaves;
        float low = -INFINITY;
        if (want <= 64) {
          const uint32_t key = order_of(gm);
          int rank = 0;
#pragma unroll
          for (int l = 0; l < 64; ++l) {
            const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), l));
            rank += o > key || (o == key && l < lane);
          }
          const uint64_t at = __ballot(rank == want - 1);
          const uint32_t pick = static_cast<uint32_t>(
              __builtin_amdgcn_readlane(static_cast<int>(key), __builtin_ctzll(at)));
          low = pick ? value_of(pick) : -INFINITY;
        }
        if (lane == 0) bars[wv] = low;
        __syncthreads();
        bar = bars[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) bar = fminf(bar, bars[w]);
      }
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (top[u][i] >= bar) {
            const int at = (step + u) * kSteps + i * kThreads + tid;
            if (at < nvec) push(cur[u][i], at);
          }
      __syncthreads();
      const int found = cnt;
      __syncthreads();
      if (found > kCap) {
        // too many at once: a step at a time, each in room for all its cells
        for (int u = step; u < min(step + kGroup, steps); ++u) {
          if (tid == 0) cnt = have;
          __syncthreads();
          for (int i = 0; i < NV; ++i) {
            const int at = u * kSteps + i * kThreads + tid;
            if (at < nvec) push(*reinterpret_cast<const u32x4*>(body + int64_t(at) * E), at);
          }
          __syncthreads();
          const int now = cnt;
          __syncthreads();
          have = select_top(buf, now, a.k);
          raise();
          __syncthreads();
        }
        if (tid == 0) cnt = have;
        __syncthreads();
      } else if (found > a.k + 64 || step + kGroup >= steps) {
        have = select_top(buf, found, a.k);
        raise();
        if (tid == 0) cnt = have;
        __syncthreads();
      } else {
        have = found;
      }
    }
#pragma unroll
    for (int u = 0; u < kGroup; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) cur[u][i] = nxt[u][i];
  }
  // ---- the waves' sums, moved to the highest reference
  s = wave_all(s, [](double x, double y) { return x + y; });
  t = wave_all(t, [](double x, double y) { return x + y; });
  if (lane == 0) {
    red[0][wv] = ref;
    red[1][wv] = s;
    red[2][wv] = t;
  }
  __syncthreads();
  if (tid == 0) {
    double r = kLowest, S = 0.0, Tt = 0.0;
    for (int w = 0; w < kWaves; ++w) r = red[0][w] > r ? red[0][w] : r;
    for (int w = 0; w < kWaves; ++w) {
      double ws = red[1][w], wt = red[2][w];
      if (red[0][w] < r) move_sums(ws, wt, double(c) * (r - red[0][w]));
      S += ws;
      Tt += wt;
    }
    if (a.parts == 1) {
      finish_row<DT>(a, row, r, S, Tt);
    } else {
      double* o = a.part_sums + (row * a.parts + part) * 3;
      o[0] = r;
      o[1] = S;
      o[2] = Tt;
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
  __shared__ int cnt;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint64_t* in = a.part_top + row * a.parts * a.k;
  if (tid == 0) cnt = 0;
  uint64_t bar = ~uint64_t(0);
  if (a.k) {
    // every part has (k / parts) entries from its own such entry up
    const int want = (a.k + a.parts - 1) / a.parts;
    if ((tid & 63) < a.parts) bar = in[(tid & 63) * a.k + want - 1];
    bar = wave_all(bar, [](uint64_t x, uint64_t y) { return x < y ? x : y; });
  }
  __syncthreads();
  if (a.k) {
    for (int i = tid; i < a.parts * a.k; i += kThreads) {
      const uint64_t e = in[i];
      if (e && e >= bar) buf[atomicAdd(&cnt, 1)] = e;
    }
    __syncthreads();
    const int found = cnt;
    const int have = select_top(buf, found, a.k);
    write_top(a, row, buf, have);
  }
  if (tid == 0) {
    const double* p = a.part_sums + row * a.parts * 3;
    const double c = double(static_cast<float>(a.inv_temp) * kLog2e);
    double r = kLowest, S = 0.0, Tt = 0.0;
    for (int w = 0; w < a.parts; ++w) r = p[3 * w] > r ? p[3 * w] : r;
    for (int w = 0; w < a.parts; ++w) {
      double ws = p[3 * w + 1], wt = p[3 * w + 2];
      if (p[3 * w] < r) move_sums(ws, wt, c * (r - p[3 * w]));
      S += ws;
      Tt += wt;
    }
    finish_row<DT>(a, row, r, S, Tt);
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

// Parts of a row: enough workgroups for the chip where rows are few, of 4096
// cells (8 a thread) at least, their candidates within the join's LDS.
int parts_of(int64_t n, int64_t vocab, int64_t k) {
  int64_t p = std::min<int64_t>(512 / std::max<int64_t>(n, 1), (vocab + 4095) / 4096);
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
  const size_t lds = a.k ? size_t(kCap) * 8 : 0;
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
  if (n == 0) return GPTQ_OK;
  Carver c(ws);
  const TokenWs w = carve_tokens(c, n, vocab, k);
  TokenArgs a{logits, ldl, int(vocab), int(k), parts_of(n, vocab, k), 0, 1.0 / double(temp), token,
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
  if (n == 0) return GPTQ_OK;
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
