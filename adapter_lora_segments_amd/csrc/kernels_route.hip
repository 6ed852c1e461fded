// Routing of rows to experts and its gradient.
//
// A row's logits lie in the registers of L lanes, V neighbours each (64 / L
// rows a wave), so every step over the experts is V operations for all the
// wave's rows at once and every sum or maximum log2(L) lane exchanges.  Many
// rows take few lanes each (work per row counts), few rows many (latency does).
// Scores are computed in 64 bits, which the vector units run at the rate of
// 32, and rounded to fp32 once: two programs then agree on every choice but
// for scores within 2^-45 of a rounding border.  A choice compares (score +
// bias in fp32, expert from behind) as one whole number below 2^44, held
// exactly in a double, so a step of the top_k is a maximum, and ties go to the
// lowest expert.
#include "device_common.hpp"
#include "route.hpp"

namespace mlora {

namespace {

// Threads of a workgroup: rows of many experts come one to a workgroup, so that
// their scores fit into LDS.
template <int V>
constexpr int kThreads = V > 16 ? 64 : 256;

constexpr float kNone = -__builtin_inff();

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }

// e^x in 64 bits for x <= 0: x = n ln 2 + r, |r| <= ln 2 / 2, the Taylor series
// of e^r to r^11 (the next term is below 2^-47).  NaN stays.
__device__ __forceinline__ double exp64(double x) {
  const double c = x < -800.0 ? -800.0 : x;          // zero, also of -infinity
  const double n = __builtin_rint(c * 1.4426950408889634);
  double r = __builtin_fma(n, -0.6931471805599453, c);
  r = __builtin_fma(n, -2.3190468138462996e-17, r);
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}
// 1 / x for x in [1, 2]: the hardware's approximation and two Newton steps (its
// error is squared by each).
__device__ __forceinline__ double reciprocal(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-x, r, 1.0), r, r);
}
__device__ __forceinline__ double sigmoid64(float x) {
  const double t = exp64(-__builtin_fabs((double)x)), r = reciprocal(1.0 + t);
  return x < 0.f ? t * r : r;
}

// Exchanges within L lanes.  Each step pairs groups that already agree, so any
// lane of the other group will do: within 16 lanes DPP moves, then swaps of
// rows.
template <int STEP>
__device__ __forceinline__ uint32_t other(uint32_t v) {
  if constexpr (STEP == 1) return __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);         // quad 1 0 3 2
  else if constexpr (STEP == 2) return __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);    // quad 2 3 0 1
  else if constexpr (STEP == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);   // mirror of 8
  else if constexpr (STEP == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);   // mirror of 16
  else return __shfl_xor((int)v, STEP);
}
template <int STEP>
__device__ __forceinline__ double other(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = other<STEP>((uint32_t)b), hi = other<STEP>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int STEP>
__device__ __forceinline__ float other(float v) {
  return __uint_as_float(other<STEP>(__float_as_uint(v)));
}
// max and min of keys (no NaN among them)
__device__ __forceinline__ double key_max(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double key_min(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
template <int L, int STEP = 1, class T, class OP>
__device__ __forceinline__ T across(T v, OP op) {
  if constexpr (STEP < L) return across<L, 2 * STEP>(op(v, other<STEP>(v)), op);
  else return v;
}
template <int L>
__device__ __forceinline__ double group_sum(double v) {
  return across<L>(v, [](double a, double b) { return a + b; });
}

// Ordered 32-bit image of a score that may be chosen: rises with it, NaN last
// (chosen first, so that it shows), never 0.
__device__ __forceinline__ uint32_t ordered(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return c != c ? 0xffffffffu : u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

// A row's softmax terms: its maximum and the reciprocal of the sum of e^(x - max).
struct Soft {
  double top, inv;
};
__device__ __forceinline__ double score_of(const RouteArgs& a, const Soft& s, float x) {
  if (x == kNone) return 0.0;
  if (a.sigmoid) return sigmoid64(x);
  return exp64((double)x - s.top) * s.inv;
}
// e[v] = e^(x - max), zero at -infinity
template <int L, int V>
__device__ __forceinline__ Soft softmax_terms(const float (&x)[V], double (&e)[V]) {
  float m = kNone;
#pragma unroll
  for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
  m = across<L>(m, [](float a, float b) { return fmaxf(a, b); });
  Soft s;
  s.top = m == kNone ? 0.0 : (double)m;
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = x[v] == kNone ? 0.0 : exp64((double)x[v] - s.top);
    sum += e[v];
  }
  sum = group_sum<L>(sum);
  s.inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  return s;
}

// Lane `sub`'s experts sub V .. of a row (-infinity past the last); whole: all
// lanes are full and 16-byte aligned.
template <class T, int V>
__device__ __forceinline__ void load_row(const T* p, int E, int sub, bool whole, float (&x)[V]) {
  constexpr int P = 16 / sizeof(T);
  if constexpr (V % P == 0) {
    if (whole) {
#pragma unroll
      for (int i = 0; i < V / P; ++i) {
        const u32x4 u = reinterpret_cast<const u32x4*>(p + sub * V)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            x[4 * i + j] = __uint_as_float(u[j]);
          } else {
            x[8 * i + 2 * j] = __uint_as_float(u[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = sub * V + v;
    x[v] = e < E ? load_logit(p + e) : kNone;
  }
}

// Compare and exchange: the larger key to a.
__device__ __forceinline__ void order2(double& a, double& b) {
  const double hi = key_max(a, b);
  b = key_min(a, b);
  a = hi;
}
// Eight keys to falling order (odd-even merge sort, 19 exchanges).
__device__ __forceinline__ void sort8(double* k) {
  constexpr int pairs[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int i = 0; i < 19; ++i) order2(k[pairs[i][0]], k[pairs[i][1]]);
}
// A bitonic eight to falling order.
__device__ __forceinline__ void merge8(double (&k)[8]) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order2(k[i], k[i + d]);
}
// The eight largest keys of a row to all of its lanes, falling: every lane
// sorts its own by eights, keeps the upper half of two sorted eights (the
// larger of first and last, second and last but one, ..., a bitonic eight), and
// so do pairs of lanes.
template <int L, int STEP = 1>
__device__ __forceinline__ void across8(double (&k)[8]) {
  if constexpr (STEP < L) {
    double o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = other<STEP>(k[7 - i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = key_max(k[i], o[i]);
    merge8(k);
    across8<L, 2 * STEP>(k);
  }
}
template <int L, int V>
__device__ __forceinline__ void top8(double (&key)[V], double (&k)[8]) {
  static_assert(V % 8 == 0, "whole eights");
#pragma unroll
  for (int h = 0; h < V / 8; ++h) {
    sort8(key + 8 * h);
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) k[i] = key[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) k[i] = key_max(k[i], key[8 * h + 7 - i]);
      merge8(k);
    }
  }
  across8<L>(k);
}

__device__ __forceinline__ int expert_of(double key) {
  const double whole = __builtin_floor(key * (1.0 / 4096.0));
  return key >= 1.0 ? 4095 - (int)__builtin_fma(-4096.0, whole, key) : -1;
}

}  // namespace

// LDS of a row: the chosen ids [top_k]; with expert groups, per run of min(V,
// group) experts its two largest ordered scores, and the groups' scores.
template <class T, int L, int V>
__global__ __launch_bounds__(kThreads<V>) void k_route(RouteArgs a, int whole, int bias_whole) {
  extern __shared__ int lds[];
  constexpr int R = kThreads<V> / L, CS = V > 1 ? 2 : 1;
  const int sub = threadIdx.x % L, rb = threadIdx.x / L;
  const int64_t row = (int64_t)blockIdx.x * R + rb;
  const bool on = row < a.rows;
  const T* const p = static_cast<const T*>(a.logits) + (on ? row : a.rows - 1) * a.ld;
  float x[V];
  load_row<T, V>(p, a.E, sub, whole, x);
  double key[V];
  Soft sm{0.0, 0.0};
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = sigmoid64(x[v]);
  } else {
    sm = softmax_terms<L, V>(x, key);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] *= sm.inv;
  }
  float b[V];
#pragma unroll
  for (int v = 0; v < V; ++v) b[v] = 0.f;
  if (a.bias) load_row<float, V>(a.bias, a.E, sub, bias_whole, b);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = sub * V + v;
    const float c = (float)key[v] + b[v];
    const bool may = x[v] != kNone && c != kNone;
    key[v] = may ? __builtin_fma((double)ordered(c), 4096.0, (double)(4095 - e)) : 0.0;
  }

  int* const sel = lds + rb * a.k;
  if (a.n_groups > 1) {
    uint32_t* const gs = reinterpret_cast<uint32_t*>(lds + R * a.k) + rb * (a.n_groups + a.E);
    uint32_t* const cs = gs + a.n_groups;
    const bool runs = a.per_group % V == 0;       // a lane's experts lie in one group
    if (runs) {
      double b1 = 0.0, b2 = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        b2 = key_max(b2, key_min(b1, key[v]));
        b1 = key_max(b1, key[v]);
      }
      if (sub * V < a.E) {
        cs[CS * sub] = (uint32_t)(b1 * (1.0 / 4096.0));
        if (V > 1) cs[CS * sub + 1] = (uint32_t)(b2 * (1.0 / 4096.0));
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = sub * V + v;
        if (e < a.E) cs[e] = (uint32_t)(key[v] * (1.0 / 4096.0));
      }
    }
    __syncthreads();
    for (int g = sub; g < a.n_groups; g += L) {
      uint32_t b1 = 0, b2 = 0;
      auto take = [&](uint32_t u) {
        b2 = max(b2, min(b1, u));
        b1 = max(b1, u);
      };
      if (runs) {
        const int n = a.per_group / V;
        for (int i = 0; i < n; ++i) {
          take(cs[CS * (g * n + i)]);
          if (V > 1) take(cs[CS * (g * n + i) + 1]);
        }
      } else {
        for (int i = 0; i < a.per_group; ++i) take(cs[g * a.per_group + i]);
      }
      if (a.top2 && b2 != 0) b1 = ordered(unordered(b1) + unordered(b2));
      gs[g] = b1;
    }
    __syncthreads();
    // a group is kept if fewer than top_groups come before it
    if (runs) {
      const int g = min(sub * V / a.per_group, a.n_groups - 1);
      const uint32_t mine = gs[g];
      int ahead = 0;
      for (int i = 0; i < a.n_groups; ++i) ahead += (gs[i] > mine || (gs[i] == mine && i < g)) ? 1 : 0;
      if (ahead >= a.top_groups) {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = 0.0;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = sub * V + v;
        if (key[v] > 0.0) {
          const int g = e / a.per_group;
          const uint32_t mine = gs[g];
          int ahead = 0;
          for (int i = 0; i < a.n_groups; ++i) ahead += (gs[i] > mine || (gs[i] == mine && i < g)) ? 1 : 0;
          if (ahead >= a.top_groups) key[v] = 0.0;
        }
      }
    }
  }

  // The sorted eight pay from the fifth expert on.
  bool done = false;
  if constexpr (V % 8 == 0) {
    if (a.k > 4 && a.k <= 8) {
      double k[8];
      top8<L, V>(key, k);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < a.k && sub == 0) sel[j] = expert_of(k[j]);
      done = true;
    }
  }
  if (!done) {
    for (int j = 0; j < a.k; ++j) {
      double m = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = key_max(m, key[v]);
      m = across<L>(m, [](double a, double b) { return key_max(a, b); });
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] == m ? 0.0 : key[v];
      if (sub == 0) sel[j] = expert_of(m);
    }
  }
  __syncthreads();
  // weights: the chosen logits once more, a lane per slot
  double total = 0.0;
  if (a.renorm) {
    for (int j = sub; j < a.k; j += L) {
      const int id = sel[j];
      total += id >= 0 ? score_of(a, sm, load_logit(p + id)) : 0.0;
    }
    total = group_sum<L>(total);
  }
  for (int j = sub; j < a.k; j += L) {
    const int id = sel[j];
    double w = id >= 0 ? score_of(a, sm, load_logit(p + id)) : 0.0;
    if (a.renorm && total != 0.0) w /= total;
    if (on) {
      a.ids[row * a.k + j] = id;
      a.weights[row * a.k + j] = (float)(w * (double)a.scale);
    }
  }
}

// dlogits of a row from its weights' gradients: u_j the score of slot j,
//   du_j = scale dw_j, or renormalised scale / S (dw_j - (sum_m dw_m u_m) / S)
//   softmax: dl_e = s_e (du_e - sum_j du_j u_j); sigmoid: du_e s_e (1 - s_e)
// where du_e sums the slots that name expert e (once a row in ids that the
// forward made; any ids are taken).  DENSE: softmax weights that are not
// renormalised, where every expert's score enters.  Else the chosen logits are
// all that is read: sum_j du_j u_j is zero, and the scores' common factor
// cancels in u / S.  LDS: the row's gradient [E].
template <class T, int L, int V, bool DENSE>
__global__ __launch_bounds__(kThreads<V>) void k_route_backward(RouteArgs a, int whole) {
  extern __shared__ float grad[];
  constexpr int R = kThreads<V> / L;
  const int sub = threadIdx.x % L, rb = threadIdx.x / L;
  const int64_t row = (int64_t)blockIdx.x * R + rb;
  const bool on = row < a.rows;
  const int64_t at = on ? row : a.rows - 1;
  const T* const p = static_cast<const T*>(a.logits) + at * a.ld;
  const int32_t* const ids = a.ids + at * a.k;
  const float* const dw = a.dweights + at * a.k;
  float* const du = grad + rb * a.E;
  for (int e = sub; e < a.E; e += L) du[e] = 0.f;
  float x[V];
  double ex[V];
  Soft sm{0.0, 1.0};
  if constexpr (DENSE) {
    load_row<T, V>(p, a.E, sub, whole, x);
    sm = softmax_terms<L, V>(x, ex);
  } else if (!a.sigmoid) {
    float m = kNone;
    for (int j = sub; j < a.k; j += L) {
      const int id = ids[j];
      if ((unsigned)id < (unsigned)a.E) m = fmaxf(m, load_logit(p + id));
    }
    m = across<L>(m, [](float a, float b) { return fmaxf(a, b); });
    sm.top = m == kNone ? 0.0 : (double)m;
  }
  double S = 0.0, dot = 0.0;
  for (int j = sub; j < a.k; j += L) {
    const int id = ids[j];
    if ((unsigned)id < (unsigned)a.E) {
      const double u = score_of(a, sm, load_logit(p + id));
      S += u;
      dot += (double)dw[j] * u;
    }
  }
  S = group_sum<L>(S);
  dot = group_sum<L>(dot);
  const double f = a.renorm ? (S == 0.0 ? 0.0 : (double)a.scale / S) : (double)a.scale;
  const double less = a.renorm && S != 0.0 ? dot / S : 0.0;
  __syncthreads();
  // of slots that name one expert the first adds them all, in order
  for (int j = sub; j < a.k; j += L) {
    const int id = ids[j];
    if ((unsigned)id >= (unsigned)a.E) continue;
    bool first = true;
    double sum = 0.0;
    for (int i = 0; i < a.k; ++i)
      if (ids[i] == id) {
        first = first && i >= j;
        sum += ((double)dw[i] - less) * f;
      }
    if (!first) continue;
    if constexpr (!DENSE) {
      const float l = load_logit(p + id);
      const double s = score_of(a, sm, l);
      // (an expert at -infinity has no gradient, whatever the others hold)
      sum = l == kNone ? 0.0 : a.sigmoid ? sum * s * (1.0 - s) : sum * s;
    }
    du[id] = (float)sum;
  }
  __syncthreads();
  if constexpr (DENSE) {
    const double inner = dot * (double)a.scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = sub * V + v;
      if (e < a.E) du[e] = x[v] == kNone ? 0.f : (float)(ex[v] * sm.inv * ((double)du[e] - inner));
    }
    __syncthreads();
  }
  if (!on) return;
  if (whole) {                           // four elements a lane
    for (int i = sub; i < a.E / 4; i += L) {
      const f32x4 g = reinterpret_cast<const f32x4*>(du)[i];
      if constexpr (sizeof(T) == 4)
        reinterpret_cast<f32x4*>(static_cast<float*>(a.dlogits) + row * a.E)[i] = g;
      else
        reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dlogits) + row * a.E)[i] =
            u32x2{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3])};
    }
  } else {
    for (int e = sub; e < a.E; e += L) {
      if constexpr (sizeof(T) == 4) static_cast<float*>(a.dlogits)[row * a.E + e] = du[e];
      else static_cast<uint16_t*>(a.dlogits)[row * a.E + e] = (uint16_t)pack_bf16x2(du[e], du[e]);
    }
  }
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class T, int L, int V>
void route_of(bool back, const RouteArgs& a, hipStream_t s) {
  constexpr int R = kThreads<V> / L;
  const unsigned grid = (unsigned)((a.rows + R - 1) / R);
  // rows that start and end on 16 bytes and fill every lane
  const bool whole = a.E == L * V && a.E * sizeof(T) % 16 == 0 && a.ld * sizeof(T) % 16 == 0 && aligned16(a.logits) &&
                     aligned16(a.dlogits);
  if (back) {
    const size_t lds = (size_t)R * a.E * 4;
    if (!a.sigmoid && !a.renorm)
      hipLaunchKernelGGL((k_route_backward<T, L, V, true>), dim3(grid), dim3(kThreads<V>), lds, s, a, whole);
    else
      hipLaunchKernelGGL((k_route_backward<T, L, V, false>), dim3(grid), dim3(kThreads<V>), lds, s, a, whole);
  } else {
    const size_t lds = (size_t)R * 4 * (a.k + (a.n_groups > 1 ? a.E + a.n_groups : 0));
    hipLaunchKernelGGL((k_route<T, L, V>), dim3(grid), dim3(kThreads<V>), lds, s, a, whole,
                       a.E == L * V && a.E % 4 == 0 && aligned16(a.bias));
  }
}

// Rows up to which a row takes a whole wave.
constexpr int64_t kFewRows = 1024;

template <class T>
void route_sized(bool back, const RouteArgs& a, hipStream_t s) {
  if (a.rows <= kFewRows) {
    if (a.E <= 64) return route_of<T, 64, 1>(back, a, s);
    if (a.E <= 128) return route_of<T, 64, 2>(back, a, s);
    if (a.E <= 256) return route_of<T, 64, 4>(back, a, s);
    if (a.E <= 512) return route_of<T, 64, 8>(back, a, s);
  }
  if (a.E <= 8) return route_of<T, 8, 1>(back, a, s);
  if (a.E <= 16) return route_of<T, 8, 2>(back, a, s);
  if (a.E <= 32) return route_of<T, 8, 4>(back, a, s);
  if (a.E <= 64) return route_of<T, 8, 8>(back, a, s);
  if (a.E <= 128) return route_of<T, 16, 8>(back, a, s);
  if (a.E <= 256) return route_of<T, 16, 16>(back, a, s);
  if (a.E <= 512) return route_of<T, 32, 16>(back, a, s);
  if (a.E <= 1024) return route_of<T, 64, 16>(back, a, s);
  if (a.E <= 2048) return route_of<T, 64, 32>(back, a, s);
  route_of<T, 64, 64>(back, a, s);
}

}  // namespace

void launch_route(bool f32, const RouteArgs& a, hipStream_t s) {
  if (f32) route_sized<float>(false, a, s);
  else route_sized<uint16_t>(false, a, s);
}
void launch_route_backward(bool f32, const RouteArgs& a, hipStream_t s) {
  if (f32) route_sized<float>(true, a, s);
  else route_sized<uint16_t>(true, a, s);
}

}  // namespace mlora
