// Routing of rows to experts and its gradient.
//
// A row's logits lie in the registers of L lanes, V values each (64 / L rows a
// wave), so every step over the experts is V operations for all the wave's
// rows at once and every sum or maximum log2(L) lane exchanges.
// Scores are computed in 64 bits, which the vector units run at the rate of
// 32, and rounded to fp32 once: two programs then agree on every choice but
// for scores within 2^-50 of a rounding border.  A choice compares (score +
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

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }

// e^x in 64 bits: x = n ln 2 + r, |r| <= ln 2 / 2, the Taylor series of e^r to
// r^12 (the next term is below 2^-52).  Below -745 zero, NaN stays.
__device__ __forceinline__ double exp64(double x) {
  const double c = x < -745.0 ? -745.0 : x > 710.0 ? 710.0 : x;
  const double n = __builtin_rint(c * 1.4426950408889634);
  double r = __builtin_fma(n, -0.6931471805599453, c);
  r = __builtin_fma(n, -2.3190468138462996e-17, r);
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
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

// Lane exchange within groups of L lanes (a power of two up to 64).
__device__ __forceinline__ double xor64(double v, int d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((int)(uint32_t)b, d), hi = __shfl_xor((int)(uint32_t)(b >> 32), d);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int L>
__device__ __forceinline__ double group_max(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    const double o = xor64(v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <int L>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += xor64(v, d);
  return v;
}
template <int L>
__device__ __forceinline__ float group_maxf(float v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Ordered 32-bit image of a score that may be chosen: rises with it, NaN last
// (chosen first, so that it shows), never 0.
__device__ __forceinline__ uint32_t ordered(float c) {
  if (c != c) return 0xffffffffu;
  const uint32_t b = __float_as_uint(c + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// A row's softmax terms: maximum and the reciprocal of the sum of e^(x - max).
struct Soft {
  double top, inv;
};
__device__ __forceinline__ double score_of(const RouteArgs& a, const Soft& s, float x) {
  if (x == -__builtin_inff()) return 0.0;
  if (a.sigmoid) return 1.0 / (1.0 + exp64(-(double)x));
  return exp64((double)x - s.top) * s.inv;
}

template <int L, int V>
__device__ __forceinline__ Soft softmax_terms(const float (&x)[V]) {
  float m = -__builtin_inff();
#pragma unroll
  for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
  m = group_maxf<L>(m);
  Soft s;
  s.top = m == -__builtin_inff() ? 0.0 : (double)m;
  double sum = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += x[v] == -__builtin_inff() ? 0.0 : exp64((double)x[v] - s.top);
  sum = group_sum<L>(sum);
  s.inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  return s;
}

template <class T, int L, int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t row, int sub, float (&x)[V]) {
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + sub;
    x[v] = e < a.E ? load_logit(p + e) : -__builtin_inff();
  }
}

}  // namespace

// Lane `sub` of a row holds experts sub, sub + L, ...; LDS: the row's chosen
// ids [top_k], with expert groups its scores [E] and the groups' scores
// [n_groups] (NaN as the largest).
template <class T, int L, int V>
__global__ __launch_bounds__(kThreads<V>) void k_route(RouteArgs a) {
  extern __shared__ int lds[];
  constexpr int R = kThreads<V> / L;
  const int sub = threadIdx.x % L, rb = threadIdx.x / L;
  const int64_t row = (int64_t)blockIdx.x * R + rb;
  const bool on = row < a.rows;
  const int64_t at = on ? row : a.rows - 1;
  float x[V];
  load_row<T, L, V>(a, at, sub, x);
  Soft sm{0.0, 0.0};
  if (!a.sigmoid) sm = softmax_terms<L, V>(x);

  int* const sel = lds + rb * a.k;
  double key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + sub;
    float c = (float)score_of(a, sm, x[v]);
    if (a.bias && e < a.E) c += a.bias[e];
    const bool may = x[v] != -__builtin_inff() && c != -__builtin_inff();
    key[v] = may ? __builtin_fma((double)ordered(c), 4096.0, (double)(4095 - e)) : 0.0;
  }
  if (a.n_groups > 1) {
    uint32_t* const cs = reinterpret_cast<uint32_t*>(lds + R * a.k) + rb * (a.E + a.n_groups);
    uint32_t* const gs = cs + a.E;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      if (e < a.E) cs[e] = key[v] > 0.0 ? (uint32_t)(key[v] * (1.0 / 4096.0)) : 0u;
    }
    __syncthreads();
    for (int g = sub; g < a.n_groups; g += L) {
      uint32_t b1 = 0, b2 = 0;
      for (int i = 0; i < a.per_group; ++i) {
        const uint32_t u = cs[g * a.per_group + i];
        b2 = max(b2, min(b1, u));
        b1 = max(b1, u);
      }
      if (a.top2 && b2 != 0) {
        const auto back = [](uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu)); };
        b1 = ordered(back(b1) + back(b2));
      }
      gs[g] = b1;
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + sub;
      if (key[v] > 0.0) {
        const int g = e / a.per_group;
        const uint32_t mine = gs[g];
        int ahead = 0;
        for (int i = 0; i < a.n_groups; ++i) ahead += (gs[i] > mine || (gs[i] == mine && i < g)) ? 1 : 0;
        if (ahead >= a.top_groups) key[v] = 0.0;
      }
    }
  }

  for (int j = 0; j < a.k; ++j) {
    double m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
    m = group_max<L>(m);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] == m ? 0.0 : key[v];
    if (sub == 0) {
      const uint64_t whole = (uint64_t)m;
      sel[j] = m > 0.0 ? 4095 - (int)(whole & 4095) : -1;
    }
  }
  __syncthreads();
  // weights: the chosen logits once more, a lane per slot
  const T* p = static_cast<const T*>(a.logits) + at * a.ld;
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
// forward made; any ids are taken).  LDS: du [E] of each row.
template <class T, int L, int V>
__global__ __launch_bounds__(kThreads<V>) void k_route_backward(RouteArgs a) {
  extern __shared__ int lds[];
  constexpr int R = kThreads<V> / L;
  const int sub = threadIdx.x % L, rb = threadIdx.x / L;
  const int64_t row = (int64_t)blockIdx.x * R + rb;
  const bool on = row < a.rows;
  const int64_t at = on ? row : a.rows - 1;
  float x[V];
  load_row<T, L, V>(a, at, sub, x);
  Soft sm{0.0, 0.0};
  if (!a.sigmoid) sm = softmax_terms<L, V>(x);
  float* const du = reinterpret_cast<float*>(lds) + rb * a.E;
  for (int e = sub; e < a.E; e += L) du[e] = 0.f;
  __syncthreads();
  const T* p = static_cast<const T*>(a.logits) + at * a.ld;
  const int32_t* ids = a.ids + at * a.k;
  const float* dw = a.dweights + at * a.k;
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
  // of slots that name one expert the first adds them all, in order
  const double f = a.renorm ? (S == 0.0 ? (double)a.scale : (double)a.scale / S) : (double)a.scale;
  const double less = a.renorm && S != 0.0 ? dot / S : 0.0;
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
    if (first) du[id] = (float)sum;
  }
  __syncthreads();
  // sum_j du_j u_j: zero where the weights are renormalised
  const double inner = a.renorm && S != 0.0 ? 0.0 : dot * (double)a.scale;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + sub;
    if (e >= a.E || !on) continue;
    const double s = score_of(a, sm, x[v]), d = (double)du[e];
    // (an expert at -inf has no gradient, whatever the others hold)
    const double full = a.sigmoid ? d * s * (1.0 - s) : s * (d - inner);
    const float g = x[v] == -__builtin_inff() ? 0.f : (float)full;
    if constexpr (sizeof(T) == 4) {
      static_cast<float*>(a.dlogits)[row * a.E + e] = g;
    } else {
      static_cast<uint16_t*>(a.dlogits)[row * a.E + e] = (uint16_t)pack_bf16x2(g, g);
    }
  }
}

namespace {

template <class T, int L, int V>
void route_of(bool back, const RouteArgs& a, hipStream_t s) {
  constexpr int R = kThreads<V> / L;
  const unsigned grid = (unsigned)((a.rows + R - 1) / R);
  if (back) {
    hipLaunchKernelGGL((k_route_backward<T, L, V>), dim3(grid), dim3(kThreads<V>), (size_t)R * a.E * 4, s, a);
  } else {
    const size_t lds = (size_t)R * 4 * (a.k + (a.n_groups > 1 ? a.E + a.n_groups : 0));
    hipLaunchKernelGGL((k_route<T, L, V>), dim3(grid), dim3(kThreads<V>), lds, s, a);
  }
}

template <class T>
void route_sized(bool back, const RouteArgs& a, hipStream_t s) {
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
