// Routing of rows to experts and its gradient.
//
// A row's logits lie in the registers of L lanes, V neighbours each (64 / L
// rows a wave), so every step over the experts is V operations for all the
// wave's rows at once and every sum or maximum log2(L) lane exchanges.  Many
// rows take few lanes each (work per row counts), few rows many (latency does).
// Scores are computed in 64 bits, which the vector units run at the rate of
// 32, and rounded to fp32 once: two programs then agree on every choice but
// for scores within 2^-45 of a rounding border.  A choice compares score + bias,
// in fp32, with the expert's number in the 29 bits that fp32 leaves of a double,
// so a step of the top_k is a maximum, and ties go to the lowest expert.
//
// Bound by instructions, not by the logits' bytes: 32768 rows of 256, sigmoid, 8
// of 256 out of 4 of 8 groups, fp32 take 21.9 us (1.5 TB/s; 18.3 without
// groups), of which about 24 instructions an expert are its score, 9 its key and
// 19 sorting; 32768 rows of 256 softmax 20.2 us, in bf16 19.7 (half the bytes: they
// do not count); of 64 in bf16, 2 or 8 chosen, 6.6 and 7.4 us; 16 rows of 64 3.2 us,
// a launch.  With 32 experts a lane in place of 16 the groups' case took as long
// (fewer exchanges, fewer waves).  Over 2048 experts a lane's 64 keys and scores
// pass its registers (256 in use, spilling to accumulation registers; one wave a
// SIMD): 4096 rows of 4096 63 us, 0.5 TB/s.
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

// A constant in scalar registers, where a multiply-add takes it as it is (the
// compiler's choice copies it into vector registers before each).
__device__ __forceinline__ double constant(double c) {
  asm("" : "+s"(c));
  return c;
}
// e^x in 64 bits for |x| <= 1e9: x = n ln 2 + r, |r| <= ln 2 / 2 (the rounding
// to n by the sum with 3 2^51, which leaves n in the low bits), and for e^r the
// polynomial of degree 10 through 1 at 0 of least relative error, 2^-51.6 (by
// Remez exchange).  NaN stays.
__device__ __forceinline__ double exp64(double x) {
  const double big = constant(6755399441055744.0);
  const double t = __builtin_fma(x, constant(1.4426950408889634), big), n = t - big;
  double r = __builtin_fma(n, constant(-0.6931471805599453), x);
  r = __builtin_fma(n, constant(-2.3190468138462996e-17), r);
  double p = constant(0x1.2a4757db84f44p-22);
  p = __builtin_fma(p, r, constant(0x1.730bd565ae4cdp-19));
  p = __builtin_fma(p, r, constant(0x1.a017fb62f39a4p-16));
  p = __builtin_fma(p, r, constant(0x1.a01967c4fae8fp-13));
  p = __builtin_fma(p, r, constant(0x1.6c16c20da84a3p-10));
  p = __builtin_fma(p, r, constant(0x1.111111337199ap-7));
  p = __builtin_fma(p, r, constant(0x1.555555552f91ep-5));
  p = __builtin_fma(p, r, constant(0x1.5555555548c99p-3));
  p = __builtin_fma(p, r, constant(0x1.000000000004bp-1));
  p = __builtin_fma(p, r, constant(0x1.0000000000029p+0));
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
}
// 1 / x for x in [1, 2^1011]: the hardware's approximation, off by e < 2^-20, times
// 1 + e + e^2.
__device__ __forceinline__ double reciprocal(double x) {
  const double r = __builtin_amdgcn_rcp(x), e = __builtin_fma(-x, r, 1.0);
  return __builtin_fma(__builtin_fma(e, e, e), r, r);
}
__device__ __forceinline__ float clamp(float x, float lo, float hi) {     // NaN stays
  const float y = x < lo ? lo : x;
  return y > hi ? hi : y;
}
// (e^700 has a reciprocal; what is below counts as zero, which it is in fp32)
__device__ __forceinline__ double sigmoid64(float x) { return reciprocal(1.0 + exp64(-(double)clamp(x, -700.f, 700.f))); }

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

// The key of a choice: c as a double, its lowest 12 bits 4095 - e where c is not
// negative and e where it is (a larger number is then a smaller key).  Not
// numbers of that kind, which the bits would make a NaN: infinity 2^1000 and NaN
// 2^1001, both with the bits; none, 2^1000 below zero, for an expert that may
// not be chosen.
constexpr uint32_t kLast = MLORA_MAX_EXPERTS - 1;      // 12 bits
constexpr double kNoKey = -0x1p1000;
__device__ __forceinline__ double with_low(double v, uint32_t low) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, v) | low);
}
__device__ __forceinline__ double key_of(float c, uint32_t last) {
  const uint32_t flip = (uint32_t)((int32_t)__float_as_uint(c) >> 31) & kLast;
  const double k = with_low((double)c, last ^ flip);
  return c == kNone ? kNoKey : k;
}
__device__ __forceinline__ bool no_key(double key) { return key < -0x1p999; }
__device__ __forceinline__ int expert_of(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  const uint32_t flip = (uint32_t)((int32_t)(b >> 32) >> 31) & kLast;
  const int e = (int)((((uint32_t)b & kLast) ^ flip) ^ kLast);
  return no_key(key) ? -1 : e;
}
__device__ __forceinline__ uint32_t image_of(double key) {
  return no_key(key) ? 0u : key >= 0x1p1001 ? 0xffffffffu : ordered((float)key);
}

// A row's softmax terms: its maximum and the reciprocal of the sum of e^(x - max).
struct Soft {
  double top, inv;
};
// x - top <= 0, where e^ of it is zero in fp32 and in every sum at most -800.
__device__ __forceinline__ double below(float x, double top) {
  const double d = (double)x - top;
  return d < -800.0 ? -800.0 : d;
}
__device__ __forceinline__ double score_of(const RouteArgs& a, const Soft& s, float x) {
  if (x == kNone) return 0.0;
  if (a.sigmoid) return x < -700.f ? 0.0 : sigmoid64(x);
  return exp64(below(x, s.top)) * s.inv;
}
// The sum of N (a power of two) neighbours as a balanced tree.  With the lanes' sums
// added the same way, neighbours first, a row's sum is one tree over its experts
// (zeros past the last) whether a lane holds one of them or 64, so its bits do not
// depend on the layout that a call's number of rows takes.
template <int N>
__device__ __forceinline__ double tree_sum(const double* v) {
  if constexpr (N == 1) return v[0];
  else return tree_sum<N / 2>(v) + tree_sum<N / 2>(v + N / 2);
}
// The same over slots: the sum of term(j) for the lane's n neighbours j = sub n .. (n
// a power of two, at most 8; the terms come one by one, so two that are complete wait
// for their neighbours).
template <class T, class F>
__device__ __forceinline__ T slot_sum(int sub, int n, F term) {
  T one{}, two{}, four{}, s{};
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    s = term(sub * n + i);
    if (!(i & 1)) { one = s; continue; }
    s = one + s;
    if (!(i & 2)) { two = s; continue; }
    s = two + s;
    if (!(i & 4)) { four = s; continue; }
    s = four + s;
  }
  return s;
}
struct TwoSums {
  double a, b;
  __device__ __forceinline__ TwoSums operator+(const TwoSums& o) const { return {a + o.a, b + o.b}; }
};
// Neighbouring slots a lane sums: the least power of two with which L lanes reach k.
// ONE (k <= L) is a kernel of its own, whose code has no loop over a lane's slots:
// with both in one, 32768 rows of 64, 8 chosen, took 7.8 us in place of 7.3.
template <int L, bool ONE>
__device__ __forceinline__ int slots_a_lane(int k) {
  int n = 1;
  if constexpr (!ONE)
    while (n * L < k) n *= 2;
  return n;
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
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = x[v] == kNone ? 0.0 : exp64(below(x[v], s.top));
  const double sum = group_sum<L>(tree_sum<V>(e));
  s.inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  return s;
}

// Lane `sub`'s experts sub V .. of a row (-infinity past the last); whole: each
// lane's are all there or all past it, and 16-byte aligned.
template <class T, int V>
__device__ __forceinline__ void load_row(const T* p, int E, int sub, bool whole, float (&x)[V]) {
  constexpr int P = 16 / sizeof(T);
  if constexpr (V % P == 0) {
    if (whole) {
      if (sub * V >= E) {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = kNone;
        return;
      }
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

}  // namespace

// LDS of a row: the chosen ids [top_k]; with expert groups, per run of min(V,
// group) experts its two largest ordered scores, and the groups' scores.
template <class T, int L, int V, bool ONE>
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
  float c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = x[v] == kNone ? kNone : (float)key[v];
  if (a.bias) {
    float b[V];
    load_row<float, V>(a.bias, a.E, sub, bias_whole, b);
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] += c[v] == kNone ? 0.f : b[v];
  }
  // (V is a power of two: 4095 - e is what the lane's experts share and V - 1 - v)
  const uint32_t last = kLast + 1 - (sub + 1) * V;
  bool odd = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    odd = odd || !(c[v] < -kNone);
    key[v] = key_of(c[v], last | (V - 1 - v));
  }
  if (__any(odd)) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!(c[v] < -kNone)) key[v] = with_low(c[v] != c[v] ? 0x1p1001 : 0x1p1000, last | (V - 1 - v));
  }

  int* const sel = lds + rb * a.k;
  if (a.n_groups > 1) {
    uint32_t* const gs = reinterpret_cast<uint32_t*>(lds + R * a.k) + rb * (a.n_groups + a.E);
    uint32_t* const cs = gs + a.n_groups;
    const bool runs = a.per_group % V == 0;       // a lane's experts lie in one group
    if (runs) {
      double b1 = kNoKey, b2 = kNoKey;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        b2 = key_max(b2, key_min(b1, key[v]));
        b1 = key_max(b1, key[v]);
      }
      if (sub * V < a.E) {
        cs[CS * sub] = image_of(b1);
        if (V > 1) cs[CS * sub + 1] = image_of(b2);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = sub * V + v;
        if (e < a.E) cs[e] = image_of(key[v]);
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
        for (int v = 0; v < V; ++v) key[v] = kNoKey;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = sub * V + v;
        if (!no_key(key[v])) {
          const int g = e / a.per_group;
          const uint32_t mine = gs[g];
          int ahead = 0;
          for (int i = 0; i < a.n_groups; ++i) ahead += (gs[i] > mine || (gs[i] == mine && i < g)) ? 1 : 0;
          if (ahead >= a.top_groups) key[v] = kNoKey;
        }
      }
    }
  }

  // The sorted eight pay from the fifth expert on (32768 rows of 64: two chosen one by one
  // 6.6 us, eight by sorting 7.4).
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
      for (int v = 0; v < V; ++v) key[v] = key[v] == m ? kNoKey : key[v];
      if (sub == 0) sel[j] = expert_of(m);
    }
  }
  __syncthreads();
  // weights: the chosen logits once more, a lane per slot (its score is kept where a lane has one)
  auto score_at = [&](int j) {
    const int id = j < a.k ? sel[j] : -1;
    return id >= 0 ? score_of(a, sm, load_logit(p + id)) : 0.0;
  };
  const int n = slots_a_lane<L, ONE>(a.k);
  double mine = slot_sum<double>(sub, n, score_at);
  double total = 0.0;
  if (a.renorm) total = group_sum<L>(mine);
  // A renormalised softmax is the softmax of the chosen logits.  Where a bias chose experts
  // so far below the row's largest that their scores leave 64 bits or, as weights beside
  // each other, could (2^-700: fp32 and a scale span 2^-276, a double 2^-1022), they are
  // taken beside the largest chosen one, as in the gradient.  (Always so costs 0.3 us.)
  if (__builtin_expect(a.renorm && !a.sigmoid && total < 0x1p-700, false)) {
    float m = kNone;
    for (int j = sub; j < a.k; j += L) m = fmaxf(m, sel[j] >= 0 ? load_logit(p + sel[j]) : kNone);
    m = across<L>(m, [](float a, float b) { return fmaxf(a, b); });
    sm.top = m == kNone ? 0.0 : (double)m;
    sm.inv = 1.0;
    mine = slot_sum<double>(sub, n, score_at);
    total = group_sum<L>(mine);
  }
  if (!on) return;
  for (int j = sub; j < a.k; j += L) {
    const int id = sel[j];
    double u = n == 1 ? mine : score_at(j);
    if (a.renorm && total != 0.0) u /= total;
    a.ids[row * a.k + j] = id;
    a.weights[row * a.k + j] = (float)(u * (double)a.scale);
  }
}

// dlogits of a row from its weights' gradients: u_j the score of slot j,
//   du_j = scale dw_j, or renormalised scale / S (dw_j - (sum_m dw_m u_m) / S)
//   softmax: dl_e = s_e (du_e - sum_j du_j u_j); sigmoid: du_e s_e (1 - s_e)
// where du_e sums the slots that name expert e (once a row in ids that the
// forward made; any ids are taken).  DENSE: softmax weights that are not
// renormalised, where every expert's score enters.  Else the chosen logits are
// all that is read: sum_j du_j u_j is zero, and the scores' common factor
// cancels in u / S.  LDS: the row's gradient [E]; dense, the sums of dw until the
// scores are there, without the scale: of an expert named once that is dw itself, so
// that dw - sum_j dw_j u_j, which cancels where one score is nearly 1, starts from no
// rounded number.  Dense, 16384 rows of 64 in bf16 6.3 us, of 256 16.2 (1 TB/s: the
// 64-bit exponentials of every expert), in fp32 18.0; not dense 4.9, 8.2 and 9.7 (the
// chosen slots' serial work and stores, 16.8 MB at 1.8 TB/s in the last), sigmoid of
// 256 in fp32 8.5 to 9.4 us.
template <class T, int L, int V, bool DENSE, bool ONE>
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
  const TwoSums sums = slot_sum<TwoSums>(sub, slots_a_lane<L, ONE>(a.k), [&](int j) {
    const int id = j < a.k ? ids[j] : -1;
    if ((unsigned)id >= (unsigned)a.E) return TwoSums{0.0, 0.0};
    const double u = score_of(a, sm, load_logit(p + id));
    return TwoSums{u, (double)dw[j] * u};
  });
  const double S = group_sum<L>(sums.a), dot = group_sum<L>(sums.b);
  const double inv = a.renorm ? (S == 0.0 ? 0.0 : 1.0 / S) : 1.0;
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
        sum += (double)dw[i] - less;
      }
    if (!first) continue;
    if constexpr (!DENSE) {
      const float l = load_logit(p + id);
      // s as score_of has it; 1 - s as e^-l s: where s is nearly 1, its rounded value no longer
      // holds the rest.  (s / S first: S may be as little as e^-700.)
      const double e = exp64(a.sigmoid ? -(double)clamp(l, -700.f, 700.f) : below(l, sm.top));
      const double s = !a.sigmoid ? e : l < -700.f ? 0.0 : reciprocal(1.0 + e);
      sum *= (double)a.scale * (s * inv);
      if (a.sigmoid) sum *= e * s;
      // (an expert at -infinity has no gradient, whatever the others hold)
      sum = l == kNone ? 0.0 : sum;
    }
    du[id] = (float)sum;
  }
  __syncthreads();
  if constexpr (DENSE) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = sub * V + v;
      if (e < a.E) du[e] = x[v] == kNone ? 0.f : (float)(ex[v] * sm.inv * (double)a.scale * ((double)du[e] - dot));
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

template <class T, int L, int V, bool ONE>
void route_of(bool back, const RouteArgs& a, hipStream_t s) {
  constexpr int R = kThreads<V> / L;
  const unsigned grid = (unsigned)((a.rows + R - 1) / R);
  // rows that start and end on 16 bytes and fill the lanes that they reach
  const bool whole = a.E % V == 0 && a.E * sizeof(T) % 16 == 0 && a.ld * sizeof(T) % 16 == 0 && aligned16(a.logits) &&
                     aligned16(a.dlogits);
  if (back) {
    const size_t lds = (size_t)R * a.E * 4;
    if (!a.sigmoid && !a.renorm)
      hipLaunchKernelGGL((k_route_backward<T, L, V, true, ONE>), dim3(grid), dim3(kThreads<V>), lds, s, a, whole);
    else
      hipLaunchKernelGGL((k_route_backward<T, L, V, false, ONE>), dim3(grid), dim3(kThreads<V>), lds, s, a, whole);
  } else {
    const size_t lds = (size_t)R * 4 * (a.k + (a.n_groups > 1 ? a.E + a.n_groups : 0));
    hipLaunchKernelGGL((k_route<T, L, V, ONE>), dim3(grid), dim3(kThreads<V>), lds, s, a, whole,
                       a.E % V == 0 && a.E % 4 == 0 && aligned16(a.bias));
  }
}
template <class T, int L, int V>
void route_of(bool back, const RouteArgs& a, hipStream_t s) {
  if constexpr (L < 64 && V > 1)            // (k is at most 64, and at most E)
    if (a.k > L) return route_of<T, L, V, false>(back, a, s);
  route_of<T, L, V, true>(back, a, s);
}

// Rows up to which a row takes a whole wave: 1024 waves, one for each of the
// chip's SIMDs (16 rows of 64 with eight lanes a row 7.0 us, with 64 3.9).
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
