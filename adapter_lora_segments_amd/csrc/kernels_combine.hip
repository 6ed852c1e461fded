// A token's expert rows, weighted and summed, and the gradients of that sum.
//   out_t = add_t + sum_j w_tj Y[t k + j]
//   dY[t k + j] = w_tj dout_t,   dw_tj = sum_i dout_ti Y[t k + j][i]
// over the slots j that a router filled; a dropped slot's row is not read (it
// may hold anything) and gets a zero gradient.  Sums in fp32, one rounding.
// One pass over the data, 16 bytes a lane and row, bound by HBM: 16384 tokens of 8
// rows of 4096 in bf16 224 us, 5.4 TB/s; 16 tokens of 2 2.4 us, a launch.
#include "device_common.hpp"
#include "route.hpp"

namespace mlora {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostGroups = (1 << 24) - 1;       // workgroups of a launch: below 2^32 threads

// 16 bytes of a row as fp32: eight bf16 or four fp32.
template <bool F32>
struct Piece {
  static constexpr int N = F32 ? 4 : 8;
  float v[N];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const u32x4 u = reinterpret_cast<const u32x4*>(base)[at];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        v[i] = __uint_as_float(u[i]);
      } else {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) u[i] = __float_as_uint(v[i]);
      else u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    reinterpret_cast<u32x4*>(base)[at] = u;
  }
};

// Lanes that share a token: a power of two that covers its 16-byte pieces, at
// most `most`.
inline int token_lanes(int pieces, int most) {
  int p = 1;
  while (p < pieces && p < most) p <<= 1;
  return p;
}

}  // namespace

// One piece of one token a thread; `split` workgroups share a token that has
// more pieces than the workgroup threads.
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_combine(CombineArgs a, int lanes, int split) {
  constexpr int N = Piece<F32>::N;
  const int pieces = a.d / N, per = kThreads / lanes;
  const int64_t t = (int64_t)(blockIdx.x / split) * per + threadIdx.x / lanes;
  const int c = (int)(blockIdx.x % split) * kThreads + (int)(threadIdx.x % lanes);
  if (t >= a.tokens || c >= pieces) return;
  Piece<F32> sum;
#pragma unroll
  for (int i = 0; i < N; ++i) sum.v[i] = 0.f;
  const int64_t slot = t * a.k;
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    if (a.ids && (uint32_t)a.ids[slot + j] >= a.limit) continue;
    const float w = a.weights ? a.weights[slot + j] : 1.f;
    Piece<F32> y;
    y.load(a.Y, (slot + j) * pieces + c);
#pragma unroll
    for (int i = 0; i < N; ++i) sum.v[i] += w * y.v[i];
  }
  if (a.add) {
    Piece<F32> y;
    y.load(a.add, t * pieces + c);
#pragma unroll
    for (int i = 0; i < N; ++i) sum.v[i] += y.v[i];
  }
  sum.store(a.out, t * pieces + c);
}

// A slot by one wave (`lanes` of one where a row has fewer pieces), with the loads
// of U pieces of dout and of its row of Y in flight; the slots of a token read
// dout once each, all but the first from the caches.  A lane's pieces are added
// in order and the lanes meet by exchanges, the same ones for any number of
// tokens and slots.  7681 tokens of 2 rows of 4104 in bf16 55 us (5.7 TB/s), of 8
// rows of 4096 (16384 tokens) 400 us (5.7 TB/s), 35 tokens of 8 rows of 8072 in
// fp32 8 us; all slots of a token by one wave took 64, 490 and 64 us: fewer
// loads in flight, since a store may be to what a later load reads.  Where no dot
// product is wanted (dweights NULL, a dropped slot) dout stands in for Y and is read
// twice, the second time from the caches.
template <bool F32, int U>
__global__ __launch_bounds__(kThreads) void k_combine_backward(CombineArgs a, int lanes) {
  constexpr int N = Piece<F32>::N;
  const int pieces = a.d / N, per = kThreads / lanes, sub = threadIdx.x % lanes;
  const int64_t slots = a.tokens * a.k;
  for (int64_t s0 = (int64_t)blockIdx.x * per; s0 < slots; s0 += (int64_t)gridDim.x * per) {
    // (below 2^31; lanes past the last slot take the last one's, but store nothing)
    const bool on = s0 + threadIdx.x / lanes < slots;
    const uint32_t slot = (uint32_t)(on ? s0 + threadIdx.x / lanes : slots - 1), t = slot / (uint32_t)a.k;
    const bool kept = !a.ids || (uint32_t)a.ids[slot] < a.limit;
    const bool dots = a.dweights && kept;
    const float w = a.weights ? a.weights[slot] : 1.f;
    const int64_t g_at = (int64_t)t * pieces, y_at = dots ? (int64_t)slot * pieces : g_at;
    const void* const y_of = dots ? a.Y : a.dout;       // a dropped slot's row is not read
    float dot = 0.f;
    for (int c0 = sub; c0 < pieces; c0 += lanes * U) {
      Piece<F32> g[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = min(c0 + lanes * u, pieces - 1);
        g[u].load(a.dout, g_at + c);
        y[u].load(y_of, y_at + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + lanes * u;
        if (c >= pieces) break;
#pragma unroll
        for (int i = 0; i < N; ++i) dot += g[u].v[i] * y[u].v[i];
        if (a.dY && on) {
          Piece<F32> o;
#pragma unroll
          for (int i = 0; i < N; ++i) o.v[i] = kept ? w * g[u].v[i] : 0.f;
          o.store(a.dY, (int64_t)slot * pieces + c);
        }
      }
    }
    if (!a.dweights) continue;
    for (int d = 1; d < lanes; d <<= 1) dot += __shfl_xor(dot, d);
    if (on && sub == 0) a.dweights[slot] = kept ? dot : 0.f;
  }
}

void launch_combine(bool f32, const CombineArgs& a, hipStream_t s) {
  const int pieces = a.d / (f32 ? 4 : 8), lanes = token_lanes(pieces, kThreads), per = kThreads / lanes;
  const int split = (pieces + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)((a.tokens + per - 1) / per * split);
  if (f32) hipLaunchKernelGGL((k_combine<true>), dim3(grid), dim3(kThreads), 0, s, a, lanes, split);
  else hipLaunchKernelGGL((k_combine<false>), dim3(grid), dim3(kThreads), 0, s, a, lanes, split);
}

namespace {

template <bool F32>
void backward_of(const CombineArgs& a, hipStream_t s) {
  const int pieces = a.d / (F32 ? 4 : 8), lanes = token_lanes(pieces, 64), per = kThreads / lanes;
  const int64_t groups = (a.tokens * a.k + per - 1) / per;
  const unsigned grid = (unsigned)(groups < kMostGroups ? groups : kMostGroups);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, a, lanes); };
  if (pieces <= lanes) go(k_combine_backward<F32, 1>);
  else if (pieces <= 2 * lanes) go(k_combine_backward<F32, 2>);
  else if (pieces <= 4 * lanes) go(k_combine_backward<F32, 4>);
  else go(k_combine_backward<F32, 8>);
}

}  // namespace

void launch_combine_backward(bool f32, const CombineArgs& a, hipStream_t s) {
  if (f32) backward_of<true>(a, s);
  else backward_of<false>(a, s);
}

}  // namespace mlora
