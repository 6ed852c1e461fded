// A token's expert rows, weighted and summed, and the gradients of that sum.
//   out_t = add_t + sum_j w_tj Y[t k + j]
//   dY[t k + j] = w_tj dout_t,   dw_tj = sum_i dout_ti Y[t k + j][i]
// over the slots j that a router filled; a dropped slot's row is not read (it
// may hold anything) and gets a zero gradient.  Sums in fp32, one rounding.
// One pass over the data, 16 bytes a lane and row, bound by HBM.
#include "device_common.hpp"
#include "route.hpp"

namespace mlora {

namespace {

constexpr int kThreads = 256;

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

// Lanes that share a token: a power of two that covers its 16-byte pieces, up
// to the workgroup.
inline int token_lanes(int pieces) {
  int p = 1;
  while (p < pieces && p < kThreads) p <<= 1;
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

// All pieces of a token by one workgroup (or a part of one): the dot products
// meet by lane exchanges, then across the token's waves in wave order.
template <bool F32>
__global__ __launch_bounds__(kThreads) void k_combine_backward(CombineArgs a, int lanes) {
  constexpr int N = Piece<F32>::N, KB = 8;
  __shared__ float part[kThreads / 64][KB];
  const int pieces = a.d / N, per = kThreads / lanes, sub = threadIdx.x % lanes, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes;
  const bool on = t < a.tokens;
  const int64_t slot = t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    float dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) dot[j] = 0.f;
    for (int c = sub; on && c < pieces; c += lanes) {
      Piece<F32> g;
      g.load(a.dout, t * pieces + c);
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (j0 + j >= a.k) break;
        const int64_t s = slot + j0 + j;
        const bool kept = !a.ids || (uint32_t)a.ids[s] < a.limit;
        const float w = kept ? (a.weights ? a.weights[s] : 1.f) : 0.f;
        if (a.dweights && kept) {
          Piece<F32> y;
          y.load(a.Y, s * pieces + c);
#pragma unroll
          for (int i = 0; i < N; ++i) dot[j] += g.v[i] * y.v[i];
        }
        if (a.dY) {
          Piece<F32> o;
#pragma unroll
          for (int i = 0; i < N; ++i) o.v[i] = kept ? w * g.v[i] : 0.f;
          o.store(a.dY, s * pieces + c);
        }
      }
    }
    if (!a.dweights) continue;
    const int in_wave = lanes < 64 ? lanes : 64;
#pragma unroll
    for (int j = 0; j < KB; ++j)
      for (int d = 1; d < in_wave; d <<= 1) dot[j] += __shfl_xor(dot[j], d);
    if (lanes > 64) {
      __syncthreads();
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int j = 0; j < KB; ++j) part[wave][j] = dot[j];
      }
      __syncthreads();
      const int first = wave - sub / 64;
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        dot[j] = part[first][j];
        for (int w = 1; w < lanes / 64; ++w) dot[j] += part[first + w][j];
      }
    }
    if (on && sub == 0) {
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (j0 + j < a.k) a.dweights[slot + j0 + j] = dot[j];
    }
  }
}

void launch_combine(bool f32, const CombineArgs& a, hipStream_t s) {
  const int pieces = a.d / (f32 ? 4 : 8), lanes = token_lanes(pieces), per = kThreads / lanes;
  const int split = (pieces + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)((a.tokens + per - 1) / per * split);
  if (f32) hipLaunchKernelGGL((k_combine<true>), dim3(grid), dim3(kThreads), 0, s, a, lanes, split);
  else hipLaunchKernelGGL((k_combine<false>), dim3(grid), dim3(kThreads), 0, s, a, lanes, split);
}

void launch_combine_backward(bool f32, const CombineArgs& a, hipStream_t s) {
  const int pieces = a.d / (f32 ? 4 : 8), lanes = token_lanes(pieces), per = kThreads / lanes;
  const unsigned grid = (unsigned)((a.tokens + per - 1) / per);
  if (f32) hipLaunchKernelGGL((k_combine_backward<true>), dim3(grid), dim3(kThreads), 0, s, a, lanes);
  else hipLaunchKernelGGL((k_combine_backward<false>), dim3(grid), dim3(kThreads), 0, s, a, lanes);
}

}  // namespace mlora
