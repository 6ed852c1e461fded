// MXFP4 quantizer: blocks of 32 elements to E2M1 codes and one E8M0 scale,
// by the OCP microscaling conversion.  Reads 2 or 4 bytes and writes 17/32
// bytes per element (plus the decoded values when asked for): HBM-bound, so
// every load, code store and value store is 16 bytes, 4 bytes or more per
// lane over consecutive lanes, and a block's maximum crosses lanes in
// registers, not through LDS.  Measured: 14336 x 4096 bf16 with values (265 MB)
// 57 us, 4.6 TB/s against 5.1 of a large copy; 8192 x 4096 bf16, codes only (85
// MB) 28 us; 1024 x 4096 fp32 down columns with values 9.2 us.
#include "device_common.hpp"
#include "experts.hpp"

namespace mlora {

namespace {

// Largest magnitude of a block (fp32 bits, sign cleared) -> shared exponent.
// 255 in the exponent field: an infinity or a NaN.
__device__ __forceinline__ int shared_exponent(uint32_t amax) {
  if (amax == 0u) return -127;
  const int ex = (int)(amax >> 23);
  // below the normal range the leading bit of the fraction sets the exponent
  const int fl = ex > 0 ? ex - 127 : -118 - __clz((int)amax);
  return max(-127, fl - 2);
}

// Code of x with shared exponent e (four bits), and the decoded value.  The
// E2M1 grid steps by 1/2 below 2, by 1 below 4 and by 2 below 8: an element
// is rounded to a whole number of steps, ties to even (an even number of
// steps is an even code), and 8 saturates to 6.  Scaling by a power of two
// is exact; elements far below the block's maximum may become subnormal but
// round to 0 all the same.
__device__ __forceinline__ uint32_t e2m1_of(float x, int e, float& value) {
  const float a = fabsf(ldexpf(x, -e));
  const float up = a < 2.f ? 2.f : (a < 4.f ? 1.f : 0.5f);
  const float down = a < 2.f ? 0.5f : (a < 4.f ? 1.f : 2.f);
  const int first = a < 2.f ? 0 : (a < 4.f ? 2 : 4);
  float m = rintf(a * up);
  m = a >= 4.f ? fminf(m, 3.f) : m;
  value = copysignf(ldexpf(m * down, e), x);
  return ((uint32_t)m + (uint32_t)first) | ((__float_as_uint(x) >> 28) & 8u);
}

template <class T>
struct Elems;  // elements of one 16-byte vector
template <>
struct Elems<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const u32x4& v, int i) {
    return __uint_as_float((i & 1) ? (v[i >> 1] & 0xFFFF0000u) : (v[i >> 1] << 16));
  }
  // exact: at most two significant bits
  static __device__ __forceinline__ void set(u32x4& v, int i, float x) {
    const uint32_t b = __float_as_uint(x) >> 16;
    v[i >> 1] = (i & 1) ? (v[i >> 1] | (b << 16)) : b;
  }
};
template <>
struct Elems<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const u32x4& v, int i) { return __uint_as_float(v[i]); }
  static __device__ __forceinline__ void set(u32x4& v, int i, float x) { v[i] = __float_as_uint(x); }
};

}  // namespace

// Blocks along a row: four lanes share a block, eight elements each.
template <class T>
__global__ __launch_bounds__(256) void k_quant_mx4_rows(const T* X, int64_t rows, int64_t cols, int64_t ld,
                                                        uint8_t* codes, uint8_t* scales, T* values) {
  constexpr int V = 8 / Elems<T>::N;              // 16-byte vectors per lane
  const int64_t per_row = cols / 8, n = rows * per_row;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;                             // n is a multiple of 4: whole blocks leave
  const int64_t r = i / per_row, c = (i - r * per_row) * 8;
  const u32x4* src = reinterpret_cast<const u32x4*>(X + r * ld + c);
  u32x4 v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = src[j];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    amax = max(amax, __float_as_uint(Elems<T>::get(v[j / Elems<T>::N], j % Elems<T>::N)) & 0x7FFFFFFFu);
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
  const bool bad = amax >= 0x7F800000u;
  const int e = shared_exponent(amax);
  uint32_t word = 0;
  u32x4 out[V];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float val;
    const uint32_t code = e2m1_of(Elems<T>::get(v[j / Elems<T>::N], j % Elems<T>::N), e, val);
    word |= code << (4 * j);
    Elems<T>::set(out[j / Elems<T>::N], j % Elems<T>::N, bad ? __builtin_nanf("") : val);
  }
  reinterpret_cast<uint32_t*>(codes)[i] = bad ? 0u : word;
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = bad ? (uint8_t)255 : (uint8_t)(e + 127);
  if (values) {
    u32x4* dst = reinterpret_cast<u32x4*>(values + r * cols + c);
#pragma unroll
    for (int j = 0; j < V; ++j) dst[j] = out[j];
  }
}

// Blocks down a column: a wave takes 32 rows and 16 vectors of columns; lane
// (c = lane % 16, g = lane / 16) holds rows 8 g .. 8 g + 7 of vector c, so a
// column's maximum is one lane's eight rows and two exchanges.
template <class T>
__global__ __launch_bounds__(256) void k_quant_mx4_down(const T* X, int64_t rows, int64_t cols, int64_t ld,
                                                        uint8_t* codes, uint8_t* scales, T* values) {
  constexpr int N = Elems<T>::N;
  const int lane = threadIdx.x & 63;
  const int64_t nb = rows / 32;
  const int64_t kb = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);   // the workgroup's waves: four blocks of rows
  const int64_t c = (int64_t)blockIdx.y * (16 * N) + (lane & 15) * N;
  if (kb >= nb) return;
  const bool on = c < cols;
  const int64_t cc = on ? c : 0;
  const int64_t r0 = kb * 32 + 8 * (lane >> 4);
  u32x4 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const u32x4*>(X + (r0 + j) * ld + cc);
  int e[N];
  bool bad[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(Elems<T>::get(v[j], i)) & 0x7FFFFFFFu);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 16));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
    bad[i] = amax >= 0x7F800000u;
    e[i] = shared_exponent(amax);
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((i & 3) == (lane >> 4)) scales[(c + i) * nb + kb] = bad[i] ? (uint8_t)255 : (uint8_t)(e[i] + 127);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t word = 0;
    u32x4 out;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float val;
      const uint32_t code = e2m1_of(Elems<T>::get(v[j], i), e[i], val);
      word |= (bad[i] ? 0u : code) << (4 * i);
      Elems<T>::set(out, i, bad[i] ? __builtin_nanf("") : val);
    }
    uint8_t* dst = codes + (r0 + j) * (cols / 2) + c / 2;
    if (N == 8) *reinterpret_cast<uint32_t*>(dst) = word;
    else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)word;
    if (values) *reinterpret_cast<u32x4*>(values + (r0 + j) * cols + c) = out;
  }
}

namespace {

template <class T>
void launch_quant(bool down, const void* X, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                  void* values, hipStream_t s) {
  const T* x = static_cast<const T*>(X);
  T* out = static_cast<T*>(values);
  if (down) {
    const int64_t wide = 16 * Elems<T>::N;
    const dim3 grid((unsigned)((rows / 32 + 3) / 4), (unsigned)((cols + wide - 1) / wide));
    hipLaunchKernelGGL((k_quant_mx4_down<T>), grid, dim3(256), 0, s, x, rows, cols, ld, codes, scales, out);
  } else {
    const int64_t n = rows * (cols / 8);
    hipLaunchKernelGGL((k_quant_mx4_rows<T>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, x, rows, cols, ld,
                       codes, scales, out);
  }
}

}  // namespace

void launch_quant_mx4(bool f32, bool down, const void* X, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                      uint8_t* scales, void* values, hipStream_t s) {
  if (rows <= 0 || cols <= 0) return;
  if (f32) launch_quant<float>(down, X, rows, cols, ld, codes, scales, values, s);
  else launch_quant<uint16_t>(down, X, rows, cols, ld, codes, scales, values, s);
}

}  // namespace mlora
