// 4-bit weights with a scale and a zero point per group of inputs: quantizer,
// decoder, and the product over few rows.
//
// A weight is s (c - z): c its code, 0 to 15, s and z its group's, bf16.  The
// product takes no rounded weight: the matrix cores multiply the activations
// by 1 + c / 128, which bf16 holds exactly (the code is its low mantissa bits,
// one AND and one OR make two of them), and over a group
//   sum_k x_k s (c_k - z) = 128 s (sum_k x_k (1 + c_k / 128) - (1 + z / 128) sum_k x_k)
// with both sums in fp32; sum_k x_k is a product with ones.
#include "expert_common.hpp"
#include "affine_choice.hpp"

namespace mlora {

namespace {

constexpr uint32_t kCodeMask = 0x000f000fu, kOnes = 0x3f803f80u;

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Eight codes (one word) as 1 + c / 128, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4 bf16_of_codes(uint32_t w) {
  u32x4 o;
  o[0] = (w & kCodeMask) | kOnes;
  o[1] = ((w >> 4) & kCodeMask) | kOnes;
  o[2] = ((w >> 8) & kCodeMask) | kOnes;
  o[3] = ((w >> 12) & kCodeMask) | kOnes;
  return o;
}
// Eight bf16 in that order.
__device__ __forceinline__ u32x4 code_order(const u32x4& x) {
  u32x4 o;
  o[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
  o[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
  o[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
  o[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
  return o;
}

// Word q of lane group g (16 lanes each) to word g of lane group q.
__device__ __forceinline__ u32x4 transpose_groups(const u32x4& w) {
  typedef unsigned int u32p __attribute__((ext_vector_type(2)));
  const u32p a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const u32p b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const u32p c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const u32p d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

template <int G>
__device__ __forceinline__ float lanes_min(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v = fminf(v, __shfl_xor(v, d));
  return v;
}
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

}  // namespace

// Eight elements a lane, GROUP / 8 neighbouring lanes a group.  Bound by HBM.
template <class T, int GROUP>
__global__ __launch_bounds__(256) void k_affine_quantize(const T* X, int64_t rows, int cols, int64_t ld, bool symmetric,
                                                       uint32_t* codes, uint32_t* params, T* values) {
  constexpr int L = GROUP / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = rows * (cols / 8);
  // (cols / 8 is a multiple of L: a group's lanes are all in or all out)
  if (i >= n) return;
  const int64_t r = i / (cols / 8);
  const int c = (int)(i - r * (cols / 8)) * 8;
  float x[8];
  if constexpr (sizeof(T) == 4) {
    const u32x4* p = reinterpret_cast<const u32x4*>(X + r * ld + c);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = __uint_as_float(a[j]);
      x[4 + j] = __uint_as_float(b[j]);
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(X + r * ld + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(a[j] << 16);
      x[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
  float lo = 0.f, hi = 0.f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
    bad = bad || !(__builtin_fabsf(x[j]) <= 3.402823466e+38f);
  }
  lo = lanes_min<L>(lo);
  hi = lanes_max<L>(hi);
  bad = lanes_max<L>(bad ? 1.f : 0.f) > 0.f;
  const float s32 = symmetric ? fmaxf(hi, -lo) / 7.f : hi / 15.f - lo / 15.f;
  const uint32_t sb = pack_bf16x2(s32, s32) & 0xffffu;
  float s = __uint_as_float(sb << 16);
  float z = symmetric ? 8.f : s > 0.f ? fminf(fmaxf(__builtin_rintf(-lo / s), 0.f), 15.f) : 0.f;
  uint32_t word = 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // a group of zeros (or one whose scale underflows): code = zero point
    const float t = s > 0.f ? __builtin_rintf(x[j] / s) : 0.f;
    const float q = fminf(fmaxf(t + z, 0.f), 15.f);
    word |= (uint32_t)(bad ? 0.f : q) << (4 * j);
    v[j] = s * (q - z);
  }
  if (bad) {
    s = __uint_as_float(0x7fc00000u);
    z = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s;
  }
  codes[i] = word;
  if ((threadIdx.x & (L - 1)) == 0) params[i / L] = (__float_as_uint(s) & 0xffff0000u) | (__float_as_uint(z) >> 16);
  if (values) {
    if constexpr (sizeof(T) == 4) {
      u32x4* p = reinterpret_cast<u32x4*>(values + r * cols + c);
      p[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      p[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      *reinterpret_cast<u32x4*>(values + r * cols + c) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  }
}

// Eight weights a lane.  Bound by HBM.
template <int GROUP>
__global__ __launch_bounds__(256) void k_affine_decode(const uint32_t* codes, const uint32_t* params, int64_t n,
                                                     u32x4* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint32_t w = codes[i], p = params[i / (GROUP / 8)];
  const float s = __uint_as_float(p & 0xffff0000u), z = __uint_as_float(p << 16);
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = pack_bf16x2(s * ((float)((w >> (8 * j)) & 15) - z), s * ((float)((w >> (8 * j + 4)) & 15) - z));
  out[i] = o;
}

// Few rows per group: every weight is read once.  As in the bf16 product, a
// workgroup of eight waves owns 16 MB rows and 16 NB columns, its waves share
// the reduction, 512 inputs a wave and pass, and their sums meet in LDS in
// wave order.  Lane l = c + 16 g: the first matrix operand is row c of the
// activations, the second column c of the weights, inputs 8 g .. 8 g + 7 of
// the step's 32, and the lane holds rows 4 g .. 4 g + 3 of its column, so a
// group's scale and zero point are the lane's own.  Rows past the tile's are
// not loaded.  Codes come 16 bytes a lane, 32 neighbours of a column; with
// groups under 128 the words are exchanged between the lane groups, so that a
// step's 32 inputs lie in one group.
template <int GROUP, int MB, int NB>
__global__ __launch_bounds__(512) void k_affine_few(ExpertArgs a) {
  constexpr int COLS = 16 * NB, NW = 8, BM = 16 * MB, PG = 128 / GROUP, SG = GROUP / 32;
  __shared__ float sums[NW][BM][COLS + 4];
  const int nN = (a.N + COLS - 1) / COLS;
  const RowTile t = RowTiles<BM, 1>(a, nN).at(a, blockIdx.x);
  if (t.mrows <= 0) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int n0 = t.tn * COLS, K = a.K;

  const uint8_t* xp[MB];
  bool mine[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    mine[m] = 16 * m + c < t.mrows;
    xp[m] = a.A + source_row(a, a.ma, t.row0 + min(16 * m + c, t.mrows - 1)) * a.lda * 2;
  }
  const uint8_t* wp[NB];
  const uint32_t* pp[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int col = min(n0 + 16 * j + c, a.N - 1);
    wp[j] = a.B + (int64_t)t.e * a.b_expert + (int64_t)col * (K / 2);
    pp[j] = reinterpret_cast<const uint32_t*>(a.b_scale) + ((int64_t)t.e * a.N + col) * (K / GROUP);
  }

  f32x4 acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = {kOnes, kOnes, kOnes, kOnes};

  for (int k0 = 512 * w; k0 < K; k0 += 512 * NW) {
    u32x4 cw[NB][4];
    uint32_t pw[NB][4][PG];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (K is a multiple of 32: a lane's 32 codes are all in or all out; those out are read
      // from the row's start and their steps left out)
      const int kc = k0 + 128 * i + 32 * g, kk = kc < K ? kc : 0;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        cw[j][i] = *reinterpret_cast<const u32x4*>(wp[j] + kk / 2);
#pragma unroll
        for (int q = 0; q < PG; ++q) {
          const int kp = k0 + 128 * i + GROUP * q;
          pw[j][i][q] = pp[j][kp < K ? kp / GROUP : 0];
        }
      }
    }
    u32x4 xv[MB][4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // GROUP 128: any order of the piece's inputs will do, so the codes stay where they are
        const int k = k0 + 128 * i + (PG == 1 ? 32 * g + 8 * q : 32 * q + 8 * g);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          xv[m][i][q] = zero4();
          if (mine[m] && k < K) xv[m][i][q] = *reinterpret_cast<const u32x4*>(xp[m] + (int64_t)k * 2);
        }
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k0 + 128 * i >= K) break;
      u32x4 cc[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) cc[j] = PG == 1 ? cw[j][i] : transpose_groups(cw[j][i]);
#pragma unroll
      for (int p = 0; p < PG; ++p) {
        if (k0 + 128 * i + GROUP * p >= K) break;
        f32x4 xs[MB], ps[MB][NB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < NB; ++j) ps[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int q = p * SG; q < (p + 1) * SG; ++q) {
          u32x4 xo[MB];
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            xo[m] = code_order(xv[m][i][q]);
            xs[m] = mfma16(xo[m], ones, xs[m]);
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const u32x4 wv = bf16_of_codes(cc[j][q]);
#pragma unroll
            for (int m = 0; m < MB; ++m) ps[m][j] = mfma16(xo[m], wv, ps[m][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float s = __uint_as_float(pw[j][i][p] & 0xffff0000u) * 128.f;
          const float z = -1.f - __uint_as_float(pw[j][i][p] << 16) * (1.f / 128.f);
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] += s * __builtin_fmaf(z, xs[m][e], ps[m][j][e]);
        }
      }
    }
  }

  // acc[m][j][e]: row 16 m + 4 g + e, column 16 j + c
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < NB; ++j) sums[w][16 * m + 4 * g + e][16 * j + c] = acc[m][j][e];
  __syncthreads();
  for (int i = threadIdx.x; i < BM * COLS / 4; i += 512) {
    const int m = i / (COLS / 4), cc = 4 * (i % (COLS / 4));
    if (m >= t.mrows || n0 + cc >= a.N) continue;
    const int s = t.row0 + m, v = a.mc.by_order ? a.order[s] : s;
    if ((unsigned)v >= (unsigned)a.rows) continue;
    f32x4 sum = *reinterpret_cast<const f32x4*>(&sums[0][m][cc]);
#pragma unroll
    for (int q = 1; q < NW; ++q) sum += *reinterpret_cast<const f32x4*>(&sums[q][m][cc]);
    const u32x2 o = {pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.C) + (int64_t)v * a.ldc + n0 + cc) = o;
  }
}

namespace {

template <class T>
void quantize_of(const void* X, int64_t rows, int64_t cols, int64_t ld, int32_t group, bool symmetric, uint8_t* codes,
                 uint32_t* params, void* values, hipStream_t s) {
  const dim3 grid((unsigned)((rows * (cols / 8) + 255) / 256));
  auto* c = reinterpret_cast<uint32_t*>(codes);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, static_cast<const T*>(X), rows, (int)cols, ld, symmetric, c,
                       params, static_cast<T*>(values));
  };
  if (group == 32) go(k_affine_quantize<T, 32>);
  else if (group == 64) go(k_affine_quantize<T, 64>);
  else go(k_affine_quantize<T, 128>);
}

template <int MB, int NB>
void few_of(const ExpertArgs& a, int32_t group, hipStream_t s) {
  const unsigned grid = (unsigned)rows_grid_of(a, 16 * MB, 16 * NB);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(512), 0, s, a); };
  if (group == 32) go(k_affine_few<32, MB, NB>);
  else if (group == 64) go(k_affine_few<64, MB, NB>);
  else go(k_affine_few<128, MB, NB>);
}

}  // namespace

void launch_affine_quantize(bool f32, const void* X, int64_t rows, int64_t cols, int64_t ld, int32_t group,
                          bool symmetric, uint8_t* codes, uint32_t* params, void* values, hipStream_t s) {
  if (f32) quantize_of<float>(X, rows, cols, ld, group, symmetric, codes, params, values, s);
  else quantize_of<uint16_t>(X, rows, cols, ld, group, symmetric, codes, params, values, s);
}

void launch_affine_decode(const uint8_t* codes, const uint32_t* params, int64_t rows, int64_t cols, int32_t group,
                        uint16_t* out, hipStream_t s) {
  const int64_t n = rows * (cols / 8);
  const dim3 grid((unsigned)((n + 255) / 256));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, reinterpret_cast<const uint32_t*>(codes), params, n,
                       reinterpret_cast<u32x4*>(out));
  };
  if (group == 32) go(k_affine_decode<32>);
  else if (group == 64) go(k_affine_decode<64>);
  else go(k_affine_decode<128>);
}

void launch_affine_few(const ExpertArgs& a, int32_t group, hipStream_t s) {
  if (affine_few_rows(a) <= 16) few_of<1, 2>(a, group, s);
  else few_of<2, 2>(a, group, s);
}

}  // namespace mlora
