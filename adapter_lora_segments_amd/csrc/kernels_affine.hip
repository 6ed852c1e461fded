// 4-bit weights with a scale and a zero point per group of inputs: quantizer,
// decoder, and the product over few rows.
//
// A weight is s (c - z): c its code, 0 to 15, s and z its group's, bf16.  The
// product takes no rounded weight: the matrix cores multiply the activations
// by 1 + c / 16, which bf16 holds exactly (the code is its high mantissa bits,
// a shift and one AND and OR make two of them), and over a group
//   sum_k x_k s (c_k - z) = 16 s (sum_k x_k (1 + c_k / 16) - (1 + z / 16) sum_k x_k)
// with both sums in fp32; sum_k x_k is a product with ones.  The difference loses
// what the ones add to the codes, about two bits of the sums (1 + c / 128, which
// saves the shift of a word's first codes, loses five and takes as long but for 1%).
// A product has 13 bits, so the sums are exact, and weights that are zero (c = z)
// give zeros, where a group's activations differ by no more than 2^(11 - log2 group)
// in size; over 4096 normal ones a column of zeros is off by 6e-5 s at most (5e-4
// with 1 + c / 128).
#include "expert_common.hpp"
#include "affine_choice.hpp"

namespace mlora {

namespace {

constexpr uint32_t kCodeMask = 0x00780078u, kOnes = 0x3f803f80u;

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Eight codes (one word) as 1 + c / 16, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4 bf16_of_codes(uint32_t w) {
  u32x4 o;
  o[0] = ((w << 3) & kCodeMask) | kOnes;
  o[1] = ((w >> 1) & kCodeMask) | kOnes;
  o[2] = ((w >> 5) & kCodeMask) | kOnes;
  o[3] = ((w >> 9) & kCodeMask) | kOnes;
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

}  // namespace

// Eight elements a lane, GROUP / 8 neighbouring lanes a group (`split` divides by
// a row's eights).  Bound by HBM, once the arithmetic is short: an element's
// quotient x / s rounded to fp32 comes from a product with 1 / s in 64 bits,
// which rounds alike, since s has 8 bits and x 24: x / s is no nearer than 2^-34
// of itself to the middle of two fp32 numbers.  14336 x 4096 in bf16 with values
// 43 us (6.2 TB/s; 59 with divisions), without 36; fp32 91 and 44 us.
template <class T, int GROUP>
__global__ __launch_bounds__(256) void k_affine_quantize(const T* X, uint32_t n, DivBy split, int cols, int64_t ld,
                                                       bool symmetric, uint32_t* codes, uint32_t* params, T* values) {
  constexpr int L = GROUP / 8;
  constexpr float kInf = __builtin_inff();
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  // (cols / 8 is a multiple of L: a group's lanes are all in or all out)
  if (i >= n) return;
  const uint32_t r = div_fast(i, split);
  const int c = (int)(i - r * (uint32_t)(cols / 8)) * 8;
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
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
    nan = nan || x[j] != x[j];
  }
  hi = nan ? kInf : hi;
  lo = across<L>(lo, [](float a, float b) { return fminf(a, b); });
  hi = across<L>(hi, [](float a, float b) { return fmaxf(a, b); });
  const bool bad = hi == kInf || lo == -kInf;
  const float s32 = symmetric ? fmaxf(hi, -lo) / 7.f : hi / 15.f - lo / 15.f;
  const uint32_t sb = pack_bf16x2(s32, s32) & 0xffffu;
  float s = __uint_as_float(sb << 16);
  // (a group of zeros, or one whose scale underflows: code = zero point)
  const double inv = s > 0.f ? 1.0 / (double)s : 0.0;
  auto steps = [&](float v) { return __builtin_rintf((float)((double)v * inv)); };
  float z = symmetric ? 8.f : fminf(fmaxf(steps(-lo), 0.f), 15.f);
  uint32_t word = 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = fminf(fmaxf(steps(x[j]) + z, 0.f), 15.f);
    word |= (uint32_t)q << (4 * j);
    v[j] = s * (q - z);
  }
  if (bad) {
    s = __uint_as_float(0x7fc00000u);
    z = 0.f;
    word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s;
  }
  codes[i] = word;
  if ((threadIdx.x & (L - 1)) == 0) params[i / L] = (__float_as_uint(s) & 0xffff0000u) | (__float_as_uint(z) >> 16);
  if (values) {
    if constexpr (sizeof(T) == 4) {
      u32x4* p = reinterpret_cast<u32x4*>(values + (int64_t)r * cols + c);
      p[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      p[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
      *reinterpret_cast<u32x4*>(values + (int64_t)r * cols + c) =
          u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
  }
}

// Eight weights a lane.  Bound by HBM, four fifths of it stores: 14336 x 4096 30 us
// (4.9 TB/s).
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

// Few rows per group: every weight is read once, so what counts is bytes in
// flight.  A workgroup of eight waves owns up to RB rows and 16 NB CS columns:
// CS waves side by side, and 8 / CS that share the reduction, neighbouring
// pieces of 128 inputs each, whose sums meet in LDS in their order.  A wave asks
// for activations and then for four pieces of weights (16 bytes a lane: 32
// neighbouring codes of a column), and multiplies when both are there; the
// activations wait in LDS, 512 inputs of every row, since the registers hold the
// weights in flight.
// Lane l = c + 16 g: the first matrix operand is row c of the activations, the
// second column c of the weights, and the lane holds rows 4 g .. 4 g + 3 of its
// column, so a group's scale and zero point are the lane's own.  With groups
// under 128 the words of a piece are exchanged between the lane groups, so that
// a step's 32 inputs lie in one group.
// What bounds it: up to K = 4096 one round of loads, decoded when they come (vector
// instructions busy 30 to 40%, matrix ones 8%, HBM half): 1 row, N = 14336 9.6 us
// (3.3 TB/s), 16 rows 12.2; 32 rows over 8 experts, N = 4096, groups of 64 22 us
// (3.4 TB/s; 512 workgroups, two a CU, at once).  Weights before activations were
// slower (10.6 us for the row).  Over longer inputs a wave takes one round after
// the other, and where N is short as well few workgroups do (K = 14336, N = 4096: 1
// row 10.4 us, 16 rows 17, 64 rows 32, the weights' bytes 6).  Asking for the
// next four pieces before these are multiplied was measured at K = 4096 only, where
// there are none: there it costs registers and gains nothing.
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

template <int GROUP, int RB, int NB, int CS>
__global__ __launch_bounds__(512, RB <= 8 ? 4 : 2) void k_affine_few(ExpertArgs a) {
  constexpr int KS = 8 / CS, COLS = 16 * NB * CS, MB = RB > 16 ? RB / 16 : 1;
  constexpr int PG = 128 / GROUP, SG = GROUP / 32, XR = 1024 + 16;
  constexpr int XB = KS * RB * XR, SB = KS * RB * (COLS + 4) * 4;
  __shared__ u32x4 lds[(XB > SB ? XB : SB) / 16];
  const int nN = (a.N + COLS - 1) / COLS;
  const RowTile t = RowTiles<RB, 1>(a, nN).at(a, blockIdx.x);
  if (t.mrows <= 0) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  const int ks = w / CS, cs = w % CS, n0 = t.tn * COLS, K = a.K;

  // a wave's pieces
  const int pieces = (K + 127) / 128, share = (pieces + KS - 1) / KS;
  const int kend = min(K, (ks + 1) * share * 128);
  // codes and parameters by 32-bit offsets from the tile's first column
  const uint8_t* const wt = a.B + (int64_t)t.e * a.b_expert + (int64_t)n0 * (K / 2);
  const uint8_t* const pt = a.b_scale + ((int64_t)t.e * a.N + n0) * (K / GROUP) * 4;
  uint32_t col[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) col[j] = (uint32_t)min(16 * NB * cs + 16 * j + c, a.N - 1 - n0);
  // activations: the waves of a part of the reduction copy its rows in turn, lane l a row's 16 bytes l
  constexpr int XC = RB / CS;
  const uint8_t* xp[XC];
#pragma unroll
  for (int r = 0; r < XC; ++r) xp[r] = a.A + source_row(a, a.ma, t.row0 + min(CS * r + cs, t.mrows - 1)) * a.lda * 2;
  char* const xw = reinterpret_cast<char*>(lds) + ks * RB * XR;

  f32x4 acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = {kOnes, kOnes, kOnes, kOnes};

  for (int i0 = 0; i0 < share; i0 += 4) {
    const int k0 = (ks * share + i0) * 128;
    u32x4 xv[XC], cw[NB][4];
    uint32_t pw[NB][4 * PG];
    {
      const int k = k0 + 8 * lane, kk = k < K ? k : 0;
#pragma unroll
      for (int r = 0; r < XC; ++r) xv[r] = *reinterpret_cast<const u32x4*>(xp[r] + (int64_t)kk * 2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (K is a multiple of 32: a lane's 32 codes are all in or all out; those out are read
      // from the column's start and their steps left out)
      const int kc = k0 + 128 * i + 32 * g, kk = kc < K ? kc : 0;
#pragma unroll
      for (int j = 0; j < NB; ++j)
        cw[j][i] = *reinterpret_cast<const u32x4*>(wt + (col[j] * (uint32_t)(K / 2) + (uint32_t)kk / 2));
    }
    if (k0 + 512 <= K) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int q = 0; q < PG; ++q) {
          const u32x4 v = *reinterpret_cast<const u32x4_a4*>(pt + (col[j] * (uint32_t)(K / GROUP) + (uint32_t)(k0 / GROUP + 4 * q)) * 4);
#pragma unroll
          for (int x = 0; x < 4; ++x) pw[j][4 * q + x] = v[x];
        }
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int q = 0; q < 4 * PG; ++q) {
          const int kp = k0 + GROUP * q, kk = kp < K ? kp : 0;
          pw[j][q] = *reinterpret_cast<const uint32_t*>(pt + (col[j] * (uint32_t)(K / GROUP) + (uint32_t)kk / GROUP) * 4);
        }
    }
    // (CS = 1: in the wave's own LDS, and a wave's accesses run in order)
    if (CS > 1 && i0 > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < XC; ++r) *reinterpret_cast<u32x4*>(xw + (CS * r + cs) * XR + 16 * lane) = code_order(xv[r]);
    if (CS > 1) __syncthreads();
    else __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k0 + 128 * i >= kend) break;
      u32x4 cc[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) cc[j] = PG == 1 ? cw[j][i] : transpose_groups(cw[j][i]);
#pragma unroll
      for (int p = 0; p < PG; ++p) {
        if (k0 + 128 * i + GROUP * p >= kend) break;
        f32x4 xs[MB], ps[MB][NB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < NB; ++j) ps[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int q = p * SG; q < (p + 1) * SG; ++q) {
          // GROUP 128: any order of the piece's inputs will do, so the codes stay where they are
          u32x4 x[MB];
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            x[m] = *reinterpret_cast<const u32x4*>(xw + (16 * m + min(c, RB - 1)) * XR + 256 * i +
                                                   (PG == 1 ? 64 * g + 16 * q : 64 * q + 16 * g));
            xs[m] = mfma16(x[m], ones, xs[m]);
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const u32x4 wv = bf16_of_codes(cc[j][q]);
#pragma unroll
            for (int m = 0; m < MB; ++m) ps[m][j] = mfma16(x[m], wv, ps[m][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint32_t pj = pw[j][PG * i + p];
          const float s = __uint_as_float(pj & 0xffff0000u) * 16.f;
          const float z = -1.f - __uint_as_float(pj << 16) * (1.f / 16.f);
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] += s * __builtin_fmaf(z, xs[m][e], ps[m][j][e]);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }

  // acc[m][j][e]: row 16 m + 4 g + e, column 16 NB cs + 16 j + c
  __syncthreads();
  typedef float Sums[RB][COLS + 4];
  Sums* const sums = reinterpret_cast<Sums*>(lds);
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (4 * g + e < RB) sums[ks][16 * m + 4 * g + e][16 * NB * cs + 16 * j + c] = acc[m][j][e];
  __syncthreads();
  for (int i = threadIdx.x; i < RB * COLS / 4; i += 512) {
    const int m = i / (COLS / 4), cc = 4 * (i % (COLS / 4));
    if (m >= t.mrows || n0 + cc >= a.N) continue;
    const int s = t.row0 + m, v = a.mc.by_order ? a.order[s] : s;
    if ((unsigned)v >= (unsigned)a.rows) continue;
    f32x4 sum = *reinterpret_cast<const f32x4*>(&sums[0][m][cc]);
#pragma unroll
    for (int q = 1; q < KS; ++q) sum += *reinterpret_cast<const f32x4*>(&sums[q][m][cc]);
    const u32x2 o = {pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.C) + (int64_t)v * a.ldc + n0 + cc) = o;
  }
}

namespace {

template <class T>
void quantize_of(const void* X, int64_t rows, int64_t cols, int64_t ld, int32_t group, bool symmetric, uint8_t* codes,
                 uint32_t* params, void* values, hipStream_t s) {
  const uint32_t n = (uint32_t)(rows * (cols / 8));      // (below 2^31)
  auto* c = reinterpret_cast<uint32_t*>(codes);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((n + 255) / 256), dim3(256), 0, s, static_cast<const T*>(X), n,
                       div_by((int32_t)(cols / 8)), (int)cols, ld, symmetric, c, params, static_cast<T*>(values));
  };
  if (group == 32) go(k_affine_quantize<T, 32>);
  else if (group == 64) go(k_affine_quantize<T, 64>);
  else go(k_affine_quantize<T, 128>);
}

template <int RB, int NB, int CS>
void few_of(const ExpertArgs& a, int32_t group, hipStream_t s) {
  const unsigned grid = (unsigned)affine_grid(a, RB, 16 * NB * CS);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(512), 0, s, a); };
  if (group == 32) go(k_affine_few<32, RB, NB, CS>);
  else if (group == 64) go(k_affine_few<64, RB, NB, CS>);
  else go(k_affine_few<128, RB, NB, CS>);
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

void launch_affine_few(const ExpertArgs& a, int32_t group, int rows, int cols, hipStream_t s) {
  if (rows == 4) return few_of<4, 1, 1>(a, group, s);
  if (rows == 8) return cols == 16 ? few_of<8, 1, 1>(a, group, s) : few_of<8, 2, 1>(a, group, s);
  if (rows == 16 && cols == 16) return few_of<16, 1, 1>(a, group, s);
  if (rows == 16) return cols == 32 ? few_of<16, 1, 2>(a, group, s) : few_of<16, 2, 2>(a, group, s);
  if (cols == 32) return few_of<32, 1, 2>(a, group, s);
  if (cols == 64) return few_of<32, 2, 2>(a, group, s);
  few_of<32, 2, 4>(a, group, s);
}

}  // namespace mlora
