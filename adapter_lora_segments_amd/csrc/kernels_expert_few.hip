// Grouped expert products over few rows (single-token serving): every
// expert's weight is read once, so the time is the weight bytes' and what
// counts is loads in flight.  Weights and activations go straight from global
// memory to registers (no LDS on the way in); a workgroup of eight waves owns
// 16 MB rows and 16 NB (k-contiguous weights) or 64 (n-contiguous) columns,
// the waves share the reduction, and their fp32 sums meet in LDS at the end in
// wave order.  A wave's activations serve its NB column blocks, so more blocks
// mean fewer loads per weight byte and fewer workgroups.
// Bound by HBM when enough workgroups are in flight: 8 rows over 8 experts of
// 4096 x 4096 bf16, twelve sets of weights in turn 38 us (190 MB of chosen
// weights a call, 5.0 TB/s), one set over and over 28 us (168 MB, 6.0 TB/s, part
// of it from the last-level cache); by latency below that: 4 rows, 4096 ->
// 14336, MXFP4 codes (31 MB) 12.4 us, 224 workgroups of 128 KB of codes each.
#include "expert_choice.hpp"
#include "expert_common.hpp"

namespace mlora {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Weight forms.
enum { W16_KC = 0, W16_NC = 1, W32_KC = 2, W32_NC = 3, W4_A16 = 4, W4_A4 = 5 };

template <int FORM, int NB>
struct FewTraits {
  static constexpr bool F32 = FORM == W32_KC || FORM == W32_NC;
  static constexpr bool WIDE = FORM == W16_NC || FORM == W32_NC;  // 64 columns, four per lane
  static constexpr int COLS = WIDE ? 64 : 16 * NB;
  static constexpr int NJ = WIDE ? 4 : NB;                        // accumulators per row block
  // one batch of loads covers this much of the reduction
  static constexpr int KD = FORM == W16_KC ? 128 : FORM == W16_NC ? 32 : FORM == W32_KC ? 64 : FORM == W32_NC ? 16
                            : 512;
};

__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ f32x4 mfma16f(float a, float b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

}  // namespace

// Lane l = c + 16 g.  The matrix instruction's first operand is the weight
// (row i = a column of Y), the second the activations (column j = a row of
// Y); lane l supplies index c of both with reduction piece g, and holds
// D[4 g + x][c]: four columns of row c.
template <int FORM, int MB, int NB>
__global__ __launch_bounds__(512) void k_expert_few(ExpertArgs a) {
  using TR = FewTraits<FORM, NB>;
  constexpr int COLS = TR::COLS, NJ = TR::NJ, KD = TR::KD, NW = 8, BM = 16 * MB;
  __shared__ float sums[NW][BM][COLS + 4];
  const int nN = (a.N + COLS - 1) / COLS;
  const RowTile t = RowTiles<BM, 1>(a, nN).at(a, blockIdx.x);
  if (t.mrows <= 0) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  const int n0 = t.tn * COLS, K = a.K;

  constexpr int ESZ = TR::F32 ? 4 : 2;
  const uint8_t* xp[MB];
  const uint8_t* xs[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int64_t row = source_row(a, a.ma, t.row0 + min(16 * m + c, t.mrows - 1));
    if constexpr (FORM == W4_A4) {
      xp[m] = a.A + row * (K / 2);
      xs[m] = a.a_scale + row * (K / 32);
    } else {
      xp[m] = a.A + row * a.lda * ESZ;
      xs[m] = nullptr;
    }
  }
  const uint8_t* const We = a.B + (int64_t)t.e * a.b_expert;
  // column block j of this lane (WIDE: its four columns)
  const uint8_t* wp[NB];
  const uint8_t* ws[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int col = TR::WIDE ? min(n0 + 4 * c, a.N - 4) : min(n0 + 16 * j + c, a.N - 1);
    ws[j] = nullptr;
    if constexpr (FORM == W4_A16 || FORM == W4_A4) {
      wp[j] = We + (int64_t)col * (K / 2);
      ws[j] = a.b_scale + ((int64_t)t.e * a.N + col) * (K / 32);
    } else if constexpr (TR::WIDE) {
      wp[j] = We + (int64_t)col * ESZ;
    } else {
      wp[j] = We + (int64_t)col * a.ldb * ESZ;
    }
  }

  f32x4 acc[MB][NJ];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int nbatch = (K + KD - 1) / KD;
  for (int it = w; it < nbatch; it += NW) {
    const int k0 = it * KD;
    if constexpr (FORM == W16_KC || FORM == W32_KC) {
      // piece i, lane group g: 16 bytes at reduction index k0 + EP (4 i + g)
      constexpr int EP = 16 / ESZ;
      u32x4 wv[NB][4], xv[MB][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + EP * (4 * i + g);
        const bool on = k < K;
        const int kk = on ? k : 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          wv[j][i] = *reinterpret_cast<const u32x4*>(wp[j] + (int64_t)kk * ESZ);
          wv[j][i] = on ? wv[j][i] : zero4();
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          xv[m][i] = *reinterpret_cast<const u32x4*>(xp[m] + (int64_t)kk * ESZ);
          xv[m][i] = on ? xv[m][i] : zero4();
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            if constexpr (FORM == W16_KC) {
              acc[m][j] = mfma16(wv[j][i], xv[m][i], acc[m][j]);
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                acc[m][j] = mfma16f(__uint_as_float(wv[j][i][x]), __uint_as_float(xv[m][i][x]), acc[m][j]);
            }
          }
    } else if constexpr (FORM == W16_NC) {
      // lane: columns 4 c .. 4 c + 3 of reduction rows k0 + 8 g + i
      u32x2 wv[8];
      u32x4 xv[MB];
      const int kx = k0 + 8 * g;
      const bool on = kx < K;          // K is a multiple of 8: a lane's rows are all in or all out
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wv[i] = *reinterpret_cast<const u32x2*>(wp[0] + (int64_t)(on ? kx + i : 0) * a.ldb * 2);
        if (!on) wv[i] = u32x2{0u, 0u};
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        xv[m] = *reinterpret_cast<const u32x4*>(xp[m] + (int64_t)(on ? kx : 0) * 2);
        if (!on) xv[m] = zero4();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {    // column 4 c + j: its eight rows packed
        u32x4 p;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[q] = __builtin_amdgcn_perm(wv[2 * q + 1][j >> 1], wv[2 * q][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[m][j] = mfma16(p, xv[m], acc[m][j]);
      }
    } else if constexpr (FORM == W32_NC) {
      // lane: columns 4 c .. 4 c + 3 of reduction rows k0 + 4 g + i
      u32x4 wv[4], xv[MB];
      const int kx = k0 + 4 * g;
      const bool on = kx < K;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wv[i] = *reinterpret_cast<const u32x4*>(wp[0] + (int64_t)(on ? kx + i : 0) * a.ldb * 4);
        if (!on) wv[i] = zero4();
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        xv[m] = *reinterpret_cast<const u32x4*>(xp[m] + (int64_t)(on ? kx : 0) * 4);
        if (!on) xv[m] = zero4();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int m = 0; m < MB; ++m)
            acc[m][j] = mfma16f(__uint_as_float(wv[i][j]), __uint_as_float(xv[m][i]), acc[m][j]);
    } else if constexpr (FORM == W4_A16) {
      // four pieces of 128: lane block g of each, 32 codes in 16 bytes
      u32x4 cw[NB][4], xv[MB][4][4];
      uint32_t sw[NB][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 128 * i;
        const int kk = k < K ? k : 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          cw[j][i] = *reinterpret_cast<const u32x4*>(wp[j] + kk / 2 + 16 * g);
          sw[j][i] = ws[j][kk / 32 + g];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 128 * i;
        const int kk = k < K ? k : 0;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            xv[m][i][q] = *reinterpret_cast<const u32x4*>(xp[m] + (int64_t)(kk + 32 * g + 8 * q) * 2);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (k0 + 128 * i >= K) break;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float sc = __uint_as_float(sw[j][i] << 23);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x4 wv = bf16_of_e2m1(cw[j][i][q], sc);
#pragma unroll
            for (int m = 0; m < MB; ++m) acc[m][j] = mfma16(wv, xv[m][i][q], acc[m][j]);
          }
        }
      }
    } else {
      // four pieces of 128: lane block g of each
      u32x4 cw[NB][4], xv[MB][4];
      int sw[NB][4], sx[MB][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 128 * i;
        const bool on = k < K;
        const int kk = on ? k : 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          cw[j][i] = *reinterpret_cast<const u32x4*>(wp[j] + kk / 2 + 16 * g);
          sw[j][i] = ws[j][kk / 32 + g];
          if (!on) {
            cw[j][i] = zero4();
            sw[j][i] = 0;
          }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          xv[m][i] = *reinterpret_cast<const u32x4*>(xp[m] + kk / 2 + 16 * g);
          sx[m][i] = xs[m][kk / 32 + g];
          if (!on) {
            xv[m][i] = zero4();
            sx[m][i] = 0;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[m][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                __builtin_bit_cast(i32x8, __builtin_shufflevector(cw[j][i], zero4(), 0, 1, 2, 3, 4, 5, 6, 7)),
                __builtin_bit_cast(i32x8, __builtin_shufflevector(xv[m][i], zero4(), 0, 1, 2, 3, 4, 5, 6, 7)),
                acc[m][j], 4, 4, 0, sw[j][i], 0, sx[m][i]);
    }
  }

  // acc[m][j][x]: row 16 m + c, column 16 j + 4 g + x, or (WIDE) 4 (4 g + x) + j
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        sums[w][16 * m + c][TR::WIDE ? 4 * (4 * g + x) + j : 16 * j + 4 * g + x] = acc[m][j][x];
  __syncthreads();
  // four columns per thread
  for (int i = threadIdx.x; i < BM * COLS / 4; i += 512) {
    const int m = i / (COLS / 4), cc = 4 * (i % (COLS / 4));
    if (m >= t.mrows || n0 + cc >= a.N) continue;
    const int s = t.row0 + m, v = a.mc.by_order ? a.order[s] : s;
    if ((unsigned)v >= (unsigned)a.rows) continue;
    f32x4 sum = *reinterpret_cast<const f32x4*>(&sums[0][m][cc]);
#pragma unroll
    for (int q = 1; q < NW; ++q) sum += *reinterpret_cast<const f32x4*>(&sums[q][m][cc]);
    if constexpr (TR::F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.C) + (int64_t)v * a.ldc + n0 + cc) = sum;
    } else {
      const u32x2 o = {pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.C) + (int64_t)v * a.ldc + n0 + cc) = o;
    }
  }
}

namespace {

template <int FORM, int MB, int NB>
void few(const ExpertArgs& a, hipStream_t s) {
  constexpr int COLS = FewTraits<FORM, NB>::COLS;
  const int64_t grid = max_row_tiles(a.rows, a.offsets ? a.n_experts : 1, 16 * MB) * ((a.N + COLS - 1) / COLS);
  hipLaunchKernelGGL((k_expert_few<FORM, MB, NB>), dim3((unsigned)grid), dim3(512), 0, s, a);
}
template <int FORM>
void few_of(int rows, int cols, const ExpertArgs& a, hipStream_t s) {
  constexpr bool wide = FORM == W16_NC || FORM == W32_NC, f4 = FORM == W4_A16 || FORM == W4_A4;
  if constexpr (wide) {
    if (rows == 16) return few<FORM, 1, 1>(a, s);
    if (rows == 32) return few<FORM, 2, 1>(a, s);
    few<FORM, 4, 1>(a, s);
  } else {
    if (rows == 16 && cols == 16) return few<FORM, 1, 1>(a, s);
    if (rows == 16 && cols == 32) return few<FORM, 1, 2>(a, s);
    if (rows == 32 && cols == 32) return few<FORM, 2, 2>(a, s);
    if constexpr (f4) {
      if (rows == 16) return few<FORM, 1, 4>(a, s);
      few<FORM, 2, 4>(a, s);
    } else {
      if (rows == 32 && cols == 16) return few<FORM, 2, 1>(a, s);
      if constexpr (FORM == W16_KC)
        if (rows == 32) return few<FORM, 2, 4>(a, s);
      few<FORM, 4, 2>(a, s);
    }
  }
}

}  // namespace

void launch_expert_few(ExpertForm form, bool b_kc, int rows, int cols, const ExpertArgs& a, hipStream_t s) {
  switch (form) {
    case ExpertForm::kBf16:
      if (b_kc) few_of<W16_KC>(rows, cols, a, s);
      else few_of<W16_NC>(rows, cols, a, s);
      break;
    case ExpertForm::kF32:
      if (b_kc) few_of<W32_KC>(rows, cols, a, s);
      else few_of<W32_NC>(rows, cols, a, s);
      break;
    case ExpertForm::kW4A16: few_of<W4_A16>(rows, cols, a, s); break;
    case ExpertForm::kW4A4: few_of<W4_A4>(rows, cols, a, s); break;
  }
}

}  // namespace mlora
