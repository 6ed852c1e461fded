// 4-bit weights with a scale and a zero point per group, over many rows: a
// tile of 32 FI rows and 128 columns a workgroup, four waves side by side (KS
// times four, which take the reduction's steps in turn).
//
// A wave's weights go from memory straight into its registers, 4 bits each:
// nobody else needs them.  They become bf16 there, s c - s z by one fused
// multiply-add in fp32 and one rounding, while the matrix instructions of the
// step before run, so no decoded copy exists.  The activations, which all four
// waves need, go through LDS, 128 inputs a step in two buffers: a step's loads
// are in flight while the step before is multiplied.
// Lane l = c + 32 h of a wave holds column c: 16 bytes are 32 neighbouring
// inputs, the step's blocks 2 u + h for u = 0, 1; word q of them and chunk
// 8 u + 4 h + q of the activations make one matrix instruction's 16 inputs.
// A block of 32 lies in one group, so its scale is the lane's own.
#include "affine_choice.hpp"
#include "expert_common.hpp"

namespace mlora {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight codes (one word) to bf16, c s + o.  Codes in the low bits of two halves
// are fp16 denormals, c 2^-24 exactly, which the mixed multiply-add takes as
// they are: s holds 2^24 of the scale.
__device__ __forceinline__ u32x4 bf16_of_word(uint32_t w, float s, float o) {
  f16x2 c[4];                        // codes j and j + 4
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = __builtin_bit_cast(f16x2, (w >> (4 * j)) & 0x000f000fu);
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = pack_bf16x2(__builtin_fmaf((float)c[2 * (j & 1)][j >> 1], s, o),
                       __builtin_fmaf((float)c[2 * (j & 1) + 1][j >> 1], s, o));
  return r;
}

// Meets the other waves once this wave's LDS accesses are done; loads stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

}  // namespace

template <int GROUP, int FI, int KS>
__global__ __launch_bounds__(256 * KS, 2) void k_affine_tile(ExpertArgs a) {
  constexpr int BM = 32 * FI, BN = 128, KD = 128, NP = BM / 16, D = 2;
  constexpr int UNIT = BM * 256, GPR = BN / 8;
  static_assert(2 * UNIT >= 32 * BN * 2, "an epilogue phase fits");
  __shared__ u32x4 lds[KS * 2 * UNIT / 16];
  const RowTile t = RowTiles<BM, 4>(a, (a.N + BN - 1) / BN).at(a, blockIdx.x);
  if (t.mrows <= 0) return;
  // part kg of the reduction takes every KS-th step
  const int kg = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int tid = threadIdx.x & 255, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31, K = a.K, n0 = t.tn * BN;
  const int nsteps = (K + KD * KS - 1) / (KD * KS);

  // activations: 16 lanes a row, thread's rows tid / 16 + 16 p
  const int xc = tid & 15, xr = tid >> 4;
  const uint8_t* xp[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p)
    xp[p] = a.A + (source_row(a, a.ma, t.row0 + min(xr + 16 * p, t.mrows - 1)) * a.lda + 8 * xc) * 2;
  // codes and parameters by 32-bit offsets from the tile's first column
  const uint8_t* const wt = a.B + (int64_t)t.e * a.b_expert + (int64_t)n0 * (K / 2);
  const uint8_t* const pt = a.b_scale + ((int64_t)t.e * a.N + n0) * (K / GROUP) * 4;
  const uint32_t col = (uint32_t)min(32 * w + l32, a.N - 1 - n0);

  u32x4 xv[D][NP], cw[D][2];
  uint32_t pw[D][2];
  auto load = [&](int step, int d) {
    const int k0 = (step * KS + kg) * KD;
    const bool on = k0 + 8 * xc < K;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      xv[d][p] = *reinterpret_cast<const u32x4*>(xp[p] + (on ? 2 * k0 : -16 * xc));
      if (!on) xv[d][p] = zero4();
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // (past the end: the column's first block, times zeros)
      const int k = k0 + 64 * u + 32 * half, kk = k < K ? k : 0;
      cw[d][u] = *reinterpret_cast<const u32x4*>(wt + (col * (uint32_t)(K / 2) + (uint32_t)kk / 2));
      if (GROUP < 128 || u == 0)
        pw[d][u] = *reinterpret_cast<const uint32_t*>(pt + (col * (uint32_t)(K / GROUP) + (uint32_t)kk / GROUP) * 4);
      else
        pw[d][u] = pw[d][0];
    }
  };
  char* const base = reinterpret_cast<char*>(lds) + kg * 2 * UNIT;
  auto put = [&](int buf, int d, int p0, int p1) {
#pragma unroll
    for (int p = p0; p < p1; ++p) {
      const int r = xr + 16 * p;
      *reinterpret_cast<u32x4*>(base + buf * UNIT + r * 256 + 16 * (xc ^ (r & 15))) = xv[d][p];
    }
  };

  f32x16 acc[FI];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int x = 0; x < 16; ++x) acc[i][x] = 0.f;

  // register set d holds a step's weights until they are bf16, and its activations until they are
  // in LDS; it then takes those of D steps later (past the end: the last step's again, unused)
#pragma unroll
  for (int d = 0; d < D; ++d) load(min(d, nsteps - 1), d);
  put(0, 0, 0, NP);
  lds_barrier();
  u32x4 x[2][FI], wv[2];
  auto read = [&](int buf, int n) {
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int r = 32 * i + l32;
      x[n & 1][i] = *reinterpret_cast<const u32x4*>(base + buf * UNIT + r * 256 +
                                                    16 * ((8 * (n >> 2) + 4 * half + (n & 3)) ^ (r & 15)));
    }
  };
  u32x4 cc[2];
  float s[2], o[2];
  auto take = [&](int d) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      cc[u] = cw[d][u];
      const float sc = __uint_as_float(pw[d][u] & 0xffff0000u);
      s[u] = sc * 16777216.f;
      o[u] = -sc * __uint_as_float(pw[d][u] << 16);
    }
  };
  auto decode = [&](int n) { wv[n & 1] = bf16_of_word(cc[n >> 2][n & 3], s[n >> 2], o[n >> 2]); };
  read(0, 0);
  take(0);
  decode(0);
  for (int step0 = 0; step0 < nsteps; step0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int step = step0 + d;
      if (step >= nsteps) break;
      // (set d: its weights are in cc, its activations in LDS)
      load(min(step + D, nsteps - 1), d);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n < 7) {
          read(step & 1, n + 1);
          decode(n + 1);
        } else {
          // the next step's first slice: its activations have been in LDS since the barrier
          read((step + 1) & 1, 0);
          take((d + 1) % D);
          decode(0);
        }
        if (n < 6) put((step + 1) & 1, (d + 1) % D, n * NP / 6, (n + 1) * NP / 6);
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[i] = mfma32(wv[n & 1], x[n & 1][i], acc[i]);
        // a matrix instruction, a read of the next slice, a share of its decoding
#pragma unroll
        for (int i = 0; i < FI; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x2, 20 / FI, 0);
        }
        if (n == 6) lds_barrier();     // the next step is in LDS, and nobody reads this one any more
      }
    }
  }
  __syncthreads();

  // the parts' sums, added in order: part kg hands its sums over in its own buffers, a fragment row at
  // a time, and the first part adds them
  if constexpr (KS > 1) {
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      if (kg > 0)
#pragma unroll
        for (int gg = 0; gg < 4; ++gg)
          *reinterpret_cast<f32x4*>(base + (gg * 256 + tid) * 16) =
              f32x4{acc[i][4 * gg], acc[i][4 * gg + 1], acc[i][4 * gg + 2], acc[i][4 * gg + 3]};
      __syncthreads();
      if (kg == 0)
#pragma unroll
        for (int p = 1; p < KS; ++p)
#pragma unroll
          for (int gg = 0; gg < 4; ++gg) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(base + p * 2 * UNIT + (gg * 256 + tid) * 16);
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[i][4 * gg + x] += v[x];
          }
      __syncthreads();
    }
    if (kg > 0) return;
  }
  // acc[i][4 gg + x]: row 32 i + l32, column 32 w + 8 gg + 4 half + x.  32 rows at a time through
  // LDS, granule c of row r at c ^ (r % GPR), so that whole rows are stored.
  const int n = n0 + 8 * (tid % GPR);
#pragma unroll
  for (int i = 0; i < FI; ++i) {
    if (32 * i >= t.mrows) break;
#pragma unroll
    for (int gg = 0; gg < 4; ++gg) {
      const u32x2 pk = {pack_bf16x2(acc[i][4 * gg], acc[i][4 * gg + 1]),
                        pack_bf16x2(acc[i][4 * gg + 2], acc[i][4 * gg + 3])};
      *reinterpret_cast<u32x2*>(base + l32 * (2 * BN) + 16 * ((4 * w + gg) ^ (l32 % GPR)) + 8 * half) = pk;
    }
    lds_barrier();
#pragma unroll
    for (int it = 0; it < 32 * GPR / 256; ++it) {
      const int r = it * (256 / GPR) + tid / GPR, m = 32 * i + r;
      if (m < t.mrows && n < a.N) {
        const int sr = t.row0 + m, v = a.mc.by_order ? a.order[sr] : sr;
        if ((unsigned)v < (unsigned)a.rows)
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.C) + (int64_t)v * a.ldc + n) =
              *reinterpret_cast<const u32x4*>(base + r * (2 * BN) + 16 * ((tid % GPR) ^ (r % GPR)));
      }
    }
    lds_barrier();
  }
}

namespace {

template <int FI, int KS>
void tile_of(const ExpertArgs& a, int32_t group, hipStream_t s) {
  const unsigned grid = (unsigned)affine_grid(a, 32 * FI, 128);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256 * KS), 0, s, a); };
  if (group == 32) go(k_affine_tile<32, FI, KS>);
  else if (group == 64) go(k_affine_tile<64, FI, KS>);
  else go(k_affine_tile<128, FI, KS>);
}

}  // namespace

void launch_affine_tile(const ExpertArgs& a, int32_t group, int rows, int parts, hipStream_t s) {
  if (rows == 64) return parts == 1 ? tile_of<2, 1>(a, group, s) : tile_of<2, 2>(a, group, s);
  if (parts == 1) return tile_of<4, 1>(a, group, s);
  tile_of<4, 2>(a, group, s);
}

}  // namespace mlora
