// 4-bit weights with a scale and a zero point per group, over many rows: a
// tile of 32 FI rows and 128 columns a workgroup, four waves side by side (KS
// times four, which take the reduction's steps in turn).
//
// A wave's weights go from memory straight into its registers, 4 bits each:
// nobody else needs them.  They become bf16 there, s c - s z by one fused
// multiply-add in fp32 and one rounding, while the matrix instructions of the
// step before run, so no decoded copy exists.  (Rounded, since the matrix cores take
// bf16: the codes as they are would need every sum scaled per group, 16 multiply-adds
// a lane for each 32 x 32 fragment and group, and sums of the activations.  Against
// 64 bits a normal case's outputs are off by 0.0022 of their size, where rounding the
// outputs alone costs 0.0017.)  The activations, which all four
// waves need, go through LDS, 128 inputs a step in two buffers: a step's loads
// are in flight while the step before is multiplied.
// Lane l = c + 32 h of a wave holds column c: 16 bytes are 32 neighbouring
// inputs, the step's blocks 2 u + h for u = 0, 1; word q of them and chunk
// 8 u + 4 h + q of the activations make one matrix instruction's 16 inputs.
// A block of 32 lies in one group, so its scale is the lane's own.
//
// What bounds it, from copies of the kernel that leave a part out: at 128 rows the
// stores of the activations to LDS (47 -> 39 us without them; without decoding no
// gain), at 64 rows decoding (55 -> 42 us without), which takes 2.5 vector
// instructions a weight whatever the rows.  Over a full chip (1024 tiles of 128 rows)
// matrix instructions are busy 45% of the cycles and vector ones 44%.  0.9 PF in
// tiles of 128 rows and 0.76 PF in tiles of 64.  Tiles of 128 x 256, with half the
// LDS reads a product, and of 96 x 128 were no faster where they fit (2048 rows over
// 8 experts 74 and 95 us, 4096 over 32 64 and 63).
// 4096 rows over 32 experts, 4096 -> 1024 66 us (640 tiles of 64 rows, a fifth
// of them padding); 2048 rows over 8 experts, 4096 -> 4096 76 to 84 us (0.8 to 0.9
// PF); 128 rows, 4096 -> 14336 26 us, 200 rows 39.
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

// The sums of a reduction's KS parts to part 0, in order: a part hands its own over in its LDS (`stride`
// bytes a part, 16 KiB used), a fragment row at a time.
template <int FI, int KS>
__device__ __forceinline__ void add_parts(f32x16 (&acc)[FI], char* lds, int stride, int kg, int tid) {
#pragma unroll
  for (int i = 0; i < FI; ++i) {
    if (kg > 0)
#pragma unroll
      for (int gg = 0; gg < 4; ++gg)
        *reinterpret_cast<f32x4*>(lds + kg * stride + (gg * 256 + tid) * 16) =
            f32x4{acc[i][4 * gg], acc[i][4 * gg + 1], acc[i][4 * gg + 2], acc[i][4 * gg + 3]};
    __syncthreads();
    if (kg == 0)
#pragma unroll
      for (int p = 1; p < KS; ++p)
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(lds + p * stride + (gg * 256 + tid) * 16);
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[i][4 * gg + x] += v[x];
        }
    __syncthreads();
  }
}

// acc[i][4 gg + x]: row 32 i + l32, column 32 w + 8 gg + 4 half + x of a tile 128 wide, thread tid of
// 256.  32 rows at a time through the 8 KiB at `base`, granule c of row r at c ^ (r % GPR), so that
// whole rows are stored.
template <int FI>
__device__ __forceinline__ void store_tile(const ExpertArgs& a, const RowTile& t, const f32x16 (&acc)[FI], char* base,
                                           int tid) {
  constexpr int BN = 128, GPR = BN / 8;
  const int lane = tid & 63, w = tid >> 6, half = lane >> 5, l32 = lane & 31;
  const int n = t.tn * BN + 8 * (tid % GPR);
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

}  // namespace

template <int GROUP, int FI, int KS>
__global__ __launch_bounds__(256 * KS, 2) void k_affine_tile(ExpertArgs a) {
  constexpr int BM = 32 * FI, BN = 128, KD = 128, NP = BM / 16, D = 2;
  constexpr int UNIT = BM * 256;
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
    // Past the reduction's end a lane reads the row's start, and its weights are zero.  (By address: a
    // load in a branch would make the compiler wait for every load in flight.)
    const int at = k0 + 8 * xc < K ? 2 * k0 : -16 * xc;
#pragma unroll
    for (int p = 0; p < NP; ++p) xv[d][p] = *reinterpret_cast<const u32x4*>(xp[p] + at);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // (past the end: the column's first block, taken times zero)
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
  auto take = [&](int step, int d) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      cc[u] = cw[d][u];
      const uint32_t p = (step * KS + kg) * KD + 64 * u + 32 * half < K ? pw[d][u] : 0u;
      const float sc = __uint_as_float(p & 0xffff0000u);
      s[u] = sc * 16777216.f;
      o[u] = -sc * __uint_as_float(p << 16);
    }
  };
  auto decode = [&](int n) { wv[n & 1] = bf16_of_word(cc[n >> 2][n & 3], s[n >> 2], o[n >> 2]); };
  read(0, 0);
  take(0, 0);
  decode(0);
  for (int step0 = 0; step0 < nsteps; step0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int step = step0 + d;
      if (step >= nsteps) break;
      // (set d: its weights are in cc, its activations in LDS)
      load(min(step + D, nsteps - 1), d);
      __builtin_amdgcn_sched_barrier(0);          // in flight from here on, not from where it is convenient
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n < 7) {
          read(step & 1, n + 1);
          decode(n + 1);
        } else {
          // the next step's first slice: its activations have been in LDS since the barrier
          read((step + 1) & 1, 0);
          take(step + 1, (d + 1) % D);
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

  if constexpr (KS > 1) {
    add_parts<FI, KS>(acc, reinterpret_cast<char*>(lds), 2 * UNIT, kg, tid);
    if (kg > 0) return;
  }
  store_tile<FI>(a, t, acc, base, tid);
}

// dX = dY W_e: the reduction runs over the weight's rows, so a lane of the
// matrix instruction needs eight rows' codes of one column.  The workgroup
// decodes a step's 64 rows x 128 columns once, a thread 32 neighbouring codes of
// a row (one group: one scale), to bf16 rows in LDS, and the transposing reads
// of LDS give the lanes their columns.
//   weights: wave p's 32 columns are a region of its own, [64][32] bf16, chunk j
//   (16 bytes) of row k at j ^ (k >> 2) ^ p mod 4, which spreads eight lanes'
//   writes and 16 lanes' reads over all banks;
//   activations: [BM][64], chunk c of row r at c ^ (r & 7).
// Both in two buffers: while step s is multiplied, step s + 1's are written and
// step s + 2's loads are in flight.  One slice of a step: 16 rows of the
// weight; lane c + 32 h takes rows 8 h .. 8 h + 7 of column c.
// 1501 rows over 4 experts of 4096 x 4096, groups of 32 79 us (101 with the weights
// decoded to memory first), 512 rows over 8 36 us (133).  Bound as the kernel above: matrix
// instructions are busy 29%, vector ones 28%, the rest waits for LDS and for the
// tile that is twice on one CU.
template <int GROUP, int FI, int KS>
__global__ __launch_bounds__(256 * KS, 2) void k_affine_dx(ExpertArgs a) {
  constexpr int BM = 32 * FI, BN = 128, KD = 64, NP = BM / 32, D = 2;
  constexpr int UA = BM * 128, UW = KD * BN * 2, PART = 2 * (UA + UW);
  __shared__ u32x4 lds[KS * PART / 16];
  const RowTile t = RowTiles<BM, 4>(a, (a.N + BN - 1) / BN).at(a, blockIdx.x);
  if (t.mrows <= 0) return;
  // part kg of the reduction takes every KS-th step
  const int kg = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int tid = threadIdx.x & 255, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31, K = a.K, N = a.N, n0 = t.tn * BN;
  const int nsteps = (K + KD * KS - 1) / (KD * KS);

  // activations: 8 lanes a row, thread's rows tid / 8 + 32 p
  const int xc = tid & 7, xr = tid >> 3;
  const uint8_t* xp[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p)
    xp[p] = a.A + (source_row(a, a.ma, t.row0 + min(xr + 32 * p, t.mrows - 1)) * a.lda + 8 * xc) * 2;
  // weights: thread's row tid / 4 of the step, columns 32 (tid % 4) .. of the tile (past N: the last ones)
  const int wr = tid >> 2, wc = tid & 3, nb = min(n0 + 32 * wc, N - 32);
  const uint8_t* const wt = a.B + (int64_t)t.e * a.b_expert + nb / 2;
  const uint8_t* const pt = a.b_scale + ((int64_t)t.e * K * (N / GROUP) + nb / GROUP) * 4;

  u32x4 xv[D][NP], cw[D];
  uint32_t pw[D];
  auto load = [&](int step, int d) {
    const int k0 = (step * KS + kg) * KD;
    const int at = k0 + 8 * xc < K ? 2 * k0 : -16 * xc;        // K is a multiple of 8
#pragma unroll
    for (int p = 0; p < NP; ++p) xv[d][p] = *reinterpret_cast<const u32x4*>(xp[p] + at);
    // (past the end: the first row, taken times zero)
    const int64_t k = k0 + wr < K ? k0 + wr : 0;
    cw[d] = *reinterpret_cast<const u32x4*>(wt + k * (N / 2));
    pw[d] = *reinterpret_cast<const uint32_t*>(pt + k * (N / GROUP) * 4);
  };
  char* const base = reinterpret_cast<char*>(lds) + kg * PART;
  auto put_x = [&](int buf, int d, int p0, int p1) {
#pragma unroll
    for (int p = p0; p < p1; ++p)
      *reinterpret_cast<u32x4*>(base + buf * UA + (xr + 32 * p) * 128 + 16 * (xc ^ (xr & 7))) = xv[d][p];
  };
  char* const wbase = base + 2 * UA;
  auto put_w = [&](int step, int d, int j0, int j1) {
    const uint32_t pk = (step * KS + kg) * KD + wr < K ? pw[d] : 0u;
    const float sc = __uint_as_float(pk & 0xffff0000u);
    const float s = sc * 16777216.f, o = -sc * __uint_as_float(pk << 16);
    const int buf = step & 1;
#pragma unroll
    for (int j = j0; j < j1; ++j)
      *reinterpret_cast<u32x4*>(wbase + buf * UW + wc * (KD * 64) + wr * 64 + 16 * ((j ^ (wr >> 2) ^ wc) & 3)) =
          bf16_of_word(cw[d][j], s, o);
  };
  // the transposing reads' lane parts: rows 8 half + sq / 4 and four further on, columns 4 (sq % 4) ..
  const int gq = lane >> 4, sq = lane & 15, nc = 16 * (gq & 1) + 4 * (sq & 3), kr = 8 * half + (sq >> 2);
  auto lane_w = [&](int k) { return (uint32_t)(w * (KD * 64) + k * 64 + 16 * (((nc >> 3) ^ (k >> 2) ^ w) & 3) + 2 * (nc & 7)); };
  const uint32_t w0 = lane_w(kr), w1 = lane_w(kr + 4);
  const MLORA_LDS char* const wl = (const MLORA_LDS char*)(MLORA_LDS void*)wbase;

  f32x16 acc[FI];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int x = 0; x < 16; ++x) acc[i][x] = 0.f;
  u32x4 x[2][FI], wv[2];
  auto read = [&](int buf, int n) {
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int r = 32 * i + l32;
      x[n & 1][i] = *reinterpret_cast<const u32x4*>(base + buf * UA + r * 128 + 16 * ((2 * n + half) ^ (r & 7)));
    }
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MLORA_LDS s16x4*)(wl + buf * UW + 1024 * n + w0));
    const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MLORA_LDS s16x4*)(wl + buf * UW + 1024 * n + w1));
    const u32x2 a0 = __builtin_bit_cast(u32x2, v0), a1 = __builtin_bit_cast(u32x2, v1);
    wv[n & 1] = u32x4{a0[0], a0[1], a1[0], a1[1]};
  };

  load(0, 0);
  load(min(1, nsteps - 1), 1);
  put_x(0, 0, 0, NP);
  put_w(0, 0, 0, 4);
  lds_barrier();
  read(0, 0);
  for (int step0 = 0; step0 < nsteps; step0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int step = step0 + d;
      if (step >= nsteps) break;
      // (set d is in LDS; past the end the last step's again, unused)
      load(min(step + D, nsteps - 1), d);
      __builtin_amdgcn_sched_barrier(0);          // in flight from here on, not from where it is convenient
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        if (n < 3) read(step & 1, n + 1);
        else read((step + 1) & 1, 0);             // in LDS since the barrier
        if (n < 2) {
          put_w(step + 1, (d + 1) % D, 2 * n, 2 * n + 2);
          put_x((step + 1) & 1, (d + 1) % D, n * NP / 2, (n + 1) * NP / 2);
        }
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[i] = mfma32(wv[n & 1], x[n & 1][i], acc[i]);
        if (n == 2) lds_barrier();                // the next step is in LDS, and nobody reads this one any more
      }
    }
  }
  __syncthreads();
  if constexpr (KS > 1) {
    add_parts<FI, KS>(acc, reinterpret_cast<char*>(lds), PART, kg, tid);
    if (kg > 0) return;
  }
  store_tile<FI>(a, t, acc, base, tid);
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

namespace {

template <int FI, int KS>
void dx_of(const ExpertArgs& a, int32_t group, hipStream_t s) {
  const unsigned grid = (unsigned)affine_grid(a, 32 * FI, 128);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256 * KS), 0, s, a); };
  if (group == 32) go(k_affine_dx<32, FI, KS>);
  else if (group == 64) go(k_affine_dx<64, FI, KS>);
  else go(k_affine_dx<128, FI, KS>);
}

}  // namespace

void launch_affine_dx(const ExpertArgs& a, int32_t group, int rows, hipStream_t s) {
  if (rows == 32) return dx_of<1, 2>(a, group, s);
  if (rows == 64) return dx_of<2, 1>(a, group, s);
  dx_of<4, 1>(a, group, s);
}

}  // namespace mlora
