// Grouped expert products for gfx950: one base weight per group of rows,
// Y = X W_e and dX = dY W_e^T over ragged row groups, dW_e = X^T dY over each
// group's rows, on matrix instructions with fp32 accumulation.
#include "expert_common.hpp"
#include "gemm_common.hpp"

namespace mlora {

// 16 zero bytes that copies past a reduction's end read.
__device__ __constant__ uint32_t g_expert_zero[64] = {0};

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// How an operand's elements lie in memory and in LDS.
//   KC: contiguous along the reduction; a unit is one row of 128 bytes per
//       tile row (64 bf16 or 32 fp32 of the reduction), chunk c (16 bytes) of
//       row r at c ^ kx8(r).
//   NC: contiguous along the output; a unit is one row of 256 output elements
//       per reduction step element.
//   F4: E2M1 codes along the reduction, 32 bytes (64 elements) per tile row,
//       chunk h of row r at h ^ ((r >> 3) & 1), and one dword of scale codes
//       per row that covers the step (it holds 128 elements' scales).
enum { KC = 0, NC = 1, F4 = 2 };

// Chunk swizzle of an n-contiguous bf16 row (see the base GEMM): XOR of 4, 8
// and 9 over bits 0, 1 and 3 of the k-row, which gives every transposing read
// group distinct banks.
__device__ __forceinline__ int nx16(int kr) { return ((kr & 1) ? 4 : 0) ^ ((kr & 2) ? 8 : 0) ^ ((kr & 8) ? 9 : 0); }
// fp32: the two half-waves of a fragment read take k-rows 4 apart; the XOR
// puts them on the two halves of the banks.
__device__ __forceinline__ int nx32(int kr) { return (kr & 4) ? 8 : 0; }

}  // namespace

// ---------------------------------------------------------------------------
// Tile kernel.  A workgroup of four waves (2 x 2) makes a 64 FI x 256 tile,
// each wave 32 FI x 128 in accumulators.  Steps of 64 bf16 (32 fp32) of the
// reduction are copied straight from global memory into LDS, double
// buffered: step t + 1 is in flight while step t is computed.
//   DW = false: C[rc(s)][n] over the rows of one group (rows form)
//   DW = true:  C_e[m][n] = sum over the group's rows (both operands NC)
// ---------------------------------------------------------------------------
template <bool F32, int AL, int BL, int FI, bool DW>
__global__ __launch_bounds__(256, 1) void k_expert_tile(ExpertArgs g) {
  constexpr int FJ = 4, BM = 64 * FI, BN = 256, ESZ = F32 ? 4 : 2, EPC = 16 / ESZ, KD = 128 / ESZ;
  constexpr int UA = BM * 128, UB = BL == F4 ? BN * 32 + BN * 4 : BN * 128;  // bytes of a step's units
  constexpr int CA = UA / 4096, CB = BL == F4 ? 2 : UB / 4096;              // 1 KiB copies per wave
  constexpr int EPI = F32 || DW ? 0 : BM * 512;                             // the epilogue's bf16 tile
  __shared__ u32x4 ring[(2 * (UA + UB) > EPI ? 2 * (UA + UB) : EPI) / 16];

  const int nN = (g.N + BN - 1) / BN;
  int e, row0, mrows, n0, klen, m0 = 0;
  if constexpr (DW) {
    const int nM = (g.M + BM - 1) / BM, TT = nM * nN;
    const int b = blockIdx.x, G = gridDim.x, xcd = b & 7, q = b >> 3, per = G >> 3, rem = G & 7;
    const int L = xcd * per + min(xcd, rem) + q;
    e = L / TT;
    const int t = L - e * TT;
    constexpr int GM = 4;
    const int grp = t / (GM * nN), fm = grp * GM, gm = min(GM, nM - fm), within = t - fm * nN;
    m0 = (fm + within % gm) * BM;
    n0 = within / gm * BN;
    int hi;
    group_rows(g, e, row0, hi);
    klen = hi - row0;
    mrows = min(BM, g.M - m0);
  } else {
    const RowTile t = row_tile<BM, 4>(g, nN);
    if (t.mrows <= 0) return;
    e = t.e;
    row0 = t.row0;
    mrows = t.mrows;
    n0 = t.tn * BN;
    klen = g.K;
  }
  const int nsteps = (klen + KD - 1) / KD;

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wrow = 32 * FI * (w >> 1), wcol = 128 * (w & 1);

  const uint8_t* const Be = DW ? g.B : g.B + (int64_t)e * g.b_expert;
  const uint8_t* const zero = reinterpret_cast<const uint8_t*>(g_expert_zero);

  // Row pointers of the k-contiguous operands' copies: copy i of a wave takes
  // tile rows 8 (CA w + i) + lane / 8, LDS position lane % 8.
  const uint8_t* ap[CA];
  int ac[CA];
  if constexpr (AL == KC) {
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int r = 8 * (CA * w + i) + (lane >> 3);
      ac[i] = (lane & 7) ^ kx8(r);
      ap[i] = g.A + (source_row(g, g.ma, row0 + min(r, mrows - 1)) * g.lda) * ESZ + 16 * ac[i];
    }
  }
  const uint8_t* bp[CB];
  int bc[CB];
  if constexpr (BL == KC) {
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int r = 8 * (CB * w + i) + (lane >> 3);
      bc[i] = (lane & 7) ^ kx8(r);
      bp[i] = Be + ((int64_t)min(n0 + r, g.N - 1) * g.ldb) * ESZ + 16 * bc[i];
    }
  }
  const uint8_t* sp = nullptr;
  if constexpr (BL == F4) {
    // copy i: tile rows 32 (2 w + i) + lane / 2, position lane % 2
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int r = 32 * (2 * w + i) + (lane >> 1);
      bc[i] = (lane & 1) ^ ((r >> 3) & 1);
      bp[i] = Be + (int64_t)min(n0 + r, g.N - 1) * (g.ldb / 2) + 16 * bc[i];
    }
    sp = g.b_scale + ((int64_t)e * g.N + min(n0 + 64 * w + lane, g.N - 1)) * (g.ldb / 32);
  }

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(MLORA_LDS void*)&ring[0]);

  // Copies of an n-contiguous unit of RW columns from column c0 of `base`.
  auto copy_nc = [&](auto rw_tag, const uint8_t* base, int64_t ld, int c0, int cmax, const RowMap& map, bool rows_map,
                     int t, uint32_t lds) {
    constexpr int RW = decltype(rw_tag)::value, CPR = RW * ESZ / 16, RPC = 64 / CPR, NCP = RW / 32;
#pragma unroll
    for (int i = 0; i < NCP; ++i) {
      const int kr = RPC * (NCP * w + i) + lane / CPR;
      const int c = (lane % CPR) ^ (F32 ? nx32(kr) : nx16(kr));
      const int k = t * KD + kr;
      const int col = min(c0 + EPC * c, cmax - EPC);
      const uint8_t* src = zero;
      if (k < klen) {
        const int64_t row = rows_map ? source_row(g, map, row0 + k) : (int64_t)k;
        src = base + (row * ld + col) * ESZ;
      }
      dma16_at(src, lds + 1024u * (uint32_t)(NCP * w + i));
    }
  };
  auto issue = [&](int t) {
    const uint32_t ua = lds0 + (uint32_t)(t & 1) * (UA + UB), ub = ua + UA;
    if constexpr (AL == KC) {
#pragma unroll
      for (int i = 0; i < CA; ++i)
        dma16_at(t * KD + EPC * ac[i] < klen ? ap[i] + 128 * (int64_t)t : zero, ua + 1024u * (uint32_t)(CA * w + i));
    } else {
      copy_nc(std::integral_constant<int, BM>(), g.A, g.lda, m0, g.M, g.ma, true, t, ua);
    }
    if constexpr (BL == KC) {
#pragma unroll
      for (int i = 0; i < CB; ++i)
        dma16_at(t * KD + EPC * bc[i] < klen ? bp[i] + 128 * (int64_t)t : zero, ub + 1024u * (uint32_t)(CB * w + i));
    } else if constexpr (BL == NC) {
      copy_nc(std::integral_constant<int, BN>(), Be, g.ldb, n0, g.N, g.mb, DW, t, ub);
    } else {
#pragma unroll
      for (int i = 0; i < CB; ++i) dma16_at(bp[i] + 32 * (int64_t)t, ub + 1024u * (uint32_t)(CB * w + i));
      dma4_at(sp + 4 * (t >> 1), ub + BN * 32 + 256u * (uint32_t)w);
    }
  };

  f32x16 acc[FI][FJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < FJ; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) acc[a][b][x] = 0.f;

  const MLORA_LDS char* const base = (const MLORA_LDS char*)(MLORA_LDS void*)&ring[0];
  // Fragment of slice ks: eight bf16 (four fp32) of the reduction per lane.
  // F4 weights: half h of the wave takes the step's block h, so slice ks of
  // the k-contiguous operand is chunk 4 h + ks instead of 2 ks + h.
  auto frag_kc = [&](uint32_t unit, int r, int ks) {
    const int c = BL == F4 ? 4 * half + ks : 2 * ks + half;
    return *(const MLORA_LDS u32x4*)(base + unit + (r * 8 + (c ^ kx8(r))) * 16);
  };
  auto frag_nc = [&](auto rw_tag, uint32_t unit, int n, int ks) {
    constexpr int RW = decltype(rw_tag)::value, CPR = RW * ESZ / 16;
    u32x4 out;
    if constexpr (F32) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int kr = 8 * ks + 4 * half + x, col = n + l32;
        out[x] = *(const MLORA_LDS uint32_t*)(base + unit + (kr * CPR + ((col >> 2) ^ nx32(kr))) * 16 + 4 * (col & 3));
      }
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      const int gq = lane >> 4, s = lane & 15;
      const int col = n + 16 * (gq & 1) + 4 * (s & 3);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kr = 16 * ks + 8 * (gq >> 1) + (s >> 2) + 4 * h;
        const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (MLORA_LDS s16x4*)(base + unit + (kr * CPR + ((col >> 3) ^ nx16(kr))) * 16 + 2 * (col & 7)));
        const u32x2 u = __builtin_bit_cast(u32x2, v);
        out[2 * h] = u[0];
        out[2 * h + 1] = u[1];
      }
    }
    return out;
  };
  auto mma = [&](f32x16& c, const u32x4& a, const u32x4& b) {
    if constexpr (F32) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[x]), __uint_as_float(b[x]), c, 0, 0, 0);
    } else {
      c = mfma32(a, b, c);
    }
  };

  if (nsteps > 0) issue(0);
  for (int t = 0; t < nsteps; ++t) {
    // step t has landed, and every wave is done with the other buffer
    wait_vm_barrier<0>();
    if (t + 1 < nsteps) issue(t + 1);
    const uint32_t ua = (uint32_t)(t & 1) * (UA + UB), ub = ua + UA;
    u32x4 codes[FJ];
    float scale[FJ];
    if constexpr (BL == F4) {
#pragma unroll
      for (int f = 0; f < FJ; ++f) {
        const int r = wcol + 32 * f + l32;
        codes[f] = *(const MLORA_LDS u32x4*)(base + ub + (r * 2 + (half ^ ((r >> 3) & 1))) * 16);
        const uint32_t sw = *(const MLORA_LDS uint32_t*)(base + ub + BN * 32 + 4 * r);
        scale[f] = __uint_as_float(((sw >> (16 * (t & 1) + 8 * half)) & 255u) << 23);
      }
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      u32x4 fa[FI], fb[FJ];
#pragma unroll
      for (int f = 0; f < FI; ++f) {
        if constexpr (AL == KC) fa[f] = frag_kc(ua, wrow + 32 * f + l32, ks);
        else fa[f] = frag_nc(std::integral_constant<int, BM>(), ua, wrow + 32 * f, ks);
      }
#pragma unroll
      for (int f = 0; f < FJ; ++f) {
        if constexpr (BL == KC) fb[f] = frag_kc(ub, wcol + 32 * f + l32, ks);
        else if constexpr (BL == NC) fb[f] = frag_nc(std::integral_constant<int, BN>(), ub, wcol + 32 * f, ks);
        else fb[f] = bf16_of_e2m1(codes[f][ks], scale[f]);
      }
#pragma unroll
      for (int fi = 0; fi < FI; ++fi)
#pragma unroll
        for (int fj = 0; fj < FJ; ++fj) mma(acc[fi][fj], fb[fj], fa[fi]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // this wave's reads are done before the next barrier lets others overwrite
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // acc[fi][fj][4 gg + x] holds C[m = wrow + 32 fi + l32][n = wcol + 32 fj + 8 gg + 4 half + x]
  if constexpr (F32 || DW) {
#pragma unroll
    for (int fi = 0; fi < FI; ++fi) {
      const int m = wrow + 32 * fi + l32;
      if (m >= mrows) continue;
      int64_t row;
      if (DW) {
        row = m0 + m;
      } else {
        const int s = row0 + m, v = g.mc.by_order ? g.order[s] : s;
        if ((unsigned)v >= (unsigned)g.rows) continue;
        row = v;
      }
      float* crow = static_cast<float*>(g.C) + (DW ? (int64_t)e * g.c_expert : 0) + row * g.ldc;
#pragma unroll
      for (int fj = 0; fj < FJ; ++fj)
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
          const int n = n0 + wcol + 32 * fj + 8 * gg + 4 * half;
          if (n >= g.N) continue;
          f32x4 v = {acc[fi][fj][4 * gg], acc[fi][fj][4 * gg + 1], acc[fi][fj][4 * gg + 2], acc[fi][fj][4 * gg + 3]};
          f32x4* dst = reinterpret_cast<f32x4*>(crow + n);
          if (DW && g.accumulate) {
            const f32x4 old = *dst;
            v += old;
          }
          *dst = v;
        }
    }
  } else {
    __syncthreads();
    char* ct = reinterpret_cast<char*>(&ring[0]);
#pragma unroll
    for (int fi = 0; fi < FI; ++fi) {
      const int m = wrow + 32 * fi + l32;
#pragma unroll
      for (int fj = 0; fj < FJ; ++fj)
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
          const int c = (wcol >> 3) + 4 * fj + gg;
          u32x2 pk;
          pk[0] = pack_bf16x2(acc[fi][fj][4 * gg + 0], acc[fi][fj][4 * gg + 1]);
          pk[1] = pack_bf16x2(acc[fi][fj][4 * gg + 2], acc[fi][fj][4 * gg + 3]);
          *reinterpret_cast<u32x2*>(ct + m * 512 + 16 * (c ^ (m & 31)) + 8 * half) = pk;
        }
    }
    __syncthreads();
    const int gc = lane & 31;
    for (int it = 0; it < BM / 8; ++it) {
      const int m = (BM / 4) * w + 2 * it + half;
      const int n = n0 + 8 * gc;
      if (m >= mrows || n >= g.N) continue;
      const int s = row0 + m, v = g.mc.by_order ? g.order[s] : s;
      if ((unsigned)v >= (unsigned)g.rows) continue;
      const u32x4 x = *reinterpret_cast<const u32x4*>(ct + m * 512 + 16 * (gc ^ (m & 31)));
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.C) + (int64_t)v * g.ldc + n) = x;
    }
  }
}

// ---------------------------------------------------------------------------
// MXFP4 x MXFP4: both operands as E2M1 codes on the scaled matrix cores.
// 256 x 256 tile, steps of 128 of the reduction: 64 bytes of codes and one
// dword of scale codes per row and operand.  Chunk c of row r sits at
// c ^ ((r >> 2) & 3), which spreads a read group's rows over the banks; lane
// r + 32 h holds row r's 32-block h of a 64-deep slice (16 bytes, the low
// nibble first) and supplies its scale.
// ---------------------------------------------------------------------------
template <int FI>
__global__ __launch_bounds__(256, 1) void k_expert_mx4(ExpertArgs g) {
  constexpr int FJ = 4, BM = 64 * FI, BN = 256;
  constexpr int UA = BM * 64, UB = BN * 64, CA = FI, CB = 4;
  constexpr int STAGE = UA + UB + (BM + BN) * 4;
  __shared__ u32x4 ring[(2 * STAGE > BM * 512 ? 2 * STAGE : BM * 512) / 16];
  const int nN = (g.N + BN - 1) / BN;
  const RowTile tile = row_tile<BM, 4>(g, nN);
  if (tile.mrows <= 0) return;
  const int e = tile.e, row0 = tile.row0, mrows = tile.mrows, n0 = tile.tn * BN;
  const int nsteps = g.K / 128;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wrow = 32 * FI * (w >> 1), wcol = 128 * (w & 1);
  const int64_t kb = g.K / 32;

  const uint8_t* ap[CA];
  const uint8_t* bp[CB];
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    const int r = 16 * (CA * w + i) + (lane >> 2);
    ap[i] = g.A + source_row(g, g.ma, row0 + min(r, mrows - 1)) * (g.K / 2) + 16 * ((lane & 3) ^ ((r >> 2) & 3));
  }
#pragma unroll
  for (int i = 0; i < CB; ++i) {
    const int r = 16 * (CB * w + i) + (lane >> 2);
    bp[i] = g.B + (int64_t)e * g.b_expert + (int64_t)min(n0 + r, g.N - 1) * (g.K / 2) +
            16 * ((lane & 3) ^ ((r >> 2) & 3));
  }
  // scale dwords: wave w copies rows 64 w .. of A (waves below FI) and of B
  const uint8_t* as = g.a_scale + source_row(g, g.ma, row0 + min(64 * min(w, FI - 1) + lane, mrows - 1)) * kb;
  const uint8_t* bs = g.b_scale + ((int64_t)e * g.N + min(n0 + 64 * w + lane, g.N - 1)) * kb;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(MLORA_LDS void*)&ring[0]);
  auto issue = [&](int t) {
    const uint32_t u = lds0 + (uint32_t)(t & 1) * STAGE;
#pragma unroll
    for (int i = 0; i < CA; ++i) dma16_at(ap[i] + 64 * (int64_t)t, u + 1024u * (uint32_t)(CA * w + i));
#pragma unroll
    for (int i = 0; i < CB; ++i) dma16_at(bp[i] + 64 * (int64_t)t, u + UA + 1024u * (uint32_t)(CB * w + i));
    if (w < FI) dma4_at(as + 4 * t, u + UA + UB + 256u * (uint32_t)w);
    dma4_at(bs + 4 * t, u + UA + UB + BM * 4 + 256u * (uint32_t)w);
  };

  f32x16 acc[FI][FJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < FJ; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) acc[a][b][x] = 0.f;
  const MLORA_LDS char* const base = (const MLORA_LDS char*)(MLORA_LDS void*)&ring[0];
  auto frag = [&](uint32_t unit, int r, int sl) -> i32x8 {
    const u32x4 p = *(const MLORA_LDS u32x4*)(base + unit + (r * 4 + ((2 * sl + half) ^ ((r >> 2) & 3))) * 16);
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(p, zero4(), 0, 1, 2, 3, 4, 5, 6, 7));
  };

  issue(0);
  for (int t = 0; t < nsteps; ++t) {
    wait_vm_barrier<0>();
    if (t + 1 < nsteps) issue(t + 1);
    const uint32_t u = (uint32_t)(t & 1) * STAGE;
    int sa[FI], sb[FJ];
#pragma unroll
    for (int f = 0; f < FI; ++f)
      sa[f] = (int)(*(const MLORA_LDS uint32_t*)(base + u + UA + UB + 4 * (wrow + 32 * f + l32)) >> (8 * half));
#pragma unroll
    for (int f = 0; f < FJ; ++f)
      sb[f] = (int)(*(const MLORA_LDS uint32_t*)(base + u + UA + UB + BM * 4 + 4 * (wcol + 32 * f + l32)) >> (8 * half));
#pragma unroll
    for (int sl = 0; sl < 2; ++sl) {
      i32x8 fa[FI], fb[FJ];
#pragma unroll
      for (int f = 0; f < FI; ++f) fa[f] = frag(u, wrow + 32 * f + l32, sl);
#pragma unroll
      for (int f = 0; f < FJ; ++f) fb[f] = frag(u + UA, wcol + 32 * f + l32, sl);
#pragma unroll
      for (int fi = 0; fi < FI; ++fi)
#pragma unroll
        for (int fj = 0; fj < FJ; ++fj) {
          if (sl == 0)
            acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[fj], fa[fi], acc[fi][fj], 4, 4, 0, sb[fj],
                                                                          0, sa[fi]);
          else
            acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[fj], fa[fi], acc[fi][fj], 4, 4, 2, sb[fj],
                                                                          2, sa[fi]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  __syncthreads();
  char* ct = reinterpret_cast<char*>(&ring[0]);
#pragma unroll
  for (int fi = 0; fi < FI; ++fi) {
    const int m = wrow + 32 * fi + l32;
#pragma unroll
    for (int fj = 0; fj < FJ; ++fj)
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) {
        const int c = (wcol >> 3) + 4 * fj + gg;
        u32x2 pk;
        pk[0] = pack_bf16x2(acc[fi][fj][4 * gg + 0], acc[fi][fj][4 * gg + 1]);
        pk[1] = pack_bf16x2(acc[fi][fj][4 * gg + 2], acc[fi][fj][4 * gg + 3]);
        *reinterpret_cast<u32x2*>(ct + m * 512 + 16 * (c ^ (m & 31)) + 8 * half) = pk;
      }
  }
  __syncthreads();
  const int gc = lane & 31;
  for (int it = 0; it < BM / 8; ++it) {
    const int m = (BM / 4) * w + 2 * it + half;
    const int n = n0 + 8 * gc;
    if (m >= mrows || n >= g.N) continue;
    const int s = row0 + m, v = g.mc.by_order ? g.order[s] : s;
    if ((unsigned)v >= (unsigned)g.rows) continue;
    const u32x4 x = *reinterpret_cast<const u32x4*>(ct + m * 512 + 16 * (gc ^ (m & 31)));
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.C) + (int64_t)v * g.ldc + n) = x;
  }
}

namespace {

template <bool F32, int AL, int BL, int FI>
void rows_tile(const ExpertArgs& a, hipStream_t s) {
  const int64_t nN = (a.N + 255) / 256;
  const int64_t grid = max_row_tiles(a.rows, a.offsets ? a.n_experts : 1, 64 * FI) * nN;
  hipLaunchKernelGGL((k_expert_tile<F32, AL, BL, FI, false>), dim3((unsigned)grid), dim3(256), 0, s, a);
}
template <bool F32, int BL>
void rows_size(const ExpertArgs& a, hipStream_t s) {
  const int64_t mean = a.rows / (a.offsets ? a.n_experts : 1);
  if (mean <= 96) rows_tile<F32, KC, BL, 1>(a, s);
  else if (mean <= 384) rows_tile<F32, KC, BL, 2>(a, s);
  else rows_tile<F32, KC, BL, 4>(a, s);
}
template <int FI>
void mx4_tile(const ExpertArgs& a, hipStream_t s) {
  const int64_t nN = (a.N + 255) / 256;
  const int64_t grid = max_row_tiles(a.rows, a.offsets ? a.n_experts : 1, 64 * FI) * nN;
  hipLaunchKernelGGL((k_expert_mx4<FI>), dim3((unsigned)grid), dim3(256), 0, s, a);
}

}  // namespace

void launch_expert_rows(ExpertForm form, bool b_kc, const ExpertArgs& a, hipStream_t s) {
  if (a.rows <= 0) return;
  const int64_t mean = a.rows / (a.offsets ? a.n_experts : 1);
  if (mean <= 32) return launch_expert_few(form, b_kc, mean <= 16 ? 1 : 2, a, s);
  switch (form) {
    case ExpertForm::kBf16:
      if (b_kc) rows_size<false, KC>(a, s);
      else rows_size<false, NC>(a, s);
      break;
    case ExpertForm::kF32:
      if (b_kc) rows_size<true, KC>(a, s);
      else rows_size<true, NC>(a, s);
      break;
    case ExpertForm::kW4A16:
      rows_size<false, F4>(a, s);
      break;
    case ExpertForm::kW4A4:
      if (mean <= 96) mx4_tile<1>(a, s);
      else if (mean <= 384) mx4_tile<2>(a, s);
      else mx4_tile<4>(a, s);
      break;
  }
}

void launch_expert_dw(bool f32, const ExpertArgs& a, hipStream_t s) {
  const int64_t E = a.offsets ? a.n_experts : 1;
  const int64_t nN = (a.N + 255) / 256;
  const int64_t grid = E * ((a.M + 255) / 256) * nN;
  if (f32) hipLaunchKernelGGL((k_expert_tile<true, NC, NC, 4, true>), dim3((unsigned)grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_expert_tile<false, NC, NC, 4, true>), dim3((unsigned)grid), dim3(256), 0, s, a);
}

}  // namespace mlora
