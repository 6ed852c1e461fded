// Grouped expert products for gfx950: one base weight per group of rows,
// Y = X W_e and dX = dY W_e^T over ragged row groups, dW_e = X^T dY over each
// group's rows, on matrix instructions with fp32 accumulation.
#include "expert_common.hpp"
#include "gemm_common.hpp"

#include <type_traits>

namespace mlora {

// 16 zero bytes that copies past a reduction's end read.
__device__ __constant__ uint32_t g_expert_zero[64] = {0};

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 bytes per lane into LDS from a wave-uniform base plus a 32-bit lane
// offset: the base lives in scalar registers.  M0 as in dma16_at.
__device__ __forceinline__ uint64_t uniform64(const void* p) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b) |
         ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) << 32);
}
__device__ __forceinline__ void dma16_sv(uint64_t sbase, uint32_t voff, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %2, %3\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds), "v"(voff), "s"(sbase)
      : "memory");
}

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

// A workgroup's tile: 64 FI rows (dW: rows of dW_e) x 256 columns of expert e.
struct Tile {
  int e, row0, mrows;   // grouped rows [row0, row0 + mrows); dW: row0 is the group's first row, mrows the tile's
  int m0, n0;           // first row of dW_e (else 0) and first column
  int klen;             // length of the reduction
};
template <int BM, bool DW>
__device__ __forceinline__ Tile find_tile(const ExpertArgs& g) {
  const int nN = (g.N + 255) / 256;
  Tile t;
  if constexpr (DW) {
    // Experts have reductions of different lengths: every expert's tiles are
    // spread over all XCDs, and up to 64 experts run longest first, so the
    // launch does not end on one XCD's long tiles.
    const int nM = (g.M + BM - 1) / BM, TT = nM * nN, share = (TT + 7) / 8;
    const int xcd = blockIdx.x & 7, q = blockIdx.x >> 3;
    int i = xcd * share + q % share;
    t.e = q / share;
    if (g.offsets && g.n_experts <= 64) {
      const int lane = threadIdx.x & 63;
      int lo = 0, hi = -1;
      if (lane < g.n_experts) group_rows(g, lane, lo, hi);
      const int n = hi - lo;
      int rank = 0;
      for (int j = 0; j < g.n_experts; ++j) {
        const int nj = __builtin_amdgcn_readlane(n, j);
        rank += nj > n || (nj == n && j < lane) ? 1 : 0;
      }
      t.e = __builtin_ctzll(__ballot(lane < g.n_experts && rank == t.e));
    }
    constexpr int GM = 4;
    const int fm = i / (GM * nN) * GM, gm = min(GM, nM - fm), within = i - fm * nN;
    t.m0 = (fm + within % gm) * BM;
    t.n0 = within / gm * 256;
    int hi;
    group_rows(g, t.e, t.row0, hi);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.klen = __builtin_amdgcn_readfirstlane(hi) - t.row0;
    t.mrows = i < TT ? min(BM, g.M - t.m0) : 0;
  } else {
    const RowTile r = row_tile<BM, 4>(g, nN);
    t = Tile{r.e, r.row0, r.mrows, 0, r.tn * 256, g.K};
  }
  return t;
}

// Row of C for tile row m, or -1 (past the tile, or an order entry that names
// no row).
__device__ __forceinline__ int out_row(const ExpertArgs& g, const Tile& t, int m) {
  if (m >= t.mrows) return -1;
  const int s = t.row0 + m, v = g.mc.by_order ? g.order[s] : s;
  return (unsigned)v < (unsigned)g.rows ? v : -1;
}

// Epilogues.  acc[fi][fj][4 gg + x] holds C[m = wrow + 32 fi + l32][n = wcol
// + 32 fj + 8 gg + 4 half + x].  fp32 goes straight to memory, four columns a
// lane; bf16 through LDS (every wave is past its last read of the ring):
// 512-byte rows of 32 16-byte granules, granule c of row m at c ^ (m & 31), so
// the rows a fragment writes and the granules a row read takes both spread
// over the banks and every store writes whole 512-byte rows.
template <int FI, bool DW>
__device__ __forceinline__ void store_f32(const ExpertArgs& g, const f32x16 (&acc)[FI][4], const Tile& t, int w,
                                          int lane) {
  const int half = lane >> 5, l32 = lane & 31, wrow = 32 * FI * (w >> 1), wcol = 128 * (w & 1);
#pragma unroll
  for (int fi = 0; fi < FI; ++fi) {
    const int m = wrow + 32 * fi + l32;
    const int row = DW ? (m < t.mrows ? t.m0 + m : -1) : out_row(g, t, m);
    if (row < 0) continue;
    float* crow = static_cast<float*>(g.C) + (DW ? (int64_t)t.e * g.c_expert : 0) + (int64_t)row * g.ldc;
#pragma unroll
    for (int fj = 0; fj < 4; ++fj) {
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) {
        const int n = t.n0 + wcol + 32 * fj + 8 * gg + 4 * half;
        if (n >= g.N) continue;
        f32x4 v = {acc[fi][fj][4 * gg], acc[fi][fj][4 * gg + 1], acc[fi][fj][4 * gg + 2], acc[fi][fj][4 * gg + 3]};
        f32x4* dst = reinterpret_cast<f32x4*>(crow + n);
        if (DW && g.accumulate) v += *dst;
        *dst = v;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}
// dW through LDS: 64 rows x 256 columns a time (one fragment row of every
// wave) in one of two 64 KiB buffers, granule c of row m at c ^ (m & 31), so
// every store instruction writes one whole row of 1 KiB.
template <int FI>
__device__ __forceinline__ void store_dw(const ExpertArgs& g, const f32x16 (&acc)[FI][4], char* ct, const Tile& t,
                                         int w, int lane) {
  const int half = lane >> 5, l32 = lane & 31, wcol = 128 * (w & 1);
  float* const c = static_cast<float*>(g.C) + (int64_t)t.e * g.c_expert;
  const int n = t.n0 + 4 * lane;
  __syncthreads();
#pragma unroll
  for (int fi = 0; fi < FI; ++fi) {
    char* buf = ct + (fi & 1) * 65536;
    const int mw = 32 * (w >> 1) + l32;
#pragma unroll
    for (int fj = 0; fj < 4; ++fj)
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) {
        const f32x4 v = {acc[fi][fj][4 * gg], acc[fi][fj][4 * gg + 1], acc[fi][fj][4 * gg + 2],
                         acc[fi][fj][4 * gg + 3]};
        *reinterpret_cast<f32x4*>(buf + mw * 1024 + 16 * (((wcol >> 2) + 8 * fj + 2 * gg + half) ^ (mw & 31))) = v;
      }
    __syncthreads();
#pragma unroll 4
    for (int it = 0; it < 16; ++it) {
      const int mr = 16 * w + it;
      const int m = 32 * FI * (mr >> 5) + 32 * fi + (mr & 31);
      f32x4 v = *reinterpret_cast<const f32x4*>(buf + mr * 1024 + 16 * (lane ^ (mr & 31)));
      if (m < t.mrows && n < g.N) {
        f32x4* dst = reinterpret_cast<f32x4*>(c + (int64_t)(t.m0 + m) * g.ldc + n);
        if (g.accumulate) v += *dst;
        *dst = v;
      }
    }
  }
}

// dW of a group without rows: zeros (kept when accumulating).
template <int BM>
__device__ __forceinline__ void store_zero(const ExpertArgs& g, const Tile& t) {
  if (g.accumulate) return;
  float* c = static_cast<float*>(g.C) + (int64_t)t.e * g.c_expert;
  const int n = t.n0 + 4 * (threadIdx.x & 63);
  if (n >= g.N) return;
  for (int m = threadIdx.x >> 6; m < t.mrows; m += 4)
    *reinterpret_cast<f32x4*>(c + (int64_t)(t.m0 + m) * g.ldc + n) = f32x4{0.f, 0.f, 0.f, 0.f};
}
template <int FI>
__device__ __forceinline__ void store_bf16(const ExpertArgs& g, const f32x16 (&acc)[FI][4], char* ct, const Tile& t,
                                           int w, int lane) {
  const int half = lane >> 5, l32 = lane & 31, wrow = 32 * FI * (w >> 1), wcol = 128 * (w & 1);
  __syncthreads();
#pragma unroll
  for (int fi = 0; fi < FI; ++fi) {
    const int m = wrow + 32 * fi + l32;
#pragma unroll
    for (int fj = 0; fj < 4; ++fj)
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
  const int gc = lane & 31, n = t.n0 + 8 * gc;
#pragma unroll 4
  for (int it = 0; it < 8 * FI; ++it) {
    const int m = 16 * FI * w + 2 * it + half;
    const int row = out_row(g, t, m);
    const u32x4 x = *reinterpret_cast<const u32x4*>(ct + m * 512 + 16 * (gc ^ (m & 31)));
    if (row >= 0 && n < g.N) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.C) + (int64_t)row * g.ldc + n) = x;
  }
}

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

  const Tile tl = find_tile<BM, DW>(g);
  if (tl.mrows <= 0) return;
  const int e = tl.e, row0 = tl.row0, mrows = tl.mrows, m0 = tl.m0, n0 = tl.n0, klen = tl.klen;
  const int nsteps = (klen + KD - 1) / KD;
  if (DW && nsteps == 0) return store_zero<BM>(g, tl);

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

  issue(0);
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

  if constexpr (F32 || DW) store_f32<FI, DW>(g, acc, tl, w, lane);
  else store_bf16<FI>(g, acc, reinterpret_cast<char*>(&ring[0]), tl, w, lane);
}

// ---------------------------------------------------------------------------
// Pipelined tile kernel for bf16 operands (and E2M1 weights): the base GEMM's
// schedule over ragged groups.  A 64 FI x 256 tile per workgroup of four
// waves, 64-deep steps, one unit of LDS per operand and step.  The ring holds
// as many steps as fit (at most six) and a step copies D steps ahead; with
// 32 KiB units (FI = 4, D = 2) five units fill the 160 KiB, unit u in slot
// u mod 5: while step s is computed, step s + 1 and the A unit of step s + 2
// are in flight.
//
// A step is four 16-deep slices with fragments double buffered in registers;
// the reads and copies sit between the MFMAs of a slice.  Step s:
//   slices 0-1: read the next slice; copy the A unit of step s + D;
//   slice 2: read slice 3; then wait until this wave's copies of step s + 1
//     have landed (later steps may be in flight) and its reads are done, and
//     meet the other waves: step s + 1 is complete in LDS and nobody reads
//     step s any more;
//   slice 3: read step s + 1's first slice; copy the B unit of step s + D.
// E2M1 weights: half h of a wave takes the step's 32-block h, whose 32 codes
// are one 16-byte read per step; word ks of it becomes slice ks's eight bf16
// by four conversions while the slice before is computed, so the weights
// cross LDS at 4 bits and no decoded copy exists.
// ---------------------------------------------------------------------------
template <int AL, int BL, int FI, bool DW, bool GATHER>
__global__ __launch_bounds__(256, 1) void k_expert_pipe(ExpertArgs g) {
  constexpr int FJ = 4, BM = 64 * FI, BN = 256, KD = 64, NS = FI * FJ;
  constexpr int UA = BM * 128, UB = BL == F4 ? BN * 32 + BN * 4 : BN * 128;
  constexpr bool RING5 = FI == 4 && BL != F4;
  constexpr int NR = RING5 ? 2 : (160 * 1024) / (UA + UB) > 6 ? 6 : (160 * 1024) / (UA + UB);
  constexpr int D = RING5 ? 2 : NR - 1;                  // steps ahead that a step copies
  constexpr int CA = UA / 4096, CB = BL == F4 ? 2 : 8;   // 1 KiB copies per wave and unit
  constexpr int CBW = CB + (BL == F4 ? 1 : 0);           // and the scale dwords
  constexpr int RING = RING5 ? 5 * UA : NR * (UA + UB);
  constexpr int LDS = DW || RING >= BM * 512 ? RING : BM * 512;   // the epilogue's bf16 tile takes BM x 512
  __shared__ u32x4 ring[LDS / 16];

  const Tile tl = find_tile<BM, DW>(g);
  if (tl.mrows <= 0) return;
  const int e = tl.e, row0 = tl.row0, mrows = tl.mrows, m0 = tl.m0, n0 = tl.n0, klen = tl.klen;
  const int nsteps = (klen + KD - 1) / KD;
  if (DW && nsteps == 0) return store_zero<BM>(g, tl);

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wrow = 32 * FI * (w >> 1), wcol = 128 * (w & 1);
  const uint8_t* const zero = reinterpret_cast<const uint8_t*>(g_expert_zero);
  const uint8_t* const Be = DW ? g.B : g.B + (int64_t)e * g.b_expert;

  // Copy sources.  k-contiguous: copy i of a wave takes tile rows 8 (C w + i)
  // + lane / 8 at LDS position lane % 8, which holds chunk (lane % 8) ^
  // kx8(row).  n-contiguous: k-rows RPC (C w + i) + lane / CPR, position lane
  // % CPR, chunk ^ nx16(k-row).
  constexpr int CPRA = BM / 8, RPCA = 64 / CPRA, CPRB = BN / 8, RPCB = 64 / CPRB;
  const uint8_t* ap[AL == KC ? CA : 1];  // rows of A anywhere: one pointer per copy
  uint32_t ao[CA], bo[CB];               // else byte offsets from a base that advances by steps
  int ac[CA], bc[CB];                    // KC: chunk; NC: k-row of the step
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    if constexpr (AL == KC) {
      const int r = 8 * (CA * w + i) + (lane >> 3);
      ac[i] = (lane & 7) ^ kx8(r);
      ao[i] = 0;
      ap[i] = g.A + source_row(g, g.ma, row0 + min(r, mrows - 1)) * g.lda * 2 + 16 * ac[i];
    } else {
      ac[i] = RPCA * (CA * w + i) + lane / CPRA;
      const int col = min(m0 + 8 * ((lane % CPRA) ^ nx16(ac[i])), g.M - 8);
      ao[i] = GATHER ? (uint32_t)(col * 2) : (uint32_t)(((int64_t)ac[i] * g.lda + col) * 2);
    }
  }
#pragma unroll
  for (int i = 0; i < CB; ++i) {
    if constexpr (BL == KC) {
      const int r = 8 * (CB * w + i) + (lane >> 3);
      bc[i] = (lane & 7) ^ kx8(r);
      bo[i] = (uint32_t)((int64_t)(min(n0 + r, g.N - 1) - n0) * g.ldb * 2 + 16 * bc[i]);
    } else if constexpr (BL == NC) {
      bc[i] = RPCB * (CB * w + i) + lane / CPRB;
      const int col = min(n0 + 8 * ((lane % CPRB) ^ nx16(bc[i])), g.N - 8);
      bo[i] = GATHER ? (uint32_t)(col * 2) : (uint32_t)(((int64_t)bc[i] * g.ldb + (col - n0)) * 2);
    } else {
      const int r = 32 * (2 * w + i) + (lane >> 1);
      bc[i] = 0;
      bo[i] = (uint32_t)((int64_t)(min(n0 + r, g.N - 1) - n0) * (g.ldb / 2) +
                         16 * ((lane & 1) ^ ((r >> 3) & 1)));
    }
  }
  const uint8_t* sp = nullptr;
  if constexpr (BL == F4) sp = g.b_scale + ((int64_t)e * g.N + min(n0 + 64 * w + lane, g.N - 1)) * (g.ldb / 32);
  // bases of step 0 and bytes per step
  const uint8_t* const baseA = AL == NC && !GATHER ? g.A + (int64_t)row0 * g.lda * 2 : g.A;
  const uint8_t* const baseB =
      BL == KC ? Be + (int64_t)n0 * g.ldb * 2
               : BL == F4 ? Be + (int64_t)n0 * (g.ldb / 2)
                          : (DW && !GATHER ? Be + ((int64_t)row0 * g.ldb + n0) * 2 : (DW ? Be : Be + (int64_t)n0 * 2));
  const int64_t stepA = (int64_t)KD * g.lda * 2;
  const int64_t stepB = BL == KC ? 128 : BL == F4 ? 32 : (int64_t)KD * g.ldb * 2;

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(MLORA_LDS void*)&ring[0]);
  auto slot = [](int u) -> uint32_t {
    if constexpr (RING5) return (uint32_t)(u % 5) * UA;
    else return (uint32_t)((u >> 1) % NR) * (UA + UB) + ((u & 1) ? UA : 0);
  };
  // Order entries of this wave's 16 k-rows of a step, by scalar loads (they
  // wait on lgkmcnt, not on the counter that tracks the copies in flight), and
  // the row that copy i of either operand reads: k-row 16 w + 2 i + lane / 32.
  static_assert(!GATHER || (AL == NC && BL == NC && FI == 4), "both operands copy two k-rows at a time");
  int oidx[GATHER ? 16 : 1];
  auto load_order = [&](int t) {
    if constexpr (GATHER) {
#pragma unroll
      for (int j = 0; j < 16; ++j) oidx[j] = ldc(g.order + row0 + min(t * KD + 16 * w + j, klen - 1));
    }
  };
  auto gathered = [&](const uint8_t* from, const RowMap& map, int64_t ld, int i, int t) -> const uint8_t* {
    const int k = row0 + t * KD + 16 * w + 2 * i;
    auto at = [&](int h) -> int64_t {
      return (map.by_order ? (int64_t)div_fast(read_row(oidx[(2 * i + h) % (GATHER ? 16 : 1)], g.rows), map.div)
                           : (int64_t)(k + h)) *
             ld * 2;
    };
    const int64_t r0 = at(0), r1 = at(1);
    return from + (half ? r1 : r0);
  };
  // Copy i of step t's A (B) unit.  CHECK: the step may pass the end of the
  // reduction, and what does reads zeros.
  auto copy_a = [&](int t, int i, auto check) {
    const uint32_t lds = lds0 + slot(2 * t) + 1024u * (uint32_t)(CA * w + i);
    if constexpr (AL == KC) {
      const uint8_t* src = ap[i] + 128 * (int64_t)t;
      dma16_at(!check.value || t * KD + 8 * ac[i] < klen ? src : zero, lds);
    } else if constexpr (GATHER) {
      dma16_at(!check.value || t * KD + ac[i] < klen ? gathered(baseA, g.ma, g.lda, i, t) + ao[i] : zero, lds);
    } else if constexpr (check.value) {
      const uint8_t* at = reinterpret_cast<const uint8_t*>(uniform64(baseA + t * stepA));
      dma16_at(t * KD + ac[i] < klen ? at + ao[i] : zero, lds);
    } else {
      dma16_sv(uniform64(baseA + t * stepA), ao[i], lds);
    }
  };
  auto copy_b = [&](int t, int i, auto check) {
    const uint32_t lds = lds0 + slot(2 * t + 1) + 1024u * (uint32_t)(CB * w + i);
    if constexpr (BL == NC && GATHER) {
      dma16_at(!check.value || t * KD + bc[i] < klen ? gathered(baseB, g.mb, g.ldb, i, t) + bo[i] : zero, lds);
    } else if constexpr (check.value) {
      const bool on = BL == NC ? t * KD + bc[i] < klen : t * KD + 8 * bc[i] < klen;
      const uint8_t* at = reinterpret_cast<const uint8_t*>(uniform64(baseB + t * stepB));
      dma16_at(on ? at + bo[i] : zero, lds);
    } else {
      dma16_sv(uniform64(baseB + t * stepB), bo[i], lds);
    }
  };
  auto copy_scales = [&](int t, auto check) {
    if constexpr (BL == F4)
      dma4_at(!check.value || t * KD < klen ? sp + 4 * (t >> 1) : zero,
              lds0 + slot(2 * t + 1) + BN * 32 + 256u * (uint32_t)w);
  };

  f32x16 acc[FI][FJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < FJ; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) acc[a][b][x] = 0.f;

  // Fragment reads: a lane part plus the step's slot, made once per step (the
  // empty asm keeps the slot from being folded into every read), plus
  // immediates.  k-contiguous: one lane part per slice; n-contiguous: one per
  // fragment, slices and the second half of the k-rows as immediates (nx16
  // depends on k-row bits 0, 1 and 3 only, which the lane fixes).
  const MLORA_LDS char* const base = (const MLORA_LDS char*)(MLORA_LDS void*)&ring[0];
  uint32_t al[4], bl[4];
  auto lane_kc = [&](int r, int ks) {
    const int c = BL == F4 ? 4 * half + ks : 2 * ks + half;
    return (uint32_t)((r * 8 + (c ^ kx8(l32))) * 16);
  };
  auto lane_nc = [&](int cpr, int col0) {
    const int gq = lane >> 4, sq = lane & 15, kr = 8 * (gq >> 1) + (sq >> 2);
    const int n = col0 + 16 * (gq & 1) + 4 * (sq & 3);
    return (uint32_t)((kr * cpr + ((n >> 3) ^ nx16(kr))) * 16 + 2 * (n & 7));
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    al[i] = AL == KC ? lane_kc(wrow + l32, i) : lane_nc(CPRA, wrow + 32 * (i < FI ? i : 0));
    if constexpr (BL == KC) bl[i] = lane_kc(wcol + l32, i);
    else if constexpr (BL == NC) bl[i] = lane_nc(CPRB, wcol + 32 * i);
    else bl[i] = (uint32_t)(((wcol + 32 * i + l32) * 2 + (half ^ ((l32 >> 3) & 1))) * 16);
  }
  struct Bases {
    uint32_t a[4], b[4];
  };
  auto step_bases = [&](int s, Bases& bs, int ks0, int ks1) {
    const uint32_t sa = slot(2 * s), sb = slot(2 * s + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (AL == NC ? i < FI : (i >= ks0 && i <= ks1)) {
        bs.a[i] = al[i] + sa;
        asm volatile("" : "+v"(bs.a[i]));
      }
      if (BL != KC || (i >= ks0 && i <= ks1)) {
        bs.b[i] = bl[i] + sb;
        asm volatile("" : "+v"(bs.b[i]));
      }
    }
  };
  auto read_tr = [&](uint32_t at, int cpr, int ks) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const MLORA_LDS char* p = base + at + 256 * cpr * ks;
    const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MLORA_LDS s16x4*)p);
    const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MLORA_LDS s16x4*)(p + 64 * cpr));
    const u32x2 u0 = __builtin_bit_cast(u32x2, v0), u1 = __builtin_bit_cast(u32x2, v1);
    return u32x4{u0[0], u0[1], u1[0], u1[1]};
  };
  u32x4 fa[2][FI], fb[2][FJ];
  u32x4 cw[FJ];       // E2M1: the step's codes of this lane's block, and its scales
  float cs[FJ];
  auto read_a = [&](const Bases& bs, int ks, int f, u32x4 (&ra)[FI]) {
    if constexpr (AL == KC) ra[f] = *(const MLORA_LDS u32x4*)(base + bs.a[ks] + 4096 * f);
    else ra[f] = read_tr(bs.a[f], CPRA, ks);
  };
  auto read_b = [&](const Bases& bs, int ks, int f, u32x4 (&rb)[FJ]) {
    if constexpr (BL == KC) rb[f] = *(const MLORA_LDS u32x4*)(base + bs.b[ks] + 4096 * f);
    else if constexpr (BL == NC) rb[f] = read_tr(bs.b[f], CPRB, ks);
    else rb[f] = bf16_of_e2m1(cw[f][ks], cs[f]);
  };
  // E2M1 codes and scales of step s (bases bs).
  auto read_codes = [&](const Bases& bs, int s, int f) {
    if constexpr (BL == F4) {
      cw[f] = *(const MLORA_LDS u32x4*)(base + bs.b[f]);
      const uint32_t sw = *(const MLORA_LDS uint32_t*)(base + slot(2 * s + 1) + BN * 32 + 4 * (wcol + 32 * f + l32));
      cs[f] = __uint_as_float(((sw >> (16 * (s & 1) + 8 * half)) & 255u) << 23);
    }
  };
  // What MFMA slot q of a slice reads of slice ks (bases bs): fragments in the
  // order the first MFMAs need them, two per slot, or one where a fragment is
  // two transposing reads or four conversions and the slice has the slots.
  constexpr int RPS = (AL == KC && BL == KC) || FI == 1 ? 2 : 1;
  auto reads_at = [&](int q, const Bases& bs, int ks, u32x4 (&ra)[FI], u32x4 (&rb)[FJ]) {
#pragma unroll
    for (int j = 0; j < RPS; ++j) {
      const int r = RPS * q + j;
      if (r == 0) read_a(bs, ks, 0, ra);
      else if (r <= FJ) read_b(bs, ks, r - 1, rb);
      else if (r < FI + FJ) read_a(bs, ks, r - FJ, ra);
    }
  };
  auto next_step_reads_at = [&](int q, const Bases& bs, int s, u32x4 (&ra)[FI], u32x4 (&rb)[FJ]) {
    if constexpr (BL != F4) {
      reads_at(q, bs, 0, ra, rb);
    } else {
      if (q < 2) {
        read_codes(bs, s, 2 * q);
        read_codes(bs, s, 2 * q + 1);
      } else if (q == 2) {
#pragma unroll
        for (int f = 0; f < FI; ++f) read_a(bs, 0, f, ra);
      }
      if (q >= NS - FJ) read_b(bs, 0, q - (NS - FJ), rb);
    }
  };
  constexpr int C0 = BL == F4 ? 3 : (FI + FJ + RPS - 1) / RPS;   // first slot that carries a copy
  // Copies j of n spread over the slots from C0 on.
  auto copies_at = [&](int q, int n, auto&& f) {
    const int room = NS - C0, per = (n + room - 1) / room;
    if (q < C0) return;
#pragma unroll
    for (int j = 0; j < per; ++j)
      if ((q - C0) * per + j < n) f((q - C0) * per + j);
  };
  auto mma = [&](int q, const u32x4 (&ra)[FI], const u32x4 (&rb)[FJ]) {
    acc[q >> 2][q & 3] = mfma32(rb[q & 3], ra[q >> 2], acc[q >> 2][q & 3]);
  };

  // Step kinds: 0, step s + D lies inside the reduction; 1, it reaches past
  // its end; 2, it does not exist: nothing is copied and the barrier waits for
  // every copy in flight.
  auto step_block = [&](int s, auto kind) {
    constexpr int KIND = decltype(kind)::value;
    constexpr bool COPY = KIND != 2;
    const std::integral_constant<bool, KIND == 1> check{};
    Bases cur;
    if (COPY) load_order(s + D);
    step_bases(s, cur, 1, 3);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 3; ++ks) {
#pragma unroll
      for (int q = 0; q < NS; ++q) {
        mma(q, fa[ks & 1], fb[ks & 1]);
        reads_at(q, cur, ks + 1, fa[(ks + 1) & 1], fb[(ks + 1) & 1]);
        if (COPY && ks < 2) copies_at(q, CA / 2, [&](int j) { copy_a(s + D, ks * (CA / 2) + j, check); });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_vm_barrier<COPY ? (D - 2) * (CA + CBW) + CA : 0>();
    Bases nxt;
    step_bases(s + 1, nxt, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      mma(q, fa[1], fb[1]);
      next_step_reads_at(q, nxt, s + 1, fa[0], fb[0]);
      if (COPY)
        copies_at(q, CBW, [&](int j) {
          if (j < CB) copy_b(s + D, j, check);
          else copy_scales(s + D, check);
        });
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // the first D steps; step 0's first slice once every wave's copies of it have landed
  const std::integral_constant<bool, true> check{};
#pragma unroll
  for (int t = 0; t < D; ++t) {
    load_order(t);
#pragma unroll
    for (int i = 0; i < CA; ++i) copy_a(t, i, check);
#pragma unroll
    for (int i = 0; i < CB; ++i) copy_b(t, i, check);
    copy_scales(t, check);
  }
  wait_vm_barrier<(D - 1) * (CA + CBW)>();
  Bases b0;
  step_bases(0, b0, 0, 0);
#pragma unroll
  for (int f = 0; f < FJ; ++f) read_codes(b0, 0, f);
#pragma unroll
  for (int f = 0; f < FI; ++f) read_a(b0, 0, f, fa[0]);
#pragma unroll
  for (int f = 0; f < FJ; ++f) read_b(b0, 0, f, fb[0]);
  int s = 0;
  for (; (s + D + 1) * KD <= klen; ++s) step_block(s, std::integral_constant<int, 0>());
  for (; s + D < nsteps; ++s) step_block(s, std::integral_constant<int, 1>());
  for (; s < nsteps; ++s) step_block(s, std::integral_constant<int, 2>());
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  if constexpr (DW) store_dw<FI>(g, acc, reinterpret_cast<char*>(&ring[0]), tl, w, lane);
  else store_bf16<FI>(g, acc, reinterpret_cast<char*>(&ring[0]), tl, w, lane);
}

// ---------------------------------------------------------------------------
// MXFP4 x MXFP4: both operands as E2M1 codes on the scaled matrix cores.
// 256 x 256 tile, steps of 128 of the reduction: 64 bytes of codes and one
// dword of scale codes per row and operand.  Chunk c of row r sits at
// c ^ ((r >> 2) & 3), which spreads a read group's rows over the banks; lane
// r + 32 h holds row r's 32-block h of a 64-deep slice (16 bytes, the low
// nibble first) and supplies its scale.  A step is two slices, 1024 cycles of
// MFMA at FI = 4, less than a copy's latency: four stages keep three steps in
// flight.  A copy of scale dwords touches a row per lane, four times the
// addresses of a copy of codes; S16 (K a multiple of 512, so a row's 16 scale
// bytes are aligned) copies four steps' scales at once instead.
// ---------------------------------------------------------------------------
template <int FI, bool S16>
__global__ __launch_bounds__(256, 1) void k_expert_mx4(ExpertArgs g) {
  constexpr int FJ = 4, BM = 64 * FI, BN = 256;
  constexpr int UA = BM * 64, UB = BN * 64, CA = FI, CB = 4, NS = FI * FJ;
  constexpr int NR = 4;                               // stages
  constexpr int STAGE = UA + UB + (S16 ? 0 : 2048);   // with the scale dwords of 256 rows of A and of B
  constexpr int SCL = NR * STAGE;                     // S16: two chunks of 16 scale bytes for 256 + 256 rows
  constexpr int COPIES = CA + CB + (S16 ? 0 : 2);     // per wave and step
  constexpr int LDS = SCL + (S16 ? 16384 : 0);
  __shared__ u32x4 ring[(LDS > BM * 512 ? LDS : BM * 512) / 16];
  const Tile tl = find_tile<BM, false>(g);
  if (tl.mrows <= 0) return;
  const int e = tl.e, row0 = tl.row0, mrows = tl.mrows, n0 = tl.n0;
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
  // scale dwords: wave w copies those of rows 64 w .. of A and of B
  const uint8_t* as = g.a_scale + source_row(g, g.ma, row0 + min(64 * w + lane, mrows - 1)) * kb;
  const uint8_t* bs = g.b_scale + ((int64_t)e * g.N + min(n0 + 64 * w + lane, g.N - 1)) * kb;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(MLORA_LDS void*)&ring[0]);
  const MLORA_LDS char* const base = (const MLORA_LDS char*)(MLORA_LDS void*)&ring[0];
  auto copy_a = [&](int t, int i) {
    const uint32_t u = lds0 + (uint32_t)(t % NR) * STAGE;
    if (i < CA) {
      dma16_at(ap[i] + 64 * (int64_t)t, u + 1024u * (uint32_t)(CA * w + i));
    } else if constexpr (S16) {
      if ((t & 3) == 0) dma16_at(as + 4 * t, lds0 + SCL + 8192u * ((t >> 2) & 1) + 1024u * (uint32_t)w);
    } else {
      dma4_at(as + 4 * t, u + UA + UB + 256u * (uint32_t)w);
    }
  };
  auto copy_b = [&](int t, int i) {
    const uint32_t u = lds0 + (uint32_t)(t % NR) * STAGE;
    if (i < CB) {
      dma16_at(bp[i] + 64 * (int64_t)t, u + UA + 1024u * (uint32_t)(CB * w + i));
    } else if constexpr (S16) {
      if ((t & 3) == 0) dma16_at(bs + 4 * t, lds0 + SCL + 4096 + 8192u * ((t >> 2) & 1) + 1024u * (uint32_t)w);
    } else {
      dma4_at(bs + 4 * t, u + UA + UB + 1024 + 256u * (uint32_t)w);
    }
  };
  // Scale dword of row r of operand op for step t.
  auto scale_at = [&](int t, int op, int r) -> uint32_t {
    if constexpr (S16)
      return *(const MLORA_LDS uint32_t*)(base + SCL + 8192 * ((t >> 2) & 1) + 4096 * op + 16 * r + 4 * (t & 3));
    else return *(const MLORA_LDS uint32_t*)(base + (uint32_t)(t % NR) * STAGE + UA + UB + 1024 * op + 4 * r);
  };

  f32x16 acc[FI][FJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < FJ; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) acc[a][b][x] = 0.f;
  u32x4 fa[2][FI], fb[2][FJ];
  int sa[FI], sb[FJ], na[FI], nb[FJ];   // scales of the step, and of the next one
  // Lane parts of the reads; fragment f is 32 rows (2048 bytes) on.
  uint32_t al[2], bl[2];
#pragma unroll
  for (int sl = 0; sl < 2; ++sl) {
    const int c = (2 * sl + half) ^ ((l32 >> 2) & 3);
    al[sl] = (uint32_t)(((wrow + l32) * 4 + c) * 16);
    bl[sl] = (uint32_t)(((wcol + l32) * 4 + c) * 16 + UA);
  }
  // Read r of slice sl of step t: fragments in the order the first MFMAs need
  // them, with their scales (shifted to this lane's block) on slice 0.
  auto read = [&](int t, int sl, int r) {
    const uint32_t u = (uint32_t)(t % NR) * STAGE;
    if (r == 0 || (r > FJ && r < FI + FJ)) {
      const int f = r == 0 ? 0 : r - FJ;
      fa[sl][f] = *(const MLORA_LDS u32x4*)(base + u + al[sl] + 2048 * f);
      if (sl == 0)
        na[f] = (int)(scale_at(t, 0, wrow + 32 * f + l32) >> (8 * half));
    } else if (r <= FJ) {
      const int f = r - 1;
      fb[sl][f] = *(const MLORA_LDS u32x4*)(base + u + bl[sl] + 2048 * f);
      if (sl == 0)
        nb[f] = (int)(scale_at(t, 1, wcol + 32 * f + l32) >> (8 * half));
    }
  };
  auto mma = [&](auto sl_tag, int q) {
    constexpr int SL = decltype(sl_tag)::value;
    const int fi = q >> 2, fj = q & 3;
    acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        __builtin_bit_cast(i32x8, __builtin_shufflevector(fb[SL][fj], zero4(), 0, 1, 2, 3, 4, 5, 6, 7)),
        __builtin_bit_cast(i32x8, __builtin_shufflevector(fa[SL][fi], zero4(), 0, 1, 2, 3, 4, 5, 6, 7)), acc[fi][fj], 4,
        4, 2 * SL, sb[fj], 2 * SL, sa[fi]);
  };
  // Step s: slice 0 reads slice 1 and copies the A unit of step
  // s + 3 into the stage that step s - 1 left; then step s + 1 has landed for
  // every wave (steps s + 2 and the A unit of s + 3 may be in flight) and
  // slice 1 reads its first slice and copies the B unit of step s + 3.  The
  // last three steps copy nothing and wait for everything.
  auto step = [&](int s, auto copy_tag) {
    constexpr bool COPY = decltype(copy_tag)::value;
    constexpr int C0 = (FI + FJ + 1) / 2, ROOM = NS - C0;
#pragma unroll
    for (int f = 0; f < FI; ++f) sa[f] = na[f];
#pragma unroll
    for (int f = 0; f < FJ; ++f) sb[f] = nb[f];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      mma(std::integral_constant<int, 0>(), q);
      read(s, 1, 2 * q);
      read(s, 1, 2 * q + 1);
      if (COPY && q >= C0) {
        constexpr int PER = (CA + 1 + ROOM - 1) / ROOM;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if ((q - C0) * PER + j < CA + 1) copy_a(s + 3, (q - C0) * PER + j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    // (counts without the scale copies of every fourth step: a stricter wait)
    wait_vm_barrier<COPY ? COPIES + CA + (S16 ? 0 : 1) : 0>();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      mma(std::integral_constant<int, 1>(), q);
      read(s + 1, 0, 2 * q);
      read(s + 1, 0, 2 * q + 1);
      if (COPY && q >= C0) {
        constexpr int PER = (CB + 1 + ROOM - 1) / ROOM;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if ((q - C0) * PER + j < CB + 1) copy_b(s + 3, (q - C0) * PER + j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  for (int t = 0; t < 3 && t < nsteps; ++t) {
#pragma unroll
    for (int i = 0; i <= CA; ++i) copy_a(t, i);
#pragma unroll
    for (int i = 0; i <= CB; ++i) copy_b(t, i);
  }
  if (nsteps >= 3) wait_vm_barrier<2 * COPIES>();
  else wait_vm_barrier<0>();
#pragma unroll
  for (int r = 0; r < FI + FJ; ++r) read(0, 0, r);
  int s = 0;
  for (; s + 3 < nsteps; ++s) step(s, std::true_type());
  for (; s < nsteps; ++s) step(s, std::false_type());
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  store_bf16<FI>(g, acc, reinterpret_cast<char*>(&ring[0]), tl, w, lane);
}

namespace {

int64_t rows_grid(const ExpertArgs& a, int bm) {
  return max_row_tiles(a.rows, a.offsets ? a.n_experts : 1, bm) * ((a.N + 255) / 256);
}
template <bool F32, int BL>
void rows_size(const ExpertArgs& a, hipStream_t s) {
  const int64_t mean = a.rows / (a.offsets ? a.n_experts : 1);
  if (mean <= 96) {
    const dim3 grid((unsigned)rows_grid(a, 64));
    if constexpr (F32) hipLaunchKernelGGL((k_expert_tile<F32, KC, BL, 1, false>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_expert_pipe<KC, BL, 1, false, false>), grid, dim3(256), 0, s, a);
  } else if (mean <= 384) {
    const dim3 grid((unsigned)rows_grid(a, 128));
    if constexpr (F32) hipLaunchKernelGGL((k_expert_tile<F32, KC, BL, 2, false>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_expert_pipe<KC, BL, 2, false, false>), grid, dim3(256), 0, s, a);
  } else {
    const dim3 grid((unsigned)rows_grid(a, 256));
    if constexpr (F32) hipLaunchKernelGGL((k_expert_tile<F32, KC, BL, 4, false>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_expert_pipe<KC, BL, 4, false, false>), grid, dim3(256), 0, s, a);
  }
}
template <int FI>
void mx4_tile(const ExpertArgs& a, hipStream_t s) {
  const int64_t nN = (a.N + 255) / 256;
  const int64_t grid = max_row_tiles(a.rows, a.offsets ? a.n_experts : 1, 64 * FI) * nN;
  if (a.K % 512 == 0) hipLaunchKernelGGL((k_expert_mx4<FI, true>), dim3((unsigned)grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_expert_mx4<FI, false>), dim3((unsigned)grid), dim3(256), 0, s, a);
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
  const int64_t grid = 8 * E * (((a.M + 255) / 256 * ((a.N + 255) / 256) + 7) / 8);
  const dim3 dg((unsigned)grid);
  if (f32) hipLaunchKernelGGL((k_expert_tile<true, NC, NC, 4, true>), dg, dim3(256), 0, s, a);
  else if (a.ma.by_order || a.mb.by_order)
    hipLaunchKernelGGL((k_expert_pipe<NC, NC, 4, true, true>), dg, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_expert_pipe<NC, NC, 4, true, false>), dg, dim3(256), 0, s, a);
}

}  // namespace mlora
