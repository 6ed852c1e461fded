// Grouped expert products for gfx950: one base weight per group of rows,
// Y = X W_e and dX = dY W_e^T over ragged row groups, dW_e = X^T dY over each
// group's rows, on matrix instructions with fp32 accumulation.
#include "expert_choice.hpp"
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

// Meets the other waves once this wave's LDS accesses are done.  Unlike
// __syncthreads it leaves copies and stores in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// How an operand's elements lie in memory and in LDS.
//   KC: contiguous along the reduction; a unit is one row of 128 bytes per
//       tile row (64 bf16 or 32 fp32 of the reduction), chunk c (16 bytes) of
//       row r at c ^ kx8(r).
//   NC: contiguous along the output; a unit is one row of the tile's output
//       elements per reduction step element.
//   F4: E2M1 codes along the reduction, 32 bytes (64 elements) per tile row,
//       chunk h of row r at h ^ ((r >> 3) & 1), and one dword of scale codes
//       per row that covers the step (it holds 128 elements' scales).
//   X4: E2M1 codes along the reduction on both sides, for the scaled matrix
//       instruction: a KC unit of 256 codes per row, and 8 scale bytes per row
//       and step in LDS of their own.  X4D: the same for rows whose scale
//       codes are aligned to dwords only.
enum { KC = 0, NC = 1, F4 = 2, X4 = 3, X4D = 4 };

// Chunk swizzle of an n-contiguous bf16 row (see the base GEMM): XOR of 4, 8
// and 9 over bits 0, 1 and 3 of the k-row, which gives every transposing read
// group distinct banks.
__device__ __forceinline__ int nx16(int kr) { return ((kr & 1) ? 4 : 0) ^ ((kr & 2) ? 8 : 0) ^ ((kr & 8) ? 9 : 0); }
// fp32: the two half-waves of a fragment read take k-rows 4 apart; the XOR
// puts them on the two halves of the banks.
__device__ __forceinline__ int nx32(int kr) { return (kr & 4) ? 8 : 0; }

// A workgroup's tile: BM rows (dW: rows of dW_e) x BN columns of expert e.
struct Tile {
  int e, row0, mrows;   // grouped rows [row0, row0 + mrows); dW: row0 is the group's first row, mrows the tile's
  int m0, n0;           // first row of dW_e (else 0) and first column
  int klen;             // length of the reduction
  int slot;             // dW: partial sums' slot, or -1: dW itself
};
// dW: where the tile's sums go, and whether they are added to what is there.
__device__ __forceinline__ float* dw_out(const ExpertArgs& g, const Tile& t) {
  return t.slot < 0 ? static_cast<float*>(g.C) + (int64_t)t.e * g.c_expert : g.part + (int64_t)t.slot * g.c_expert;
}
__device__ __forceinline__ bool dw_adds(const ExpertArgs& g, const Tile& t) { return g.accumulate && t.slot < 0; }
template <int BM, int BN, bool DW>
__device__ __forceinline__ Tile find_tile(const ExpertArgs& g) {
  const int nN = (g.N + BN - 1) / BN;
  Tile t;
  if constexpr (DW) {
    const int nM = (g.M + BM - 1) / BM, TT = nM * nN;
    const int xcd = blockIdx.x & 7, q = blockIdx.x >> 3;
    int i;
    t.slot = -1;
    if (g.chunk > 0) {
      // Chunks of equal length: a contiguous run of tiles for each XCD.
      const DwChunks chunks(g);
      const int T = chunks.total * TT, per = T >> 3, rem = T & 7;
      const int L = xcd * per + min(xcd, rem) + q;
      const bool on = q < per + (xcd < rem ? 1 : 0);
      const DwChunk c = chunks.at(g, on ? L / TT : chunks.total);
      i = c.rows >= 0 ? L % TT : TT;
      t.e = c.e;
      t.row0 = c.row0;
      t.klen = max(c.rows, 0);
      t.slot = c.slot;
    } else {
      // Experts have reductions of different lengths: every expert's tiles are
      // spread over all XCDs, and up to 64 experts run longest first, so the
      // launch does not end on one XCD's long tiles.
      const int share = (TT + 7) / 8;
      i = xcd * share + q % share;
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
      int hi;
      group_rows(g, t.e, t.row0, hi);
      t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
      t.klen = __builtin_amdgcn_readfirstlane(hi) - t.row0;
    }
    constexpr int GM = 4;
    const int fm = i / (GM * nN) * GM, gm = max(1, min(GM, nM - fm)), within = i - fm * nN;
    t.m0 = (fm + within % gm) * BM;
    t.n0 = within / gm * BN;
    t.mrows = i < TT ? min(BM, g.M - t.m0) : 0;
  } else {
    const RowTile r = RowTiles<BM, 4>(g, nN).at(g, blockIdx.x);
    t = Tile{r.e, r.row0, r.mrows, 0, r.tn * BN, g.K, -1};
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
// + 32 fj + 8 gg + 4 half + x].  fp32 kernel: straight to memory, four columns
// a lane.
template <int FI, int FJ, bool DW>
__device__ __forceinline__ void store_f32(const ExpertArgs& g, const f32x16 (&acc)[FI][FJ], const Tile& t, int wrow,
                                          int wcol, int lane) {
  const int half = lane >> 5, l32 = lane & 31;
#pragma unroll
  for (int fi = 0; fi < FI; ++fi) {
    const int m = wrow + 32 * fi + l32;
    const int row = DW ? (m < t.mrows ? t.m0 + m : -1) : out_row(g, t, m);
    if (row < 0) continue;
    float* crow = (DW ? dw_out(g, t) : static_cast<float*>(g.C)) + (int64_t)row * g.ldc;
#pragma unroll
    for (int fj = 0; fj < FJ; ++fj) {
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) {
        const int n = t.n0 + wcol + 32 * fj + 8 * gg + 4 * half;
        if (n >= g.N) continue;
        f32x4 v = {acc[fi][fj][4 * gg], acc[fi][fj][4 * gg + 1], acc[fi][fj][4 * gg + 2], acc[fi][fj][4 * gg + 3]};
        f32x4* dst = reinterpret_cast<f32x4*>(crow + n);
        if (DW && dw_adds(g, t)) v += *dst;
        *dst = v;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}
// dW through LDS: 64 rows x BN columns a time (one fragment row of every wave)
// in one of two buffers, granule c of row m at c ^ (m & 31), so every store
// instruction writes whole rows.
template <int FI, int FJ>
__device__ __forceinline__ void store_dw(const ExpertArgs& g, const f32x16 (&acc)[FI][FJ], char* ct, const Tile& t,
                                         int w, int lane) {
  constexpr int BN = 64 * FJ, GPR = BN / 4, RPI = 64 / GPR;
  const int half = lane >> 5, l32 = lane & 31, wcol = 32 * FJ * (w & 1);
  float* const c = dw_out(g, t);
  const bool adds = dw_adds(g, t);
  const int n = t.n0 + 4 * (lane % GPR);
  __syncthreads();
#pragma unroll
  for (int fi = 0; fi < FI; ++fi) {
    char* buf = ct + (fi & 1) * (64 * BN * 4);
    const int mw = 32 * (w >> 1) + l32;
#pragma unroll
    for (int fj = 0; fj < FJ; ++fj)
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) {
        const f32x4 v = {acc[fi][fj][4 * gg], acc[fi][fj][4 * gg + 1], acc[fi][fj][4 * gg + 2],
                         acc[fi][fj][4 * gg + 3]};
        *reinterpret_cast<f32x4*>(buf + mw * (BN * 4) + 16 * (((wcol >> 2) + 8 * fj + 2 * gg + half) ^ (mw & 31))) = v;
      }
    __syncthreads();
#pragma unroll 4
    for (int it = 0; it < 16 / RPI; ++it) {
      const int mr = 16 * w + RPI * it + lane / GPR;
      const int m = 32 * FI * (mr >> 5) + 32 * fi + (mr & 31);
      f32x4 v = *reinterpret_cast<const f32x4*>(buf + mr * (BN * 4) + 16 * ((lane % GPR) ^ (mr & 31)));
      if (m < t.mrows && n < g.N) {
        f32x4* dst = reinterpret_cast<f32x4*>(c + (int64_t)(t.m0 + m) * g.ldc + n);
        if (adds) v += *dst;
        *dst = v;
      }
    }
  }
}

// dW of a group without rows: zeros (kept when accumulating).
template <int BN>
__device__ __forceinline__ void store_zero(const ExpertArgs& g, const Tile& t) {
  if (dw_adds(g, t)) return;
  constexpr int GPR = BN / 4;
  float* c = dw_out(g, t);
  const int n = t.n0 + 4 * (threadIdx.x % GPR);
  if (n >= g.N) return;
  for (int m = threadIdx.x / GPR; m < t.mrows; m += 256 / GPR)
    *reinterpret_cast<f32x4*>(c + (int64_t)(t.m0 + m) * g.ldc + n) = f32x4{0.f, 0.f, 0.f, 0.f};
}
}  // namespace

// ---------------------------------------------------------------------------
// fp32 tile kernel.  A workgroup of four waves (2 x 2) makes a 64 FI x 64 NJ
// tile, each wave 32 FI x 32 NJ in accumulators.  Steps of 32 of the reduction
// are copied straight from global memory into LDS, double buffered: step t + 1
// is in flight while step t is computed.  fp32 matrix instructions run at a
// sixteenth of the bf16 rate, so a step's 16384 cycles (FI = 4) hide its copies
// without a deeper ring.
//   DW = false: C[rc(s)][n] over the rows of one group (rows form)
//   DW = true:  C_e[m][n] = sum over the group's rows (both operands NC)
// Bound by the matrix instructions: 8 x 1000 rows x 2048 x 2048 dW takes 539 us,
// 124 TFLOP/s against 154 of a large library product (tile 256 x 256; 558 with
// 128 x 128).
// ---------------------------------------------------------------------------
template <int AL, int BL, int FI, int NJ, bool DW>
__global__ __launch_bounds__(256, 1) void k_expert_f32(ExpertArgs g) {
  constexpr int BM = 64 * FI, BN = 64 * NJ, KD = 32;
  constexpr int UA = BM * 128, UB = BN * 128;          // bytes of a step's units
  constexpr int CA = UA / 4096, CB = UB / 4096;        // 1 KiB copies per wave
  __shared__ u32x4 ring[2 * (UA + UB) / 16];

  const Tile tl = find_tile<BM, BN, DW>(g);
  if (tl.mrows <= 0) return;
  const int e = tl.e, row0 = tl.row0, mrows = tl.mrows, m0 = tl.m0, n0 = tl.n0, klen = tl.klen;
  const int nsteps = (klen + KD - 1) / KD;
  if (DW && nsteps == 0) return store_zero<BN>(g, tl);

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wrow = 32 * FI * (w >> 1), wcol = 32 * NJ * (w & 1);
  const uint8_t* const Be = DW ? g.B : g.B + (int64_t)e * g.b_expert;
  const uint8_t* const zero = reinterpret_cast<const uint8_t*>(g_expert_zero);

  // k-contiguous: copy i of a wave takes tile rows 8 (C w + i) + lane / 8, LDS
  // position lane % 8.
  const uint8_t* ap[CA];
  const uint8_t* bp[CB];
  int ac[CA], bc[CB];
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    const int r = 8 * (CA * w + i) + (lane >> 3);
    ac[i] = (lane & 7) ^ kx8(r);
    ap[i] = AL == KC ? g.A + source_row(g, g.ma, row0 + min(r, mrows - 1)) * g.lda * 4 + 16 * ac[i] : g.A;
  }
#pragma unroll
  for (int i = 0; i < CB; ++i) {
    const int r = 8 * (CB * w + i) + (lane >> 3);
    bc[i] = (lane & 7) ^ kx8(r);
    bp[i] = BL == KC ? Be + (int64_t)min(n0 + r, g.N - 1) * g.ldb * 4 + 16 * bc[i] : Be;
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(MLORA_LDS void*)&ring[0]);

  // Copies of an n-contiguous unit of RW columns from column c0 of `from`.
  auto copy_nc = [&](auto rw_tag, const uint8_t* from, int64_t ld, int c0, int cmax, const RowMap& map, bool mapped,
                     int t, uint32_t lds) {
    constexpr int RW = decltype(rw_tag)::value, CPR = RW / 4, RPC = 64 / CPR, NCP = RW / 32;
#pragma unroll
    for (int i = 0; i < NCP; ++i) {
      const int kr = RPC * (NCP * w + i) + lane / CPR;   // (CPR < 64: several rows a copy)
      const int col = min(c0 + 4 * ((lane % CPR) ^ nx32(kr)), cmax - 4);
      const int k = t * KD + kr;
      const uint8_t* src = zero;
      if (k < klen) src = from + ((mapped ? source_row(g, map, row0 + k) : (int64_t)k) * ld + col) * 4;
      dma16_at(src, lds + 1024u * (uint32_t)(NCP * w + i));
    }
  };
  auto issue = [&](int t) {
    const uint32_t ua = lds0 + (uint32_t)(t & 1) * (UA + UB), ub = ua + UA;
    if constexpr (AL == KC) {
#pragma unroll
      for (int i = 0; i < CA; ++i)
        dma16_at(t * KD + 4 * ac[i] < klen ? ap[i] + 128 * (int64_t)t : zero, ua + 1024u * (uint32_t)(CA * w + i));
    } else {
      copy_nc(std::integral_constant<int, BM>(), g.A, g.lda, m0, g.M, g.ma, true, t, ua);
    }
    if constexpr (BL == KC) {
#pragma unroll
      for (int i = 0; i < CB; ++i)
        dma16_at(t * KD + 4 * bc[i] < klen ? bp[i] + 128 * (int64_t)t : zero, ub + 1024u * (uint32_t)(CB * w + i));
    } else {
      copy_nc(std::integral_constant<int, BN>(), Be, g.ldb, n0, g.N, g.mb, DW, t, ub);
    }
  };

  f32x16 acc[FI][NJ];
#pragma unroll
  for (int a = 0; a < FI; ++a)
#pragma unroll
    for (int b = 0; b < NJ; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) acc[a][b][x] = 0.f;

  const MLORA_LDS char* const base = (const MLORA_LDS char*)(MLORA_LDS void*)&ring[0];
  // Four values of the reduction per lane: slice ks, half h holds 8 ks + 4 h ..
  auto frag = [&](auto kc_tag, auto rw_tag, uint32_t unit, int r0, int ks) {
    constexpr int CPR = decltype(rw_tag)::value / 4;
    const int r = r0 + l32;
    u32x4 out;
    if constexpr (decltype(kc_tag)::value) {
      out = *(const MLORA_LDS u32x4*)(base + unit + (r * 8 + ((2 * ks + half) ^ kx8(r))) * 16);
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int kr = 8 * ks + 4 * half + x;
        out[x] = *(const MLORA_LDS uint32_t*)(base + unit + (kr * CPR + ((r >> 2) ^ nx32(kr))) * 16 + 4 * (r & 3));
      }
    }
    return out;
  };

  issue(0);
  for (int t = 0; t < nsteps; ++t) {
    // step t has landed, and every wave is done with the other buffer
    wait_vm_barrier<0>();
    if (t + 1 < nsteps) issue(t + 1);
    const uint32_t ua = (uint32_t)(t & 1) * (UA + UB), ub = ua + UA;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      u32x4 fa[FI], fb[NJ];
#pragma unroll
      for (int f = 0; f < FI; ++f)
        fa[f] = frag(std::integral_constant<bool, AL == KC>(), std::integral_constant<int, BM>(), ua, wrow + 32 * f, ks);
#pragma unroll
      for (int f = 0; f < NJ; ++f)
        fb[f] = frag(std::integral_constant<bool, BL == KC>(), std::integral_constant<int, BN>(), ub, wcol + 32 * f, ks);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int fi = 0; fi < FI; ++fi)
#pragma unroll
          for (int fj = 0; fj < NJ; ++fj)
            acc[fi][fj] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(fb[fj][x]), __uint_as_float(fa[fi][x]),
                                                               acc[fi][fj], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    // this wave's reads are done before the next barrier lets others overwrite
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  store_f32<FI, NJ, DW>(g, acc, tl, wrow, wcol, lane);
}

// ---------------------------------------------------------------------------
// Pipelined tile kernel for bf16 operands (and E2M1 weights): the base GEMM's
// schedule over ragged groups.  A 64 FI x 64 NJ tile per workgroup of four
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
//
// Bound by the matrix instructions where tiles are full (32768 rows over 64
// skewed experts, 4096 -> 14336: 4.34 ms, 1090 TFLOP/s counting the padding of
// last tiles, 890 without; dW of 7680 rows x 4096 x 4096 over 4 experts 241 us,
// 1070 TFLOP/s).  MXFP4 x MXFP4, 8192 rows, 4096 -> 14336: 292 us, 3.3
// PFLOP/s, of which matrix and address instructions alone take 200 and the
// stores 34: the scales take the place of a fifth unit, so a copy has three
// quarters of a step to land.  bf16 x MXFP4, 4096 rows over 32 experts, 4096 ->
// 1024: 60 us (about 192 tiles of 128 x 256, half full on average, on 256 CUs).
// ---------------------------------------------------------------------------
template <int AL, int BL, int FI, int NJ, bool DW, int GATHER>
__global__ __launch_bounds__(256, 1) void k_expert_pipe(ExpertArgs) {
  constexpr bool S4 = AL >= X4, S16 = AL == X4;          // both operands E2M1; their scales' alignment
  constexpr bool AK = AL != NC, BK = BL == KC || S4;     // k-contiguous 128-byte rows
  constexpr int BM = 64 * FI, BN = 64 * NJ, KD = S4 ? 256 : 64, EPC = S4 ? 32 : 8;
  // Waves along M: with E2M1 weights each wave decodes its own columns, so the
  // four waves share the columns out and all take every row.
  constexpr int WM = BL == F4 ? 1 : 2, FIW = BM / 32 / WM, FJW = BN / 32 / (4 / WM), NS = FIW * FJW;
  constexpr int UA = BM * 128, UB = BL == F4 ? BN * 32 + 1024 : BN * 128;
  // Ring: five units (RING5), four units (RING4: the scales take the rest), or
  // NR whole steps; D: steps ahead that a step copies.
  constexpr bool RING5 = UA + UB == 65536 && !S4, RING4 = UA + UB == 65536 && S4;
  constexpr int SCL = !S4 ? 0 : NJ < 4 ? 32768 : 16384, FIT = (160 * 1024 - SCL) / (UA + UB);
  // Small tiles (few MFMAs a slice) read a whole step's fragments ahead (those
  // of 64 x 256 with both operands' scales would not fit the registers).
  constexpr bool SMALL = !DW && NS <= 4 && !(S4 && NJ == 4);
  constexpr int NR = RING5 || RING4 ? 2 : FIT > 6 ? 6 : FIT;
  constexpr int D = RING5 || RING4 ? 2 : NR - 1;
  constexpr int CA = UA / 4096, CB = UB / 4096;          // 1 KiB copies per wave and unit
  constexpr int CBW = CB + (BL == F4 ? 1 : 0);           // and the scale dwords
  constexpr int RING = RING5 ? 5 * UA : NR * (UA + UB);
  // What the first D steps of a tile leave free: the epilogue's rows.
  constexpr int SPARE = RING5 ? 4 * UA : RING4 ? 2 * UA : (NR - 1) * (UA + UB);
  static_assert(DW || (RING5 || RING4 ? UA : UA + UB) >= (WM == 2 ? 64 : 32) * 2 * BN, "an epilogue phase fits");
  __shared__ u32x4 ring[(RING + SCL) / 16];

  const RowTiles<BM, 4> tiles(kernel_args(), DW ? 0 : (kernel_args().N + BN - 1) / BN);
  auto rows_tile = [&](int b) {
    const ExpertArgs& g = kernel_args();
    const RowTile r = tiles.at(g, b);
    return Tile{r.e, r.row0, r.mrows, 0, r.tn * BN, g.K, -1};
  };
  Tile tl;
  if constexpr (DW) tl = find_tile<BM, BN, DW>(kernel_args());
  else tl = rows_tile(blockIdx.x);
  if (tl.mrows <= 0) return;
  const int klen = tl.klen, nsteps = (klen + KD - 1) / KD;
  if (DW && nsteps == 0) return store_zero<BN>(kernel_args(), tl);

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wrow = WM == 2 ? 32 * FIW * (w >> 1) : 0, wcol = 32 * FJW * (WM == 2 ? w & 1 : w);
  const uint8_t* const zero = reinterpret_cast<const uint8_t*>(g_expert_zero);
  // bytes of a row of either operand
  auto a_row = [](const ExpertArgs& g) -> int64_t { return S4 ? g.lda / 2 : g.lda * 2; };
  auto b_row = [](const ExpertArgs& g) -> int64_t { return BL == F4 || S4 ? g.ldb / 2 : g.ldb * 2; };

  // Copy sources.  k-contiguous: copy i of a wave takes tile rows 8 (C w + i)
  // + lane / 8 at LDS position lane % 8, which holds chunk (lane % 8) ^
  // kx8(row).  n-contiguous: k-rows RPC (C w + i) + lane / CPR, position lane
  // % CPR, chunk ^ nx16(k-row).
  constexpr int CPRA = BM / 8, RPCA = 64 / CPRA, CPRB = BN / 8, RPCB = 64 / CPRB;
  const uint8_t* ap[AK ? CA : 1];  // rows of A anywhere: one pointer per copy
  uint32_t ao[CA], bo[CB];               // else byte offsets from a base that advances by steps
  int ac[CA], bc[CB];                    // KC: chunk; NC: k-row of the step
  // scale codes: F4 and X4 rows of B, wave w copying those of rows 64 w ..; X4 rows of A the same way
  const uint8_t* sp = nullptr;
  const uint8_t* sq = nullptr;
  // bases of step 0 and bytes per step
  const uint8_t* baseA = nullptr;
  const uint8_t* baseB = nullptr;
  const int64_t arow = a_row(kernel_args()), brow = b_row(kernel_args());   // dead where not used below
  const int64_t stepA = KD * arow;
  const int64_t stepB = BK ? 128 : BL == F4 ? 32 : KD * brow;
  auto place = [&](const Tile& t) {
    // (opaque: else the loop over tiles keeps every lane's share of this in
    // registers beside the accumulators)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const ExpertArgs& g = kernel_args();
    const int64_t arow = a_row(g), brow = b_row(g);
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      if constexpr (AK) {
        const int r = 8 * (CA * w + i) + (lane >> 3);
        ac[i] = (lane & 7) ^ kx8(r);
        ao[i] = 0;
        ap[i] = g.A + source_row(g, g.ma, t.row0 + min(r, t.mrows - 1)) * arow + 16 * ac[i];
      } else {
        ac[i] = RPCA * (CA * w + i) + lane / CPRA;
        const int col = min(t.m0 + 8 * ((lane % CPRA) ^ nx16(ac[i])), g.M - 8);
        ao[i] = (uint32_t)((GATHER & 1 ? 0 : ac[i] * arow) + col * 2);
      }
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      if constexpr (BK) {
        const int r = 8 * (CB * w + i) + (lane >> 3);
        bc[i] = (lane & 7) ^ kx8(r);
        bo[i] = (uint32_t)((min(t.n0 + r, g.N - 1) - t.n0) * brow + 16 * bc[i]);
      } else if constexpr (BL == NC) {
        bc[i] = RPCB * (CB * w + i) + lane / CPRB;
        const int col = min(t.n0 + 8 * ((lane % CPRB) ^ nx16(bc[i])), g.N - 8);
        bo[i] = (uint32_t)(GATHER & 2 ? col * 2 : bc[i] * brow + (col - t.n0) * 2);
      } else {
        const int r = 32 * (CB * w + i) + (lane >> 1);
        bc[i] = 0;
        bo[i] = (uint32_t)((min(t.n0 + r, g.N - 1) - t.n0) * brow + 16 * ((lane & 1) ^ ((r >> 3) & 1)));
      }
    }
    if constexpr (BL == F4 || S4)
      sp = g.b_scale + ((int64_t)t.e * g.N + min(t.n0 + 64 * w + lane, g.N - 1)) * (g.ldb / 32);
    if constexpr (S4) sq = g.a_scale + source_row(g, g.ma, t.row0 + min(64 * w + lane, t.mrows - 1)) * (g.lda / 32);
    const uint8_t* Be = DW ? g.B : g.B + (int64_t)t.e * g.b_expert;
    baseA = AL == NC && !(GATHER & 1) ? g.A + t.row0 * arow : g.A;
    baseB = BL != NC ? Be + t.n0 * brow : (GATHER & 2 ? Be : Be + (DW ? t.row0 * brow : 0) + t.n0 * 2);
  };

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(MLORA_LDS void*)&ring[0]);
  const uint32_t lds_a = lds0 + 1024u * (uint32_t)(CA * w), lds_b = lds0 + 1024u * (uint32_t)(CB * w);
  // (readfirstlane: the compiler may count steps in a vector register, and an
  // LDS address of a copy has to be scalar)
  auto slot = [](int v) -> uint32_t {
    const int u = __builtin_amdgcn_readfirstlane(v);
    if constexpr (RING5) return (uint32_t)(u % 5) * UA;
    else if constexpr (RING4) return (uint32_t)(u & 3) * UA;
    else return (uint32_t)((u >> 1) % NR) * (UA + UB) + ((u & 1) ? UA : 0);
  };
  // Order entries of this wave's 16 k-rows of a step, by scalar loads (they
  // wait on lgkmcnt, not on the counter that tracks the copies in flight).
  // Copy i of either operand reads k-rows 16 w + RPC i + lane / CPR: the lane's
  // entry is selected first, so the row behind it is computed once per copy
  // and lane and not in scalar registers for every row.
  static_assert(!GATHER || (AL == NC && BL == NC && BM == BN), "both operands copy the same k-rows");
  int oidx[GATHER ? 16 : 1];
  const int32_t* const order = GATHER ? kernel_args().order : nullptr;
  const DivBy diva = kernel_args().ma.div, divb = kernel_args().mb.div;   // GATHER only
  const int nrows = kernel_args().rows;
  auto load_order = [&](int t, auto check) {
    if constexpr (GATHER != 0 && check.value) {
#pragma unroll
      for (int j = 0; j < 16; ++j) oidx[j] = ldc(order + tl.row0 + min(t * KD + 16 * w + j, klen - 1));
    } else if constexpr (GATHER != 0) {
      typedef int i32x16 __attribute__((ext_vector_type(16), aligned(4)));
      const i32x16 v = *(const __attribute__((address_space(4))) i32x16*)(order + tl.row0 + t * KD + 16 * w);
#pragma unroll
      for (int j = 0; j < 16; ++j) oidx[j] = v[j];
    }
  };
  static_assert(!GATHER || RPCA == 2 || RPCA == 4, "k-rows of a copy");
  // masks of the lanes on odd k-rows of a copy and on its rows 2 and 3 (opaque:
  // of selects by lane the compiler makes one chain over all 16 entries)
  int odd = GATHER && (lane / CPRA & 1) ? -1 : 0, upper = GATHER && (lane / CPRA & 2) ? -1 : 0;
  if constexpr (GATHER != 0) asm volatile("" : "+v"(odd), "+v"(upper));
  auto gathered = [&](const uint8_t* from, const DivBy& div, int64_t row_bytes, int i) -> const uint8_t* {
    auto entry = [&](int h) { return oidx[(RPCA * i + h) % (GATHER ? 16 : 1)]; };
    auto pick = [](int mask, int b, int a) { return (mask & b) | (~mask & a); };
    int v = pick(odd, entry(1), entry(0));
    if constexpr (RPCA == 4) v = pick(upper, pick(odd, entry(3), entry(2)), v);
    return from + (uint64_t)div_fast(read_row(v, nrows), div) * (uint32_t)row_bytes;
  };
  // Copy i of step t's A (B) unit.  CHECK: the step may pass the end of the
  // reduction, and what does reads zeros.
  auto copy_a = [&](int t, int i, auto check) {
    const uint32_t lds = lds_a + slot(2 * t) + 1024u * i;
    if constexpr (AK) {
      const uint8_t* src = ap[i] + 128 * (int64_t)t;
      dma16_at(!check.value || t * KD + EPC * ac[i] < klen ? src : zero, lds);
    } else if constexpr (GATHER & 1) {
      dma16_at(!check.value || t * KD + ac[i] < klen ? gathered(baseA + ao[i], diva, arow, i) : zero, lds);
    } else if constexpr (check.value) {
      const uint8_t* at = reinterpret_cast<const uint8_t*>(uniform64(baseA + t * stepA));
      dma16_at(t * KD + ac[i] < klen ? at + ao[i] : zero, lds);
    } else {
      dma16_sv(uniform64(baseA + t * stepA), ao[i], lds);
    }
  };
  auto copy_b = [&](int t, int i, auto check) {
    const uint32_t lds = lds_b + slot(2 * t + 1) + 1024u * i;
    if constexpr (BL == NC && (GATHER & 2) != 0) {
      dma16_at(!check.value || t * KD + bc[i] < klen ? gathered(baseB + bo[i], divb, brow, i) : zero, lds);
    } else if constexpr (check.value) {
      const bool on = BL == NC ? t * KD + bc[i] < klen : t * KD + EPC * bc[i] < klen;
      const uint8_t* at = reinterpret_cast<const uint8_t*>(uniform64(baseB + t * stepB));
      dma16_at(on ? at + bo[i] : zero, lds);
    } else {
      dma16_sv(uniform64(baseB + t * stepB), bo[i], lds);
    }
  };
  // X4 scale codes: 8 bytes per row and step.  A copy of dwords touches a row
  // per lane, four times the addresses of a copy of codes, so where a row's 16
  // bytes are aligned (S16: K a multiple of 512) two steps' codes are copied at
  // once: [chunk][operand][row] of 16 bytes; else [step][dword][operand][row]
  // of 4.  A ring of NCH chunks (2 NCH steps): a chunk's copy, D + 1 steps
  // ahead at most, meets the place of one whose reads are over.  (The waits
  // below count neither: they are stricter by what is in flight.)
  constexpr int NCH = SCL > 0 ? SCL / 8192 : 1;
  static_assert(!S4 || (NCH == 2 ? D <= 2 : D <= 4), "the ring of scales covers the steps in flight");
  auto copy_scales = [&](int t, auto check) {
    if constexpr (BL == F4) {
      dma4_at(!check.value || t * KD < klen ? sp + 4 * (t >> 1) : zero,
              lds0 + slot(2 * t + 1) + BN * 32 + 256u * (uint32_t)w);
    } else if constexpr (S4) {
      if constexpr (S16) {
        // even steps: A's codes of the two steps from t on; odd steps: B's of
        // the two after t, so every step has one copy and no branch
        const int odd = __builtin_amdgcn_readfirstlane(t & 1), c = __builtin_amdgcn_readfirstlane((t + 1) >> 1);
        dma16_at(c * 512 < klen ? (odd ? sp : sq) + 16 * c : zero,
                 lds0 + RING + 8192u * (c % NCH) + 4096u * odd + 1024u * (uint32_t)w);
      } else {
        const uint32_t at =
            lds0 + RING + 4096u * (uint32_t)__builtin_amdgcn_readfirstlane(t % (2 * NCH)) + 256u * (uint32_t)w;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const bool on = t * KD + 128 * d < klen;
          dma4_at(on ? sq + 8 * t + 4 * d : zero, at + 2048 * d);
          dma4_at(on ? sp + 8 * t + 4 * d : zero, at + 2048 * d + 1024);
        }
      }
    }
  };

  f32x16 acc[FIW][FJW];

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
    al[i] = AK ? lane_kc(wrow + l32, i) : lane_nc(CPRA, wrow + 32 * (i < FIW ? i : 0));
    if constexpr (BK) bl[i] = lane_kc(wcol + l32, i);
    else if constexpr (BL == NC) bl[i] = lane_nc(CPRB, wcol + 32 * (i < FJW ? i : 0));
    else bl[i] = (uint32_t)(((wcol + 32 * (i < FJW ? i : 0) + l32) * 2 + (half ^ ((l32 >> 3) & 1))) * 16);
  }
  struct Bases {
    uint32_t a[4], b[4], sa, sb;   // and X4's scales of A and B
  };
  auto step_bases = [&](int s, Bases& bs, int ks0, int ks1) {
    const uint32_t sa = slot(2 * s), sb = slot(2 * s + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (AL == NC ? i < FIW : (i >= ks0 && i <= ks1)) {
        bs.a[i] = al[i] + sa;
        asm volatile("" : "+v"(bs.a[i]));
      }
      if (BK ? (i >= ks0 && i <= ks1) : i < FJW) {
        bs.b[i] = bl[i] + sb;
        asm volatile("" : "+v"(bs.b[i]));
      }
    }
    if constexpr (S4) {
      const uint32_t at = RING + (S16 ? 8192u * ((s >> 1) % NCH) + 8u * (s & 1) : 4096u * (s % (2 * NCH)));
      bs.sa = at + (S16 ? 16u : 4u) * (uint32_t)(wrow + l32);
      bs.sb = at + (S16 ? 4096u : 1024u) + (S16 ? 16u : 4u) * (uint32_t)(wcol + l32);
      asm volatile("" : "+v"(bs.sa), "+v"(bs.sb));
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
  u32x4 fa[2][FIW], fb[2][FJW];
  u32x4 cw[FJW];                    // F4: the step's codes of this lane's block, and their scale
  float cs[FJW];
  int sa[2][FIW], sb[2][FJW];       // X4: scale dwords of slices 0-1 and 2-3, shifted to this lane's block
  auto read_a = [&](const Bases& bs, int ks, int f, u32x4 (&ra)[FIW]) {
    if constexpr (AK) ra[f] = *(const MLORA_LDS u32x4*)(base + bs.a[ks] + 4096 * f);
    else ra[f] = read_tr(bs.a[f], CPRA, ks);
  };
  auto read_b = [&](const Bases& bs, int ks, int f, u32x4 (&rb)[FJW]) {
    if constexpr (BK) rb[f] = *(const MLORA_LDS u32x4*)(base + bs.b[ks] + 4096 * f);
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
  // X4: scale dword d of fragment f, from either operand's base.
  auto read_scale = [&](uint32_t at, int d, int f) {
    return (int)(*(const MLORA_LDS uint32_t*)(base + at + (S16 ? 512 * f + 4 * d : 128 * f + 2048 * d)) >> (8 * half));
  };
  // What MFMA slot q of a slice reads of slice ks (bases bs):
  // fragments in the order the first MFMAs need them, two per slot, or one
  // where a fragment is two transposing reads or four conversions and the
  // slice has a slot for each; X4: with the scales of slices ks and ks + 1.
  constexpr int RPS = (AK && BK) || FI == 1 || FIW + FJW > NS ? 2 : 1;
  static_assert(FIW + FJW <= RPS * NS, "a slice's slots read all of the next one's fragments");
  auto reads_at = [&](int q, const Bases& bs, int ks, u32x4 (&ra)[FIW], u32x4 (&rb)[FJW]) {
#pragma unroll
    for (int j = 0; j < RPS; ++j) {
      const int r = RPS * q + j;
      if (r == 0 || (r > FJW && r < FIW + FJW)) {
        const int f = r == 0 ? 0 : r - FJW;
        read_a(bs, ks, f, ra);
        if (S4 && (ks & 1) == 0) sa[ks >> 1][f] = read_scale(bs.sa, ks >> 1, f);
      } else if (r <= FJW) {
        read_b(bs, ks, r - 1, rb);
        if (S4 && (ks & 1) == 0) sb[ks >> 1][r - 1] = read_scale(bs.sb, ks >> 1, r - 1);
      }
    }
  };
  auto next_step_reads_at = [&](int q, const Bases& bs, int t, u32x4 (&ra)[FIW], u32x4 (&rb)[FJW]) {
    if constexpr (BL != F4) {
      reads_at(q, bs, 0, ra, rb);
    } else {
      // the step's codes first, its conversions last
      if (q < FJW) read_codes(bs, t, q);
#pragma unroll
      for (int f = 0; f < FIW; ++f)
        if (q == (NS >= FIW + 2 * FJW ? FJW + f : FJW - 1)) read_a(bs, 0, f, ra);
      if (q >= NS - FJW) read_b(bs, 0, q - (NS - FJW), rb);
    }
  };
  // first slot that carries a copy
  constexpr int READS = (FIW + FJW + RPS - 1) / RPS, C0 = READS < NS / 2 ? READS : NS / 2;
  // Copies j of n spread over the slots from C0 on.
  auto copies_at = [&](int q, int n, auto&& f) {
    const int room = NS - C0, per = (n + room - 1) / room;
    if (q < C0) return;
#pragma unroll
    for (int j = 0; j < per; ++j)
      if ((q - C0) * per + j < n) f((q - C0) * per + j);
  };
  auto mma = [&](int q, int ks, const u32x4 (&ra)[FIW], const u32x4 (&rb)[FJW]) {
    const int fi = q / FJW, fj = q % FJW;
    if constexpr (S4) {
      const i32x8 b8 = __builtin_bit_cast(i32x8, __builtin_shufflevector(rb[fj], zero4(), 0, 1, 2, 3, 4, 5, 6, 7));
      const i32x8 a8 = __builtin_bit_cast(i32x8, __builtin_shufflevector(ra[fi], zero4(), 0, 1, 2, 3, 4, 5, 6, 7));
      const int sbv = sb[ks >> 1][fj], sav = sa[ks >> 1][fi];
      if (ks & 1)
        acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[fi][fj], 4, 4, 2, sbv, 2, sav);
      else
        acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[fi][fj], 4, 4, 0, sbv, 0, sav);
    } else {
      acc[fi][fj] = mfma32(rb[fj], ra[fi], acc[fi][fj]);
    }
  };

  // Step kinds: 0, step s + D lies inside the reduction; 1, it reaches past
  // its end; 2, it does not exist: nothing is copied and the barrier waits for
  // every copy in flight.  RING4 has no spare unit for A: its unit of step
  // s + 1 is copied in slice 0 of step s (kind 3: step s + 1 is the last).
  auto step_block = [&](int s, auto kind) {
    constexpr int KIND = decltype(kind)::value;
    constexpr bool COPY = KIND < 2, COPY_A = RING4 ? KIND != 2 : COPY;
    const std::integral_constant<bool, KIND != 0> check{};
    Bases cur;
    if (COPY) load_order(s + D, check);
    step_bases(s, cur, 1, 3);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 3; ++ks) {
#pragma unroll
      for (int q = 0; q < NS; ++q) {
        mma(q, ks, fa[ks & 1], fb[ks & 1]);
        reads_at(q, cur, ks + 1, fa[(ks + 1) & 1], fb[(ks + 1) & 1]);
        if (RING4 && COPY_A && ks == 0) copies_at(q, CA, [&](int j) { copy_a(s + 1, j, check); });
        if (!RING4 && COPY_A && ks < 2) copies_at(q, CA / 2, [&](int j) { copy_a(s + D, ks * (CA / 2) + j, check); });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_vm_barrier<COPY && !RING4 ? (D - 2) * (CA + CBW) + CA : 0>();
    Bases nxt;
    step_bases(s + 1, nxt, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      mma(q, 3, fa[1], fb[1]);
      next_step_reads_at(q, nxt, s + 1, fa[0], fb[0]);
      if (COPY)
        copies_at(q, CB + 1, [&](int j) {
          if (j < CB) copy_b(s + D, j, check);
          else copy_scales(s + D, check);
        });
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // SMALL: a step's MFMAs are too few to hide an LDS read, so step s reads all
  // of step s + 1's fragments (set 1 - P) while its MFMAs take their own (set
  // P).  At its barrier step s + 1 has landed and every wave holds step s in
  // registers; the copies of step s + D go to the slot of step s - 1.
  constexpr int SET = SMALL ? 2 : 1;
  u32x4 ga[SET][4][FIW], gb[SET][BL == F4 ? 1 : 4][FJW];   // F4: the codes of the step
  float gc[SET][FJW];
  int gsa[SET][2][FIW], gsb[SET][2][FJW];
  auto read_ahead = [&](const Bases& bs, int t, int set, int r) {
    if constexpr (BL == F4) {
      if (r < FJW) {
        read_codes(bs, t, r);
        gb[set][0][r] = cw[r];
        gc[set][r] = cs[r];
      } else if (r < FJW + 4 * FIW) {
        const int ks = (r - FJW) / FIW, f = (r - FJW) % FIW;
        ga[set][ks][f] = *(const MLORA_LDS u32x4*)(base + bs.a[ks] + 4096 * f);
      }
    } else if (r < 4 * (FIW + FJW)) {
      const int ks = r / (FIW + FJW), f = r % (FIW + FJW);
      if (f < FIW) {
        if constexpr (AK) ga[set][ks][f] = *(const MLORA_LDS u32x4*)(base + bs.a[ks] + 4096 * f);
        if (S4 && (ks & 1) == 0) gsa[set][ks >> 1][f] = read_scale(bs.sa, ks >> 1, f);
      } else {
        const int j = f - FIW;
        if constexpr (BK) gb[set][ks][j] = *(const MLORA_LDS u32x4*)(base + bs.b[ks] + 4096 * j);
        else gb[set][ks][j] = read_tr(bs.b[j], CPRB, ks);
        if (S4 && (ks & 1) == 0) gsb[set][ks >> 1][j] = read_scale(bs.sb, ks >> 1, j);
      }
    }
  };
  auto small_step = [&](int s, auto par, auto kind) {
    constexpr int P = decltype(par)::value, KIND = decltype(kind)::value;
    constexpr bool COPY = KIND < 2;
    const std::integral_constant<bool, KIND != 0> check{};
    constexpr int SLOTS = 4 * NS, READS = BL == F4 ? FJW + 4 * FIW : 4 * (FIW + FJW);
    constexpr int RPQ = (READS + SLOTS - 1) / SLOTS, NC = CA + CB + (BL == F4 || S4 ? 1 : 0);
    constexpr int CPQ = (NC + SLOTS - 1) / SLOTS;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_vm_barrier<COPY ? (D - 2) * (CA + CBW) : 0>();
    Bases nxt;
    step_bases(s + 1, nxt, 0, 3);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
      const int ks = q / NS, fi = q % NS / FJW, fj = q % FJW;
#pragma unroll
      for (int j = 0; j < RPQ; ++j) read_ahead(nxt, s + 1, 1 - P, RPQ * q + j);
      if constexpr (S4) {
        const i32x8 b8 =
            __builtin_bit_cast(i32x8, __builtin_shufflevector(gb[P][ks][fj], zero4(), 0, 1, 2, 3, 4, 5, 6, 7));
        const i32x8 a8 =
            __builtin_bit_cast(i32x8, __builtin_shufflevector(ga[P][ks][fi], zero4(), 0, 1, 2, 3, 4, 5, 6, 7));
        const int sbv = gsb[P][ks >> 1][fj], sav = gsa[P][ks >> 1][fi];
        if (ks & 1)
          acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[fi][fj], 4, 4, 2, sbv, 2, sav);
        else
          acc[fi][fj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc[fi][fj], 4, 4, 0, sbv, 0, sav);
      } else if constexpr (BL == F4) {
        acc[fi][fj] = mfma32(bf16_of_e2m1(gb[P][0][fj][ks], gc[P][fj]), ga[P][ks][fi], acc[fi][fj]);
      } else {
        acc[fi][fj] = mfma32(gb[P][ks][fj], ga[P][ks][fi], acc[fi][fj]);
      }
      if (COPY) {
#pragma unroll
        for (int j = 0; j < CPQ; ++j) {
          const int c = CPQ * q + j;
          if (c < CA) copy_a(s + D, c, check);
          else if (c < CA + CB) copy_b(s + D, c - CA, check);
          else if (c < NC) copy_scales(s + D, check);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The first D steps of a tile.
  auto prologue = [&]() {
    const std::integral_constant<bool, true> check{};
    if constexpr (S16) dma16_at(sp, lds0 + RING + 4096u + 1024u * (uint32_t)w);   // B's scales of steps 0 and 1
#pragma unroll
    for (int t = 0; t < D; ++t) {
      load_order(t, check);
      if (!(RING4 && t == 1)) {
#pragma unroll
        for (int i = 0; i < CA; ++i) copy_a(t, i, check);
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) copy_b(t, i, check);
      copy_scales(t, check);
    }
  };
  auto main_loop = [&]() {
#pragma unroll
    for (int a = 0; a < FIW; ++a)
#pragma unroll
      for (int b = 0; b < FJW; ++b)
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[a][b][x] = 0.f;
    // step 0's first reads once every wave's copies of it have landed
    wait_vm_barrier<RING4 ? CB : (D - 1) * (CA + CBW)>();
    Bases b0;
    if constexpr (SMALL) {
      step_bases(0, b0, 0, 3);
#pragma unroll
      for (int r = 0; r < 4 * (FIW + FJW); ++r) read_ahead(b0, 0, 0, r);
      const std::integral_constant<int, 0> even{};
      const std::integral_constant<int, 1> odd{};
      int s = 0;
      for (; (s + D + 2) * KD <= klen; s += 2) {
        small_step(s, even, std::integral_constant<int, 0>());
        small_step(s + 1, odd, std::integral_constant<int, 0>());
      }
      for (; s + 1 + D < nsteps; s += 2) {
        small_step(s, even, std::integral_constant<int, 1>());
        small_step(s + 1, odd, std::integral_constant<int, 1>());
      }
      if (s + D < nsteps) {
        small_step(s, even, std::integral_constant<int, 1>());
        ++s;
        for (; s < nsteps; s += 2) {
          small_step(s, odd, std::integral_constant<int, 2>());
          if (s + 1 < nsteps) small_step(s + 1, even, std::integral_constant<int, 2>());
        }
      } else {
        for (; s < nsteps; s += 2) {
          small_step(s, even, std::integral_constant<int, 2>());
          if (s + 1 < nsteps) small_step(s + 1, odd, std::integral_constant<int, 2>());
        }
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      return;
    }
    step_bases(0, b0, 0, 0);
#pragma unroll
    for (int f = 0; f < FJW; ++f) read_codes(b0, 0, f);
#pragma unroll
    for (int f = 0; f < FIW; ++f) {
      read_a(b0, 0, f, fa[0]);
      if (S4) sa[0][f] = read_scale(b0.sa, 0, f);
    }
#pragma unroll
    for (int f = 0; f < FJW; ++f) {
      read_b(b0, 0, f, fb[0]);
      if (S4) sb[0][f] = read_scale(b0.sb, 0, f);
    }
    int s = 0;
    for (; (s + D + 1) * KD <= klen; ++s) step_block(s, std::integral_constant<int, 0>());
    for (; s + D < nsteps; ++s) step_block(s, std::integral_constant<int, 1>());
    if constexpr (RING4)
      for (; s + 1 < nsteps; ++s) step_block(s, std::integral_constant<int, 3>());
    for (; s < nsteps; ++s) step_block(s, std::integral_constant<int, 2>());
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  };

  place(tl);
  prologue();
  if constexpr (DW) {
    main_loop();
    store_dw<FIW, FJW>(kernel_args(), acc, reinterpret_cast<char*>(&ring[0]), tl, w, lane);
  } else {
    // The grid is one workgroup per CU: each takes every gridDim.x-th tile and
    // starts the next one's copies before it stores this one's rows.
    char* const ct = reinterpret_cast<char*>(&ring[0]) + SPARE;
    // An epilogue phase: PR rows of GPR 16-byte granules; a store instruction
    // covers RPI of them, a wave stores PI times.
    constexpr int PR = WM == 2 ? 64 : 32, GPR = BN / 8, RPI = 64 / GPR, PI = PR / 4 / RPI;
    for (int b = blockIdx.x;;) {
      main_loop();
      b += gridDim.x;
      const Tile nx = rows_tile(b);
      int lane = threadIdx.x & 63;           // opaque, as in place
      asm volatile("" : "+v"(lane));
      const int half = lane >> 5, l32 = lane & 31;
      const ExpertArgs& g = kernel_args();
      // Phase p stores fragment row p of every wave.  Lane l holds the row of
      // C that the wave's l-th stored row goes to (or -1), loaded before the
      // copies (a load's use waits for every copy issued before it).
      const int lp = (lane / (PR / 4)) % FIW, lr = PR / 4 * w + lane % (PR / 4);
      const int lm = 32 * FIW * (lr >> 5) + 32 * lp + (lr & 31), ls = tl.row0 + min(lm, tl.mrows - 1);
      const int lv = g.mc.by_order ? g.order[ls] : ls;
      int orow = lm < tl.mrows && (unsigned)lv < (unsigned)g.rows ? lv : -1;
      asm volatile("" : "+v"(orow));
      __syncthreads();                       // every wave is past its last read of the ring
      const int n = tl.n0 + 8 * (lane % GPR);
      if (nx.mrows > 0) {
        place(nx);
        prologue();
      }
      // Granule c of row r at c ^ (r % GPR), so the rows a fragment writes and
      // the granules a row read takes both spread over the banks and every
      // store writes whole rows.
#pragma unroll
      for (int p = 0; p < FIW; ++p) {
        const int r = (WM == 2 ? 32 * (w >> 1) : 0) + l32;
#pragma unroll
        for (int fj = 0; fj < FJW; ++fj)
#pragma unroll
          for (int gg = 0; gg < 4; ++gg) {
            const int c = (wcol >> 3) + 4 * fj + gg;
            u32x2 pk;
            pk[0] = pack_bf16x2(acc[p][fj][4 * gg + 0], acc[p][fj][4 * gg + 1]);
            pk[1] = pack_bf16x2(acc[p][fj][4 * gg + 2], acc[p][fj][4 * gg + 3]);
            *reinterpret_cast<u32x2*>(ct + r * (2 * BN) + 16 * (c ^ (r % GPR)) + 8 * half) = pk;
          }
        lds_barrier();
#pragma unroll
        for (int it = 0; it < PI; ++it) {
          const int mr = PR / 4 * w + RPI * it + lane / GPR;
          const u32x4 x = *reinterpret_cast<const u32x4*>(ct + mr * (2 * BN) + 16 * ((lane % GPR) ^ (mr % GPR)));
          const int row = __shfl(orow, p * (PR / 4) + RPI * it + lane / GPR);
          if (row >= 0 && n < g.N)
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.C) + row * g.ldc + n) = x;
          __builtin_amdgcn_sched_barrier(0);
        }
        if (p + 1 < FIW) lds_barrier();
      }
      if (nx.mrows <= 0) break;
      tl = nx;
    }
  }
}


namespace {

// Pipelined kernel: at most one workgroup per CU (the ring takes its LDS),
// each walking the tiles.
template <int AL, int BL, int FI, int NJ>
void rows_pipe(const ExpertArgs& a, hipStream_t s) {
  const int64_t most = rows_grid(a, 64 * FI, 64 * NJ), grid = most < kCus ? most : kCus;
  hipLaunchKernelGGL((k_expert_pipe<AL, BL, FI, NJ, false, 0>), dim3((unsigned)grid), dim3(256), 0, s, a);
}
template <int BL, int FI, int NJ>
void rows_f32_tile(const ExpertArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_expert_f32<KC, BL, FI, NJ, false>), dim3((unsigned)rows_grid(a, 64 * FI, 64 * NJ)), dim3(256),
                     0, s, a);
}
}  // namespace

namespace {

template <int AL, int BL, int N>
void rows_bf16(ExpertForm form, bool b_kc, const Choice (&list)[N], double weight_bytes, const ExpertArgs& a,
               hipStream_t s) {
  const Choice& t = choose(list, false, a, weight_bytes);
  const int r = t.rows, c = t.cols;
  if (t.few) return launch_expert_few(form, b_kc, r, c, a, s);
  if (r == 64 && c == 128) return rows_pipe<AL, BL, 1, 2>(a, s);
  if (r == 64) return rows_pipe<AL, BL, 1, 4>(a, s);
  if (r == 128 && c == 128) return rows_pipe<AL, BL, 2, 2>(a, s);
  if (r == 128) return rows_pipe<AL, BL, 2, 4>(a, s);
  if constexpr (AL == KC)
    if (c == 128) return rows_pipe<AL, BL, 4, 2>(a, s);
  rows_pipe<AL, BL, 4, 4>(a, s);
}
template <int BL, int N>
void rows_f32(const Choice (&list)[N], bool b_kc, const ExpertArgs& a, hipStream_t s) {
  const Choice& t = choose(list, true, a, 4.0 * a.K * a.N);
  const int r = t.rows, c = t.cols;
  if (t.few) return launch_expert_few(ExpertForm::kF32, b_kc, r, c, a, s);
  if constexpr (BL == KC)     // (n-contiguous weights: the few-row kernel is faster wherever this tile would do)
    if (r == 64 && c == 64) return rows_f32_tile<BL, 1, 1>(a, s);
  if (r == 64 && c == 128) return rows_f32_tile<BL, 1, 2>(a, s);
  if (r == 64) return rows_f32_tile<BL, 1, 4>(a, s);
  if (r == 128 && c == 128) return rows_f32_tile<BL, 2, 2>(a, s);
  if (r == 128) return rows_f32_tile<BL, 2, 4>(a, s);
  rows_f32_tile<BL, 4, 4>(a, s);
}

}  // namespace

void launch_expert_rows(ExpertForm form, bool b_kc, const ExpertArgs& a, hipStream_t s) {
  if (a.rows <= 0) return;
  const double elems = (double)a.K * a.N;
  switch (form) {
    case ExpertForm::kBf16:
      if (b_kc) rows_bf16<KC, KC>(form, true, kBf16Nk, 2 * elems, a, s);
      else rows_bf16<KC, NC>(form, false, kBf16Kn, 2 * elems, a, s);
      break;
    case ExpertForm::kF32:
      if (b_kc) rows_f32<KC>(kF32Nk, true, a, s);
      else rows_f32<NC>(kF32Kn, false, a, s);
      break;
    case ExpertForm::kW4A16: rows_bf16<KC, F4>(form, true, kW4A16, elems * 17 / 32, a, s); break;
    case ExpertForm::kW4A4:
      if (a.K % 512 == 0) rows_bf16<X4, X4>(form, true, kW4A4, elems * 17 / 32, a, s);
      else rows_bf16<X4D, X4D>(form, true, kW4A4, elems * 17 / 32, a, s);
      break;
  }
}

namespace {

// dW of the groups with several chunks: their sums added in order.
__global__ __launch_bounds__(256) void k_expert_dw_sum(ExpertArgs a, int pieces) {
  const int e = blockIdx.x / pieces, piece = blockIdx.x - e * pieces;
  int many, first;
  DwChunks(a).of_group(a, e, many, first);
  if (many <= 1) return;
  const int64_t n = a.c_expert / 4;              // vectors of four (M or N is a multiple of 4)
  const f32x4* part = reinterpret_cast<const f32x4*>(a.part + (int64_t)first * a.c_expert);
  f32x4* out = reinterpret_cast<f32x4*>(static_cast<float*>(a.C) + (int64_t)e * a.c_expert);
  const int64_t i = (int64_t)piece * 256 + threadIdx.x;
  if (i >= n) return;
  f32x4 sum = part[i];
  int c = 1;
  for (; c + 3 < many; c += 4) {   // four loads in flight, added in order
    const f32x4 v0 = part[c * n + i], v1 = part[(c + 1) * n + i], v2 = part[(c + 2) * n + i], v3 = part[(c + 3) * n + i];
    sum = (((sum + v0) + v1) + v2) + v3;
  }
  for (; c < many; ++c) sum += part[c * n + i];
  if (a.accumulate) sum += out[i];
  out[i] = sum;
}

template <int BM>
int64_t dw_grid(const ExpertArgs& a) {
  const int64_t E = a.offsets ? a.n_experts : 1;
  const int64_t tt = (int64_t)((a.M + BM - 1) / BM) * ((a.N + BM - 1) / BM);
  if (a.chunk > 0) return ((a.rows / a.chunk + E) * tt + 7) / 8 * 8;
  return 8 * E * ((tt + 7) / 8);
}
template <int FI>
void dw_pipe(const ExpertArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)dw_grid<64 * FI>(a));
  switch ((a.ma.by_order ? 1 : 0) + (a.mb.by_order ? 2 : 0)) {
    case 0: hipLaunchKernelGGL((k_expert_pipe<NC, NC, FI, FI, true, 0>), grid, dim3(256), 0, s, a); break;
    case 1: hipLaunchKernelGGL((k_expert_pipe<NC, NC, FI, FI, true, 1>), grid, dim3(256), 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_expert_pipe<NC, NC, FI, FI, true, 2>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((k_expert_pipe<NC, NC, FI, FI, true, 3>), grid, dim3(256), 0, s, a);
  }
}
template <int FI>
void dw_f32(const ExpertArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_expert_f32<NC, NC, FI, FI, true>), dim3((unsigned)dw_grid<64 * FI>(a)), dim3(256), 0, s, a);
}

}  // namespace

void launch_expert_dw(bool f32, const ExpertArgs& a, hipStream_t s) {
  const int64_t E = a.offsets ? a.n_experts : 1;
  const int tile = dw_tile(f32, E, a.M, a.N);
  if (f32) {
    if (tile == 256) dw_f32<4>(a, s);
    else if (tile == 128) dw_f32<2>(a, s);
    else dw_f32<1>(a, s);
  } else {
    if (tile == 256) dw_pipe<4>(a, s);
    else dw_pipe<2>(a, s);
  }
  if (a.chunk > 0) {
    const int64_t blocks = (a.c_expert / 4 + 255) / 256;
    hipLaunchKernelGGL(k_expert_dw_sum, dim3((unsigned)(E * blocks)), dim3(256), 0, s, a, (int)blocks);
  }
}

}  // namespace mlora
