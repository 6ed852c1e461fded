// Launch interface of the grouped expert products, the row grouping and the
// MXFP4 quantizer (host side).  As in kernels.hpp, launchers check nothing:
// the C interface validates shapes and sizes before calling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string>

#include "../../include/mlora.h"

namespace mlora {

// The message mlora_last_error() returns on this thread (api.cpp).
void set_last_error(const std::string& msg);

// ---------------- row grouping ----------------

// Rows per workgroup of the two-kernel form and its number of workgroups:
// at most kGroupMaxParts parts, so every workgroup can sum the parts' counts
// before its own by itself.
constexpr int64_t kGroupMinPart = 4096;
constexpr int64_t kGroupMaxParts = 256;
// Rows up to which one workgroup does everything in one launch.
constexpr int64_t kGroupOneLaunch = 8192;
inline int64_t group_part_rows(int64_t rows) {
  const int64_t even = (rows + kGroupMaxParts - 1) / kGroupMaxParts;
  return even > kGroupMinPart ? (even + 1023) / 1024 * 1024 : kGroupMinPart;
}
// counts: [parts][n_groups] ints of workspace (unused by the one-launch form).
void launch_group_rows(const int32_t* ids, int64_t rows, int32_t n_groups, int32_t* offsets, int32_t* order,
                       int32_t* counts, hipStream_t s);

// ---------------- MXFP4 quantizer ----------------

// codes [rows][cols / 2]; scales [rows][cols / 32], or [cols][rows / 32] with
// down; values NULL or [rows][cols] of X's type.
void launch_quant_mx4(bool f32, bool down, const void* X, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                      uint8_t* scales, void* values, hipStream_t s);

// ---------------- grouped products ----------------

// Unsigned division of values below 2^31 by a fixed divisor: n / d =
// umulhi(n, mul) >> shift (d > 1), n for d = 1 (mul = 0).
struct DivBy {
  uint32_t mul;
  int32_t shift;
};
inline DivBy div_by(int32_t d) {
  if (d <= 1) return {0u, 0};
  int l = 0;
  while ((1 << l) < d) ++l;                                  // ceil(log2 d)
  const uint64_t m = ((uint64_t)1 << (31 + l)) / (uint64_t)d + 1;
  return {(uint32_t)m, l - 1};
}

// How the rows of an operand or output lie: grouped row s at row s, or at
// order[s] / top_k.
struct RowMap {
  int32_t by_order;
  DivBy div;
};

// One product over all experts.
//   rows form (forward, dX): C[rc(s)][n] = sum_k A[ra(s)][k] B_e(k, n)
//   dW form: C_e[m][n] = sum_s A[ra(s)][m] B[rb(s)][n] (fp32 C)
struct ExpertArgs {
  const uint8_t* A;
  const uint8_t* B;
  int64_t lda, ldb, ldc;        // row strides in elements of the operand's format
  int64_t b_expert;             // bytes from one expert's B to the next (rows form)
  int64_t c_expert;             // elements from one expert's C to the next (dW form)
  void* C;
  RowMap ma, mb, mc;
  const int32_t* offsets;       // NULL: one expert over all rows
  const int32_t* order;
  int32_t rows, n_experts;
  int32_t M, N, K;              // dW form: M x N outputs per expert; rows form: N, K
  const uint8_t* a_scale;       // MXFP4 scale codes of A [..][K / 32], B [N][K / 32] per expert
  const uint8_t* b_scale;
  int32_t accumulate;           // dW form: add to C
  int32_t chunk;                // dW form: rows of a group summed by one workgroup, 0: all
  float* part;                  // sums of the chunks of groups that have several, [slot][M][N]
};

// Pieces of at most c > 0 rows that n >= 0 rows make.  (n + c - 1) / c would
// wrap: a dW chunk takes up to 2^23 of up to 2^31 - 257 rows.
constexpr int pieces_of(int n, int c) { return n > 0 ? (n - 1) / c + 1 : 0; }

// Workgroups of a launch: their threads (512 each at most) fit 32 bits.
constexpr int64_t kMaxGrid = ((int64_t)1 << 23) - 1;

// Rows a dW chunk takes, 0 for no chunks: where the 128 x 128 tiles of all
// experts do not fill the 256 CUs, long groups are cut into pieces that would,
// of at least 1024 rows (bf16) or 256 (fp32): a piece's partial sums are
// written and read once, 2 x 64 KiB a tile, so more or shorter pieces cost more
// than they spread.  Measured (us, uncut and cut, one expert): bf16 136 x 864,
// 4000 rows 30 and 17, 16000 rows 100 and 21; 512 x 1024, 16000 rows 100 and
// 31; 2048 x 2048 (256 tiles), 4000 rows 41 and 78 with pieces of 1024.  fp32
// 136 x 864, 1000 rows 29 and 15, 16000 rows 404 and 73; 512 x 1024 over 16
// experts (512 tiles), 8000 skewed rows 116 and 140 with pieces of 256.
inline int64_t dw_tiles128(int64_t m, int64_t n) { return ((m + 127) / 128) * ((n + 127) / 128); }
inline int64_t dw_least(bool f32) { return f32 ? 256 : 1024; }
inline int64_t dw_chunk(bool f32, int64_t rows, int64_t experts, int64_t m, int64_t n) {
  const int64_t t = dw_tiles128(m, n);
  if (experts * t >= 256) return 0;
  const int64_t even = ((rows * t + 255) / 256 + 63) / 64 * 64, c = even > dw_least(f32) ? even : dw_least(f32);
  return rows > c ? c : 0;
}
// Bytes of the partial sums of at most `rows` rows: a group of more than one
// chunk of c rows has at most 2 / c chunks a row.
inline int64_t dw_part_bytes(bool f32, int64_t rows, int64_t experts, int64_t m, int64_t n) {
  const int64_t t = dw_tiles128(m, n);
  if (experts * t >= 256 || rows <= dw_least(f32)) return 0;
  const int64_t a = 2 * rows / dw_least(f32), b = 512 / t;
  return (a < b ? a : b) * m * n * 4;
}

enum class ExpertForm { kBf16, kF32, kW4A16, kW4A4 };

// rows form; b_kc: B_e(k, n) at B[n * ldb + k], else at B[k * ldb + n]
// (MXFP4 weights are always k-contiguous).
void launch_expert_rows(ExpertForm form, bool b_kc, const ExpertArgs& a, hipStream_t s);
// The same for few rows per group, in one of the tiles of rows x cols that
// expert_choice.hpp chooses from.
void launch_expert_few(ExpertForm form, bool b_kc, int rows, int cols, const ExpertArgs& a, hipStream_t s);
// dW form, bf16 or fp32 operands, both n-contiguous; with a.chunk a second
// kernel adds the chunks of a group in order.
void launch_expert_dw(bool f32, const ExpertArgs& a, hipStream_t s);

}  // namespace mlora
