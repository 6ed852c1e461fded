// Which kernel and tile a grouped product takes, on the host, from sizes and
// types alone.
#pragma once

#include <cmath>

#include "experts.hpp"

namespace mlora {

// Largest number of row tiles that `rows` rows in at most `experts` groups
// can make.
inline int64_t max_row_tiles(int64_t rows, int64_t experts, int bm) {
  return rows / bm + (experts < rows ? experts : rows);
}

inline int64_t rows_grid(const ExpertArgs& a, int bm, int bn) {
  return max_row_tiles(a.rows, a.offsets ? a.n_experts : 1, bm) * ((a.N + bn - 1) / bn);
}
constexpr int64_t kCus = 256;

// Which kernel and tile a product takes.  Its time is predicted for each as
//   start + K max(lone * ceil(rounds), busy * rounds),  at least the time that
// reading the weights takes, with rounds = tiles / 256 CUs: `lone` is a tile's
// time per element of the reduction while it has its CU and the caches to
// itself, `busy` the same when the chip is full (clocks drop, the L2s are
// shared).  The few-row kernel has several workgroups on a CU: no ceil.  The
// groups' sizes are not known here: the number of groups with rows is that of
// rows thrown at the groups evenly, and a group has half a partial tile.
// Measured with groups of equal size (us; K = 4096): bf16 weights
// [d_out][d_in], N = 4096: one expert of 4 rows 9.2 with 16x16 few-row tiles,
// 24 with 64x128 and 78 with 256x256 tiles; of 160 rows 57, 25 and 80; of 2048
// rows 104 (64x128), 64 (256x128), 89 (256x256); eight of 2048 rows 969, 538,
// 462.  MXFP4 weights, bf16 activations, N = 14336: 4 rows 17.1 (16x16), 13.8
// (16x32), 12.4 (16x64), 27 (64x128); eight experts of 32 rows 152 (16x64), 88
// (64x256).  fp32, N = 4096: 48 rows 37 (64x16 few-row), 97 (64x64); 512 rows
// 285 and 160; 2048 rows 618 (64x64), 527 (128x256).
struct Choice {
  bool few;
  int rows, cols;               // tile
  double start, lone, busy;     // us, us per element of the reduction
  double rate;                  // bytes of weights per us
};
constexpr Choice kBf16Nk[] = {{true, 16, 16, 3.0, .0015, .0016, 5.2e6},   {true, 16, 32, 3.0, .0024, .0029, 5.0e6},
                              {true, 32, 16, 3.0, .0028, .0026, 4.3e6},   {true, 32, 32, 3.0, .0036, .0042, 4.6e6},
                              {true, 32, 64, 3.0, .0054, .0076, 4.6e6},   {true, 64, 32, 3.0, .0055, .0061, 3.8e6},
                              {false, 64, 128, 4.5, .0048, .0074, 4.2e6}, {false, 64, 256, 4.9, .0070, .0121, 5.4e6},
                              {false, 128, 128, 6.0, .0059, .0104, 4.2e6}, {false, 128, 256, 6.9, .0100, .0181, 5.5e6},
                              {false, 256, 128, 6.8, .0092, .0164, 4.1e6}, {false, 256, 256, 10.0, .0166, .0281, 5.0e6}};
constexpr Choice kBf16Kn[] = {{true, 16, 64, 3.0, .0027, .0049, 5.0e6},   {true, 32, 64, 3.0, .0030, .0053, 5.1e6},
                              {true, 64, 64, 3.0, .0037, .0095, 5.0e6},   {false, 64, 128, 5.0, .0048, .0076, 4.8e6},
                              {false, 64, 256, 5.5, .0073, .0121, 5.2e6}, {false, 128, 128, 6.0, .0063, .0106, 4.8e6},
                              {false, 128, 256, 7.0, .0104, .0186, 5.2e6}, {false, 256, 128, 6.8, .0095, .0162, 4.2e6},
                              {false, 256, 256, 10.0, .0175, .0286, 4.6e6}};
constexpr Choice kF32Nk[] = {{true, 16, 16, 3.0, .0040, .0048, 4.7e6},   {true, 16, 32, 3.0, .0052, .0078, 5.2e6},
                             {true, 32, 16, 3.0, .0058, .0063, 4.3e6},   {true, 32, 32, 3.0, .0080, .0098, 4.8e6},
                             {true, 64, 32, 3.0, .0130, .0134, 3.2e6},   {false, 64, 64, 3.5, .0231, .0185, 4.0e6},
                             {false, 64, 128, 3.7, .0389, .0353, 4.0e6}, {false, 64, 256, 4.0, .0686, .0708, 4.0e6},
                             {false, 128, 128, 3.8, .0675, .0647, 4.0e6}, {false, 128, 256, 4.1, .1247, .1285, 4.0e6},
                             {false, 256, 256, 5.0, .2350, .2500, 4.0e6}};
constexpr Choice kF32Kn[] = {{true, 16, 64, 3.0, .0080, .0094, 5.2e6},   {true, 32, 64, 3.0, .0118, .0111, 5.0e6},
                             {true, 64, 64, 3.0, .0190, .0206, 3.0e6},
                             {false, 64, 128, 3.7, .0389, .0353, 4.5e6}, {false, 64, 256, 4.0, .0686, .0708, 4.5e6},
                             {false, 128, 128, 3.8, .0675, .0647, 4.5e6}, {false, 128, 256, 4.1, .1247, .1285, 4.5e6},
                             {false, 256, 256, 5.0, .2350, .2500, 4.5e6}};
constexpr Choice kW4A16[] = {{true, 16, 16, 3.2, .0011, .0013, 2.6e6},   {true, 16, 32, 3.2, .0016, .0018, 3.3e6},
                             {true, 16, 64, 3.2, .0024, .0029, 3.7e6},   {true, 32, 32, 3.2, .0026, .0029, 2.8e6},
                             {true, 32, 64, 3.2, .0036, .0044, 2.9e6},   {false, 64, 128, 4.8, .0046, .0081, 2.3e6},
                             {false, 64, 256, 5.8, .0062, .0115, 3.1e6}, {false, 128, 128, 5.2, .0069, .0100, 2.2e6},
                             {false, 128, 256, 7.1, .0101, .0155, 2.6e6}, {false, 256, 128, 6.9, .0098, .0160, 1.5e6},
                             {false, 256, 256, 10.1, .0170, .0270, 1.8e6}};
constexpr Choice kW4A4[] = {{true, 16, 16, 3.2, .0007, .0010, 2.9e6},   {true, 16, 32, 3.2, .0011, .0013, 3.8e6},
                            {true, 16, 64, 3.2, .0021, .0025, 3.4e6},   {true, 32, 32, 3.2, .0017, .0019, 3.4e6},
                            {true, 32, 64, 3.2, .0026, .0033, 3.2e6},   {false, 64, 128, 4.1, .0020, .0030, 4.6e6},
                            {false, 64, 256, 4.2, .0029, .0045, 5.6e6}, {false, 128, 128, 4.2, .0024, .0039, 4.4e6},
                            {false, 128, 256, 5.4, .0037, .0069, 5.0e6}, {false, 256, 256, 8.0, .0055, .0121, 3.7e6}};

// (fixed: one workgroup per tile also in the tiled kernel; the last entry's grid
// always fits a launch.)
template <int N>
const Choice& choose(const Choice (&list)[N], bool fixed, const ExpertArgs& a, double weight_bytes) {
  double groups = 1;
  if (a.offsets && a.n_experts > 1) {
    // less the chance that a group gets none of the rows
    groups = a.n_experts * (1 - std::pow(1.0 - 1.0 / a.n_experts, a.rows));
  }
  const double mean = a.rows / groups;
  int best = -1;
  double best_us = 0;
  for (int i = 0; i < N; ++i) {
    const Choice& c = list[i];
    if ((c.few || fixed) && i + 1 < N && rows_grid(a, c.rows, c.cols) > kMaxGrid) continue;
    double tiles = groups == 1 ? (a.rows + c.rows - 1) / c.rows : mean / c.rows + 0.5;
    if (tiles < 1) tiles = 1;
    const double rounds = groups * tiles * ((a.N + c.cols - 1) / c.cols) / kCus;
    const double lone = c.few ? c.lone : c.lone * (double)(int64_t)(rounds + 0.999), busy = c.busy * rounds;
    double us = c.start + a.K * (lone > busy ? lone : busy);
    // fewer workgroups than CUs do not reach the full rate
    const double fill = 0.5 + 0.75 * rounds;
    const double read = c.start + groups * weight_bytes / (c.rate * (fill < 1 ? fill : 1));
    if (read > us) us = read;
    if (best < 0 || us < best_us) {
      best = i;
      best_us = us;
    }
  }
  return list[best];
}

// dW tiles.  A group's sizes are not known here, and one workgroup sums all of a
// group's rows: the longest group sets a lower bound, which small tiles keep
// low.  bf16: 256 x 256 where they fill the chip, one expert has 32 of them and
// they are not mostly padding, else 128 x 128; fp32: 256 x 256 or 128 x 128
// where one expert's nearly fill the chip, else 64 x 64.  Measured (us): bf16
// 8 x 512 x 1024, 100 rows each 17.0 (256) and 9.6 (128); 8 x 2048 x 2048, 1000
// rows each 82 and 118; 64 x 512 x 1024, 32000 skewed rows 167 and 96 (but 32 x
// 1000 rows 52 and 77).  fp32 (256, 128, 64): 16 x 832 x 2212, 2000 skewed rows
// 177, 102, 99; 2048 x 2048, 1000 rows 266, 86, 94; 8 of them 539, 558, 633;
// 32 x 4096 x 4096, 100 rows each 1423, 1543, 1587.
inline int dw_tile(bool f32, int64_t E, int64_t M, int64_t N) {
  const int64_t t256 = ((M + 255) / 256) * ((N + 255) / 256), t128 = dw_tiles128(M, N);
  const bool padded = 8 * t256 > 3 * t128 && E * t128 < kMaxGrid / 2;      // over 1.5 times the area
  if (f32) return t256 >= 256 && !padded ? 256 : t128 >= 192 ? 128 : 64;
  return E * t256 >= 160 && t256 >= 32 && !padded ? 256 : 128;
}

}  // namespace mlora
