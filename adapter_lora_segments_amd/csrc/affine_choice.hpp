// Which kernel and tile a product over 4-bit weights takes, on the host, from
// sizes alone.
#pragma once

#include <cmath>

#include "affine.hpp"

namespace mlora {

// Workgroups that rows of at most `n_experts` groups in tiles of bm rows and bn
// columns can make.
inline int64_t affine_grid(const ExpertArgs& a, int bm, int bn) {
  const int64_t groups = a.offsets ? a.n_experts : 1;
  return (a.rows / bm + (groups < a.rows ? groups : a.rows)) * ((a.N + bn - 1) / bn);
}

// Rows a group has if they are spread evenly over the groups (all of them, or
// as many as there are rows).
inline double affine_rows(const ExpertArgs& a) {
  const double groups = a.offsets ? (a.n_experts < a.rows ? a.n_experts : a.rows) : 1;
  return a.rows / groups;
}

// Up to this many rows a group the codes are multiplied as they are: a step of
// decoding has a full fragment of rows at best.
constexpr double kAffineExact = 16;

// From this many rows a group on, the weights are decoded to bf16 in memory
// first and the bf16 product runs over them: 2.5 bytes a weight once more,
// against tiles that decode on the way at 0.7 of its rate.  Measured (us,
// decoded first and in tiles): 1024 rows, 4096 -> 14336 128 and 136; 512 rows,
// 4096 -> 4096 43 and 27; 2048 rows over 8 experts, 4096 -> 4096 175 and 76;
// 8192 rows, 4096 -> 14336 766 and 1050; dX of 1024 rows 163 and 163, of 2048
// rows 227 and 281, of 2048 rows over 8 experts of 4096 x 4096 176 and 88.
constexpr int64_t kAffineDecoded = 1024;

// A tile of rows x cols: of the few-row kernel (split: waves side by side, the
// others share the reduction) or of the tiled one (split: parts of the
// reduction).  Times as in expert_choice.hpp: start + K max(lone, busy rounds),
// at least that of reading the weights, `lone` being the time per input of a
// tile on a CU of its own and `busy` that of a tile on a full chip.  Fitted to
// sweeps (us; K = 4096): 1 row, N = 14336 10.2 with 4 x 16 tiles, 10.0 with 4 x
// 32 and N = 1024 4.9 and 6.2; 8 rows, N = 14336 13.2 (8 x 16), 11.2 (8 x 32);
// 16 rows 21.8 (16 x 16), 13.9 (16 x 32), 12.5 (16 x 64), and N = 1024 6.0, 7.9,
// 10.2; 32 rows 21.6 (32 x 32), 16.0 (32 x 64), 21.8 (32 x 128); 8 experts of 32
// rows, N = 4096 48, 35, 27, of 64 rows 31 (64 x 128), 42 (32 x 128), of 256
// rows 93 (64 x 128), 77 (128 x 128); 64 rows, N = 14336 33 and, in two parts,
// 25 (64 x 128).
struct AffineChoice {
  bool few;
  int rows, cols, split;
  double start, lone, busy, rate;
};
constexpr AffineChoice kAffine[] = {
    {true, 4, 16, 1, 3.0, .00046, .00045, 5.1e6},  {true, 8, 16, 1, 3.0, .00056, .00072, 4.6e6},
    {true, 8, 32, 1, 3.0, .00085, .00117, 4.6e6},  {true, 16, 16, 1, 3.0, .00072, .00131, 4.0e6},
    {true, 16, 32, 2, 3.0, .00120, .00147, 4.2e6}, {true, 16, 64, 2, 3.0, .00180, .00233, 4.2e6},
    {true, 32, 32, 2, 3.0, .00176, .00265, 3.4e6}, {true, 32, 64, 2, 3.0, .00270, .00350, 3.4e6},
    {true, 32, 128, 4, 3.0, .00450, .00480, 3.4e6},
    {false, 64, 128, 1, 3.0, .00700, .00550, 3.0e6},  {false, 64, 128, 2, 3.5, .00560, .00610, 3.0e6},
    {false, 128, 128, 1, 3.0, .00990, .00920, 3.0e6}, {false, 128, 128, 2, 3.5, .00800, .00980, 3.0e6}};

// The same for dX, whose tiled kernel has them all.  K = 4096, N = 4096 (us;
// 32, 64 and 128 rows): 256 rows 29, 35, 49; 512 rows over 8 experts 46, 38, 53;
// 2048 rows over 8 153, 107, 89; 8192 rows 596, 398, 330.
constexpr AffineChoice kAffineDx[] = {{false, 32, 128, 2, 3.0, .00560, .00500, 3.0e6},
                                      {false, 64, 128, 1, 3.0, .00820, .00640, 3.0e6},
                                      {false, 128, 128, 1, 3.0, .01130, .01000, 3.0e6}};

inline double affine_us(const AffineChoice& c, const ExpertArgs& a, double weight_bytes) {
  double groups = 1;
  if (a.offsets && a.n_experts > 1) groups = a.n_experts * (1 - std::pow(1.0 - 1.0 / a.n_experts, a.rows));
  const double mean = a.rows / groups;
  double tiles = groups == 1 ? (a.rows + c.rows - 1) / c.rows : mean / c.rows + 0.5;
  if (tiles < 1) tiles = 1;
  const double rounds = groups * tiles * ((a.N + c.cols - 1) / c.cols) / 256.0;
  const double busy = c.busy * rounds;
  const double us = c.start + a.K * (c.lone > busy ? c.lone : busy);
  const double fill = 0.5 + 0.75 * rounds;        // fewer workgroups than CUs do not reach the full rate
  const double read = c.start + groups * weight_bytes / (c.rate * (fill < 1 ? fill : 1));
  return us > read ? us : read;
}

// (The few-row kernel's last entry and the list's last one always fit a launch.)
template <int N>
const AffineChoice& affine_choose(const AffineChoice (&list)[N], const ExpertArgs& a, int32_t group) {
  const double bytes = (double)a.K * a.N * (0.5 + 4.0 / group);
  const bool exact = list[0].few && affine_rows(a) <= kAffineExact;
  int best = -1;
  double best_us = 0;
  for (int i = 0; i < N; ++i) {
    const AffineChoice& c = list[i];
    const bool last = exact ? c.few && !list[i + 1].few : i + 1 == N;
    if ((exact && !c.few) || (!last && affine_grid(a, c.rows, c.cols) > kMaxGrid)) continue;
    const double us = affine_us(c, a, bytes);
    if (best < 0 || us < best_us) {
      best = i;
      best_us = us;
    }
  }
  return list[best];
}

}  // namespace mlora
