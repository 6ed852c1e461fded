// Which form a product with 4-bit codes takes, on the host, from sizes alone.
#pragma once

#include "affine.hpp"

namespace mlora {

// Workgroups that rows of at most `n_experts` groups in tiles of bm rows and bn
// columns can make.
inline int64_t rows_grid_of(const ExpertArgs& a, int bm, int bn) {
  const int64_t groups = a.offsets ? a.n_experts : 1;
  return (a.rows / bm + (groups < a.rows ? groups : a.rows)) * ((a.N + bn - 1) / bn);
}

// Rows a group has if they are spread evenly.
inline double affine_few_rows(const ExpertArgs& a) {
  const double groups = a.offsets ? (a.n_experts < a.rows ? a.n_experts : a.rows) : 1;
  return a.rows / groups;
}

// Rows a group up to which the codes are multiplied as they are; above, the
// weights are decoded to bf16 first.
constexpr double kAffineFew = 64;

}  // namespace mlora
