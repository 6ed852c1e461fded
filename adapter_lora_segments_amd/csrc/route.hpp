// Launch interface of routing and combining (host side).  Launchers check
// nothing: the C interface (api_route.cpp) validates sizes before calling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mlora.h"

namespace mlora {

struct RouteArgs {
  const void* logits;           // [rows][ld] bf16 or fp32
  int64_t rows, ld;
  const float* bias;            // [n_experts] or NULL (forward)
  int32_t* ids;                 // [rows][top_k], written by the forward, read by the backward
  float* weights;               // [rows][top_k] (forward)
  const float* dweights;        // [rows][top_k] (backward)
  void* dlogits;                // [rows][n_experts] of the logits' type (backward)
  int32_t E, k, n_groups, per_group, top_groups;
  int32_t sigmoid, top2, renorm;
  float scale;
};

void launch_route(bool f32, const RouteArgs& a, hipStream_t s);
void launch_route_backward(bool f32, const RouteArgs& a, hipStream_t s);

struct CombineArgs {
  const void* Y;                // [tokens * k][d]
  const int32_t* ids;           // [tokens][k] or NULL: every slot counts
  const float* weights;         // [tokens][k] or NULL: 1
  const void* add;              // [tokens][d] or NULL
  void* out;                    // [tokens][d] (forward)
  const void* dout;             // [tokens][d] (backward)
  void* dY;                     // [tokens * k][d] or NULL
  float* dweights;              // [tokens][k] or NULL
  int64_t tokens;
  int32_t k, d;
  uint32_t limit;               // slots whose id is below it count
};

void launch_combine(bool f32, const CombineArgs& a, hipStream_t s);
void launch_combine_backward(bool f32, const CombineArgs& a, hipStream_t s);

}  // namespace mlora
