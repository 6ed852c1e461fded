// C interface of routing and combining (include/mlora.h): argument checks and
// launches.  Host state: none; device state: the caller's buffers.
#include <hip/hip_runtime.h>

#include "../../include/mlora.h"
#include "api_common.hpp"
#include "route.hpp"

namespace {

using mlora::api_aligned;
using mlora::api_fail;
using mlora::api_launched;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
// workgroups of a launch: their 256 threads fit 32 bits
constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;

// Message of the first thing wrong with a router or a call's sizes, or NULL.
const char* router_error(const mlora_router* r, mlora_dtype dtype, int64_t rows, int64_t ld, mlora_status* st) {
  *st = MLORA_ERR_INVALID_ARG;
  if (!r) return "route: router is NULL";
  if (r->n_experts < 1 || r->n_experts > MLORA_MAX_EXPERTS) return "route: n_experts must be in [1, 4096]";
  if (r->score != MLORA_SCORE_SOFTMAX && r->score != MLORA_SCORE_SIGMOID) return "route: unknown score";
  if (r->expert_groups < 1 || r->expert_groups > 64 || r->n_experts % r->expert_groups)
    return "route: expert_groups must be in [1, 64] and divide n_experts";
  if (r->top_groups < 1 || r->top_groups > r->expert_groups) return "route: top_groups must be in [1, expert_groups]";
  if (r->group_score != MLORA_GROUP_MAX && r->group_score != MLORA_GROUP_TOP2) return "route: unknown group_score";
  if (r->top_k < 1 || r->top_k > 64 || r->top_k > r->n_experts / r->expert_groups * r->top_groups)
    return "route: top_k must be in [1, 64] and at most the experts of top_groups groups";
  if (r->renormalize != 0 && r->renormalize != 1) return "route: renormalize is 0 or 1";
  if (dtype != MLORA_BF16 && dtype != MLORA_FP32) return "route: unknown dtype";
  if (rows < 0 || rows > kMaxRows) return "route: rows must be in [0, 2^31)";
  if (ld < r->n_experts) return "route: ld must be at least n_experts";
  *st = MLORA_ERR_UNSUPPORTED;
  // as few as one row a workgroup with many experts
  if (rows > kMaxGrid * (r->n_experts > 1024 ? 1 : 4)) return "route: too many rows for one launch";
  *st = MLORA_OK;
  return nullptr;
}

mlora::RouteArgs router_args(const mlora_router& r, const void* logits, int64_t rows, int64_t ld) {
  mlora::RouteArgs a{};
  a.logits = logits;
  a.rows = rows;
  a.ld = ld;
  a.E = r.n_experts;
  a.k = r.top_k;
  a.n_groups = r.top_groups < r.expert_groups ? r.expert_groups : 1;     // all groups: no choice among them
  a.per_group = r.n_experts / r.expert_groups;
  a.top_groups = r.top_groups;
  a.sigmoid = r.score == MLORA_SCORE_SIGMOID;
  a.top2 = r.group_score == MLORA_GROUP_TOP2;
  a.renorm = r.renormalize;
  a.scale = r.scale;
  return a;
}

const char* combine_error(mlora_dtype dtype, int64_t tokens, int32_t top_k, int64_t d, int32_t n_experts, mlora_status* st) {
  *st = MLORA_ERR_INVALID_ARG;
  if (dtype != MLORA_BF16 && dtype != MLORA_FP32) return "combine: unknown dtype";
  if (top_k < 1 || top_k > 64) return "combine: top_k must be in [1, 64]";
  if (tokens < 0 || tokens > kMaxRows / top_k) return "combine: tokens * top_k must be in [0, 2^31)";
  if (d <= 0 || d % (dtype == MLORA_BF16 ? 8 : 4))
    return "combine: d must be a positive multiple of 8 (bf16) or 4 (fp32)";
  if (n_experts < 0) return "combine: n_experts must be 0 (any) or positive";
  *st = MLORA_ERR_UNSUPPORTED;
  if (d > MLORA_MAX_EXPERT_DIM) return "combine: d is at most 2^20";
  const int64_t split = (d / (dtype == MLORA_BF16 ? 8 : 4) + 255) / 256;
  if (tokens > kMaxGrid / split) return "combine: too many tokens for one launch";
  *st = MLORA_OK;
  return nullptr;
}

}  // namespace

extern "C" {

mlora_status mlora_route(const mlora_router* router, const void* logits, mlora_dtype dtype, int64_t rows, int64_t ld,
                         const float* bias, int32_t* ids, float* weights, void* stream) {
  mlora_status st;
  if (const char* msg = router_error(router, dtype, rows, ld, &st)) return api_fail(st, msg);
  if (rows == 0) return MLORA_OK;
  if (!logits || !ids || !weights) return api_fail(MLORA_ERR_INVALID_ARG, "route: logits, ids and weights must be non-NULL");
  if (!api_aligned(logits, dtype == MLORA_BF16 ? 2 : 4) || !api_aligned(bias, 4) || !api_aligned(ids, 4) ||
      !api_aligned(weights, 4))
    return api_fail(MLORA_ERR_INVALID_ARG, "route: pointers must be aligned to their elements");
  mlora::RouteArgs a = router_args(*router, logits, rows, ld);
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  mlora::launch_route(dtype == MLORA_FP32, a, static_cast<hipStream_t>(stream));
  return api_launched();
}

mlora_status mlora_route_backward(const mlora_router* router, const void* logits, mlora_dtype dtype, int64_t rows,
                                  int64_t ld, const int32_t* ids, const float* dweights, void* dlogits, void* stream) {
  mlora_status st;
  if (const char* msg = router_error(router, dtype, rows, ld, &st)) return api_fail(st, msg);
  if (rows == 0) return MLORA_OK;
  if (!logits || !ids || !dweights || !dlogits)
    return api_fail(MLORA_ERR_INVALID_ARG, "route backward: logits, ids, dweights and dlogits must be non-NULL");
  const uintptr_t unit = dtype == MLORA_BF16 ? 2 : 4;
  if (!api_aligned(logits, unit) || !api_aligned(dlogits, unit) || !api_aligned(ids, 4) || !api_aligned(dweights, 4))
    return api_fail(MLORA_ERR_INVALID_ARG, "route backward: pointers must be aligned to their elements");
  mlora::RouteArgs a = router_args(*router, logits, rows, ld);
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  mlora::launch_route_backward(dtype == MLORA_FP32, a, static_cast<hipStream_t>(stream));
  return api_launched();
}

mlora_status mlora_combine(const void* Y, mlora_dtype dtype, int64_t tokens, int32_t top_k, int64_t d,
                           const int32_t* ids, int32_t n_experts, const float* weights, const void* add, void* out,
                           void* stream) {
  mlora_status st;
  if (const char* msg = combine_error(dtype, tokens, top_k, d, n_experts, &st)) return api_fail(st, msg);
  if (tokens == 0) return MLORA_OK;
  if (!Y || !out) return api_fail(MLORA_ERR_INVALID_ARG, "combine: Y and out must be non-NULL");
  if (!api_aligned(Y, 16) || !api_aligned(add, 16) || !api_aligned(out, 16) || !api_aligned(ids, 4) ||
      !api_aligned(weights, 4))
    return api_fail(MLORA_ERR_INVALID_ARG, "combine: Y, add and out must be 16-byte, ids and weights 4-byte aligned");
  mlora::CombineArgs a{};
  a.Y = Y;
  a.ids = ids;
  a.weights = weights;
  a.add = add;
  a.out = out;
  a.tokens = tokens;
  a.k = top_k;
  a.d = (int32_t)d;
  a.limit = n_experts ? (uint32_t)n_experts : 0x80000000u;
  mlora::launch_combine(dtype == MLORA_FP32, a, static_cast<hipStream_t>(stream));
  return api_launched();
}

mlora_status mlora_combine_backward(const void* dout, const void* Y, mlora_dtype dtype, int64_t tokens, int32_t top_k,
                                    int64_t d, const int32_t* ids, int32_t n_experts, const float* weights, void* dY,
                                    float* dweights, void* stream) {
  mlora_status st;
  if (const char* msg = combine_error(dtype, tokens, top_k, d, n_experts, &st)) return api_fail(st, msg);
  if (tokens == 0 || (!dY && !dweights)) return MLORA_OK;
  if (!dout || (dweights && !Y))
    return api_fail(MLORA_ERR_INVALID_ARG, "combine backward: dout and Y (for dweights) must be non-NULL");
  if (!api_aligned(dout, 16) || !api_aligned(Y, 16) || !api_aligned(dY, 16) || !api_aligned(ids, 4) ||
      !api_aligned(weights, 4) || !api_aligned(dweights, 4))
    return api_fail(MLORA_ERR_INVALID_ARG, "combine backward: dout, Y and dY must be 16-byte, the others 4-byte aligned");
  mlora::CombineArgs a{};
  a.Y = Y;
  a.ids = ids;
  a.weights = weights;
  a.dout = dout;
  a.dY = dY;
  a.dweights = dweights;
  a.tokens = tokens;
  a.k = top_k;
  a.d = (int32_t)d;
  a.limit = n_experts ? (uint32_t)n_experts : 0x80000000u;
  mlora::launch_combine_backward(dtype == MLORA_FP32, a, static_cast<hipStream_t>(stream));
  return api_launched();
}

}  // extern "C"
