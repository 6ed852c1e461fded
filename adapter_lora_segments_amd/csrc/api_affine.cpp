// C interface of the 4-bit weights with group scales (include/mlora.h):
// argument checks and launches.  Host state: none; device state: the caller's
// buffers.
#include <hip/hip_runtime.h>

#include "../../include/mlora.h"
#include "api_common.hpp"
#include "affine_choice.hpp"

namespace {

using mlora::api_aligned;
using mlora::api_fail;
using mlora::api_launched;
using mlora::kMaxGrid;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }

// Whether a call decodes the weights into the workspace first.  A call of
// fewer rows does not unless this one does.
bool decodes(const mlora_affine_shape& s) { return s.rows >= mlora::kAffineDecoded * s.n_experts; }

// Message of the first thing wrong with a shape, or NULL.
const char* shape_error(const mlora_affine_shape* s, mlora_status* st) {
  *st = MLORA_ERR_INVALID_ARG;
  if (!s) return "affine: shape is NULL";
  if (s->rows < 0 || s->rows > kMaxRows) return "affine: rows must be in [0, 2^31)";
  if (s->n_experts < 1 || s->n_experts > MLORA_MAX_EXPERTS) return "affine: n_experts must be in [1, 4096]";
  if (!group_ok(s->group)) return "affine: group must be 32, 64 or 128";
  if (s->d_in <= 0 || s->d_in % s->group) return "affine: d_in must be a positive multiple of group";
  if (s->d_out <= 0 || s->d_out % 8) return "affine: d_out must be a positive multiple of 8";
  if (s->top_k < 1 || s->top_k > 64) return "affine: top_k must be in [1, 64]";
  if (s->rows % s->top_k) return "affine: rows must be a multiple of top_k";
  for (int32_t f : {s->x_by_order, s->y_by_order})
    if (f != 0 && f != 1) return "affine: x_by_order and y_by_order are 0 or 1";
  if (s->top_k > 1 && !s->x_by_order) return "affine: top_k > 1 needs x_by_order";
  *st = MLORA_ERR_UNSUPPORTED;
  if (s->d_in > MLORA_MAX_EXPERT_DIM || s->d_out > MLORA_MAX_EXPERT_DIM) return "affine: d_in and d_out are at most 2^20";
  if (s->n_experts * s->d_out > ((int64_t)1 << 40) / s->d_in) return "affine: more than 2^40 weights";
  // launch bounds: tiles of 128 x 128 (larger ones of the decoded products, smaller
  // ones where they fit; few rows a group: 32 x 128), and where the weights are decoded
  // first, a lane per eight of them
  const int64_t d = (s->d_in > s->d_out ? s->d_in : s->d_out) + 127;
  const int64_t groups = s->n_experts < s->rows ? s->n_experts : s->rows;
  if (s->rows / 128 + 2 * groups > kMaxGrid / (d / 128) ||
      (decodes(*s) && s->n_experts * s->d_out > kMaxGrid * 256 / (s->d_in / 8)))
    return "affine: too many tiles for one launch";
  *st = MLORA_OK;
  return nullptr;
}

mlora::ExpertArgs base_args(const mlora_affine_shape& s, const int32_t* offsets, const int32_t* order) {
  mlora::ExpertArgs a{};
  a.offsets = offsets;
  a.order = order;
  a.rows = (int32_t)s.rows;
  a.n_experts = s.n_experts;
  return a;
}

mlora::ExpertArgs forward_args(const mlora_affine_shape& s, const int32_t* offsets, const int32_t* order) {
  mlora::ExpertArgs a = base_args(s, offsets, order);
  a.lda = s.d_in;
  a.ldb = s.d_in;
  a.ldc = s.d_out;
  a.ma = {s.x_by_order, mlora::div_by(s.top_k)};
  a.mc = {s.y_by_order, {0, 0}};
  a.N = (int32_t)s.d_out;
  a.K = (int32_t)s.d_in;
  return a;
}

int64_t weights_of(const mlora_affine_shape& s) { return (int64_t)s.n_experts * s.d_in * s.d_out; }

mlora_status check_call(const mlora_affine_shape& s, const int32_t* offsets, const int32_t* order, void* ws,
                        size_t ws_bytes, int64_t need) {
  if (!offsets && s.n_experts != 1) return api_fail(MLORA_ERR_INVALID_ARG, "affine: offsets may be NULL with one expert only");
  if (!order && (s.x_by_order || s.y_by_order))
    return api_fail(MLORA_ERR_INVALID_ARG, "affine: x_by_order and y_by_order need order");
  if (!api_aligned(offsets, 4) || !api_aligned(order, 4))
    return api_fail(MLORA_ERR_INVALID_ARG, "affine: offsets and order must be 4-byte aligned");
  if (need > 0) {
    if (!ws || !api_aligned(ws, 16))
      return api_fail(MLORA_ERR_INVALID_ARG, "affine: workspace must be non-NULL and 16-byte aligned");
    if ((uint64_t)ws_bytes < (uint64_t)need) return api_fail(MLORA_ERR_WORKSPACE, "affine: workspace too small");
  }
  return MLORA_OK;
}

// All experts' weights decoded into ws.
mlora_status decode(const mlora_affine_shape& s, const uint8_t* q, void* ws, hipStream_t cs) {
  const int64_t rows = s.n_experts * s.d_out;
  mlora::launch_affine_decode(q, reinterpret_cast<const uint32_t*>(q + mlora::affine_code_bytes(rows, s.d_in)), rows, s.d_in,
                            s.group, static_cast<uint16_t*>(ws), cs);
  return api_launched();
}

}  // namespace

extern "C" {

mlora_status mlora_affine_bytes(int64_t rows, int64_t cols, int32_t group, int64_t* bytes) {
  if (!bytes) return api_fail(MLORA_ERR_INVALID_ARG, "affine: bytes is NULL");
  if (!group_ok(group)) return api_fail(MLORA_ERR_INVALID_ARG, "affine: group must be 32, 64 or 128");
  if (rows < 0 || cols <= 0 || cols % group)
    return api_fail(MLORA_ERR_INVALID_ARG, "affine: rows >= 0 and cols a positive multiple of group");
  if (cols > MLORA_MAX_EXPERT_DIM || rows > ((int64_t)1 << 42))
    return api_fail(MLORA_ERR_UNSUPPORTED, "affine: matrix too large");
  *bytes = mlora::affine_code_bytes(rows, cols) + mlora::affine_param_bytes(rows, cols, group);
  return MLORA_OK;
}

mlora_status mlora_affine_quantize(const void* X, mlora_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                 int32_t group, int32_t symmetric, void* q, void* values, void* stream) {
  if (dtype != MLORA_BF16 && dtype != MLORA_FP32) return api_fail(MLORA_ERR_INVALID_ARG, "affine quantize: unknown dtype");
  if (symmetric != 0 && symmetric != 1) return api_fail(MLORA_ERR_INVALID_ARG, "affine quantize: symmetric must be 0 or 1");
  int64_t bytes;
  const mlora_status st = mlora_affine_bytes(rows, cols, group, &bytes);
  if (st != MLORA_OK) return st;
  if (ld < cols || ld % (dtype == MLORA_BF16 ? 8 : 4))
    return api_fail(MLORA_ERR_INVALID_ARG, "affine quantize: ld >= cols and a multiple of 8 (bf16) or 4 (fp32)");
  if (rows > kMaxGrid * 256 / (cols / 8))
    return api_fail(MLORA_ERR_UNSUPPORTED, "affine quantize: matrix too large for one launch");
  if (rows == 0) return MLORA_OK;
  if (!X || !q) return api_fail(MLORA_ERR_INVALID_ARG, "affine quantize: X and q must be non-NULL");
  if (!api_aligned(X, 16) || !api_aligned(q, 16) || !api_aligned(values, 16))
    return api_fail(MLORA_ERR_INVALID_ARG, "affine quantize: device pointers must be 16-byte aligned");
  uint8_t* codes = static_cast<uint8_t*>(q);
  mlora::launch_affine_quantize(dtype == MLORA_FP32, X, rows, cols, ld, group, symmetric != 0, codes,
                              reinterpret_cast<uint32_t*>(codes + mlora::affine_code_bytes(rows, cols)), values,
                              static_cast<hipStream_t>(stream));
  return api_launched();
}

mlora_status mlora_affine_workspace(const mlora_affine_shape* shape, int64_t* forward, int64_t* backward) {
  mlora_status st;
  if (const char* msg = shape_error(shape, &st)) return api_fail(st, msg);
  if (forward) *forward = decodes(*shape) ? 2 * weights_of(*shape) : 0;
  if (backward) *backward = decodes(*shape) ? 2 * weights_of(*shape) : 0;
  return MLORA_OK;
}

mlora_status mlora_affine_forward(const mlora_affine_shape* shape, const void* X, const void* q, const int32_t* offsets,
                                const int32_t* order, void* Y, void* workspace, size_t ws_bytes, void* stream) {
  mlora_status st;
  if (const char* msg = shape_error(shape, &st)) return api_fail(st, msg);
  const mlora_affine_shape& s = *shape;
  const bool codes = !decodes(s);
  st = check_call(s, offsets, order, workspace, ws_bytes, codes ? 0 : 2 * weights_of(s));
  if (st != MLORA_OK) return st;
  if (!q || (s.rows > 0 && (!X || !Y))) return api_fail(MLORA_ERR_INVALID_ARG, "affine forward: X, q and Y must be non-NULL");
  if (!api_aligned(X, 16) || !api_aligned(q, 16) || !api_aligned(Y, 16))
    return api_fail(MLORA_ERR_INVALID_ARG, "affine forward: device pointers must be 16-byte aligned");
  if (s.rows == 0) return MLORA_OK;
  hipStream_t cs = static_cast<hipStream_t>(stream);
  mlora::ExpertArgs a = forward_args(s, offsets, order);
  a.A = static_cast<const uint8_t*>(X);
  a.C = Y;
  const uint8_t* const w = static_cast<const uint8_t*>(q);
  if (codes) {
    a.B = w;
    a.b_expert = s.d_in * s.d_out / 2;
    a.b_scale = w + mlora::affine_code_bytes(s.n_experts * s.d_out, s.d_in);
    const mlora::AffineChoice& c = mlora::affine_choose(mlora::kAffine, a, s.group);
    if (c.few) mlora::launch_affine_few(a, s.group, c.rows, c.cols, cs);
    else mlora::launch_affine_tile(a, s.group, c.rows, c.split, cs);
  } else {
    st = decode(s, w, workspace, cs);
    if (st != MLORA_OK) return st;
    a.B = static_cast<const uint8_t*>(workspace);
    a.b_expert = s.d_in * s.d_out * 2;
    mlora::launch_expert_rows(mlora::ExpertForm::kBf16, true, a, cs);
  }
  return api_launched();
}

mlora_status mlora_affine_backward(const mlora_affine_shape* shape, const void* dY, const void* q, const int32_t* offsets,
                                 const int32_t* order, void* dX, void* workspace, size_t ws_bytes, void* stream) {
  mlora_status st;
  if (const char* msg = shape_error(shape, &st)) return api_fail(st, msg);
  const mlora_affine_shape& s = *shape;
  const bool codes = !decodes(s);
  st = check_call(s, offsets, order, workspace, ws_bytes, codes ? 0 : 2 * weights_of(s));
  if (st != MLORA_OK) return st;
  if (!q || (s.rows > 0 && (!dY || !dX))) return api_fail(MLORA_ERR_INVALID_ARG, "affine backward: dY, q and dX must be non-NULL");
  if (!api_aligned(dY, 16) || !api_aligned(q, 16) || !api_aligned(dX, 16))
    return api_fail(MLORA_ERR_INVALID_ARG, "affine backward: device pointers must be 16-byte aligned");
  if (s.rows == 0) return MLORA_OK;
  hipStream_t cs = static_cast<hipStream_t>(stream);
  mlora::ExpertArgs a = base_args(s, offsets, order);
  a.A = static_cast<const uint8_t*>(dY);
  a.C = dX;
  a.lda = s.d_out;
  a.ldb = s.d_in;
  a.ldc = s.d_in;
  a.ma = {s.y_by_order, {0, 0}};
  a.mc = {s.x_by_order, {0, 0}};
  a.N = (int32_t)s.d_in;
  a.K = (int32_t)s.d_out;
  const uint8_t* const w = static_cast<const uint8_t*>(q);
  if (codes) {
    a.B = w;
    a.b_expert = s.d_in * s.d_out / 2;
    a.b_scale = w + mlora::affine_code_bytes(s.n_experts * s.d_out, s.d_in);
    mlora::launch_affine_dx(a, s.group, mlora::affine_choose(mlora::kAffineDx, a, s.group).rows, cs);
  } else {
    st = decode(s, w, workspace, cs);
    if (st != MLORA_OK) return st;
    a.B = static_cast<const uint8_t*>(workspace);
    a.b_expert = s.d_in * s.d_out * 2;
    mlora::launch_expert_rows(mlora::ExpertForm::kBf16, false, a, cs);
  }
  return api_launched();
}

}  // extern "C"
