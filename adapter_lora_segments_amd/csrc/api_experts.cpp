// C interface of the grouped expert products, the row grouping and the MXFP4
// quantizer (include/mlora.h): argument checks and launches.  Host state:
// none; device state: the caller's buffers.
#include <hip/hip_runtime.h>

#include <new>
#include <string>

#include "../../include/mlora.h"
#include "experts.hpp"
#include "kernels.hpp"

namespace {

// No exception leaves a C entry, not even from building a message.
mlora_status fail(mlora_status st, const char* msg) noexcept {
  try {
    mlora::set_last_error(msg);
  } catch (...) {
  }
  return st;
}

mlora_status launched() noexcept {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return MLORA_OK;
  try {
    mlora::set_last_error(std::string("kernel launch: ") + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")");
  } catch (...) {
  }
  return MLORA_ERR_HIP;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
using mlora::kMaxGrid;

// Message of the first thing wrong with a shape, or NULL.
const char* shape_error(const mlora_expert_shape& s, mlora_status* st) {
  *st = MLORA_ERR_INVALID_ARG;
  if (s.rows < 0 || s.rows > kMaxRows) return "expert: rows must be in [0, 2^31)";
  if (s.n_experts < 1 || s.n_experts > MLORA_MAX_EXPERTS) return "expert: n_experts must be in [1, 4096]";
  if (s.dtype != MLORA_BF16 && s.dtype != MLORA_FP32) return "expert: unknown dtype";
  if (s.w_layout != MLORA_W0_KN && s.w_layout != MLORA_W0_NK) return "expert: w_layout must be KN or NK";
  const int64_t unit = s.dtype == MLORA_BF16 ? 8 : 4;
  if (s.d_in <= 0 || s.d_out <= 0 || s.d_in % unit || s.d_out % unit)
    return "expert: d_in and d_out must be positive multiples of 8 (bf16) or 4 (fp32)";
  if (s.top_k < 1 || s.top_k > 64) return "expert: top_k must be in [1, 64]";
  if (s.rows % s.top_k) return "expert: rows must be a multiple of top_k";
  if (s.top_k > 1 && !s.x_by_order) return "expert: top_k > 1 needs x_by_order";
  for (int32_t f : {s.x_by_order, s.y_by_order, s.grad_accumulate})
    if (f != 0 && f != 1) return "expert: x_by_order, y_by_order and grad_accumulate are 0 or 1";
  if (s.w_format != MLORA_W0_BF16 && s.w_format != MLORA_W0_MXFP4)
    return "expert: w_format must be MLORA_W0_BF16 or MLORA_W0_MXFP4";
  if (s.act_format != MLORA_ACT_BF16 && s.act_format != MLORA_ACT_MXFP4)
    return "expert: act_format must be MLORA_ACT_BF16 or MLORA_ACT_MXFP4";
  *st = MLORA_ERR_UNSUPPORTED;
  if (s.d_in > MLORA_MAX_EXPERT_DIM || s.d_out > MLORA_MAX_EXPERT_DIM) return "expert: d_in and d_out are at most 2^20";
  if (s.w_format == MLORA_W0_MXFP4 &&
      (s.dtype != MLORA_BF16 || s.w_layout != MLORA_W0_NK || s.d_in % 128 != 0))
    return "expert: MXFP4 weights need bf16, the NK layout and d_in a multiple of 128";
  if (s.act_format == MLORA_ACT_MXFP4 && s.w_format != MLORA_W0_MXFP4)
    return "expert: MXFP4 activations need MXFP4 weights";
  // launch bounds at 256 x 256 tiles (smaller ones are taken where they fit),
  // and those of the MXFP4 conversions, a thread per 8 activations or 32 weights
  const int64_t d = (s.d_in > s.d_out ? s.d_in : s.d_out) + 255;
  const int64_t tiles = s.rows / 256 + (s.n_experts < s.rows ? s.n_experts : s.rows);
  const int64_t dw = (((s.d_in + 255) / 256) * ((s.d_out + 255) / 256) + 7) / 8 * 8;
  if (tiles > kMaxGrid / (d / 256) || dw > kMaxGrid / s.n_experts ||
      (s.act_format == MLORA_ACT_MXFP4 && s.rows > kMaxGrid * 256 / (s.d_in / 8)) ||
      (s.w_format == MLORA_W0_MXFP4 && s.n_experts * s.d_out > kMaxGrid * 256 / (s.d_in / 32)))
    return "expert: too many tiles for one launch";
  *st = MLORA_OK;
  return nullptr;
}

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

// Workspace bytes of a forward (quantized activations) and of a backward's dX
// (the decoded MXFP4 weight) and dW (partial sums of long groups).
int64_t forward_ws(const mlora_expert_shape& s) {
  if (s.act_format != MLORA_ACT_MXFP4) return 0;
  const int64_t t = s.x_by_order ? s.rows / s.top_k : s.rows;
  return round16(t * s.d_in / 2) + round16(t * s.d_in / 32);
}
int64_t dx_ws(const mlora_expert_shape& s) {
  return s.w_format == MLORA_W0_MXFP4 ? 2 * (int64_t)s.n_experts * s.d_in * s.d_out : 0;
}
int64_t dw_ws(const mlora_expert_shape& s) {
  return s.w_format == MLORA_W0_MXFP4 ? 0 : mlora::dw_part_bytes(s.dtype == MLORA_FP32, s.rows, s.n_experts, s.d_in, s.d_out);
}

mlora_status check_call(const mlora_expert_shape* s, const int32_t* offsets, const int32_t* order, void* ws,
                        size_t ws_bytes, int64_t need) {
  if (!offsets && s->n_experts != 1) return fail(MLORA_ERR_INVALID_ARG, "expert: offsets may be NULL with one expert only");
  if (!order && (s->x_by_order || s->y_by_order))
    return fail(MLORA_ERR_INVALID_ARG, "expert: x_by_order and y_by_order need order");
  if (!aligned(offsets, 4) || !aligned(order, 4))
    return fail(MLORA_ERR_INVALID_ARG, "expert: offsets and order must be 4-byte aligned");
  if (need > 0) {
    if (!ws || !aligned(ws, 16)) return fail(MLORA_ERR_INVALID_ARG, "expert: workspace must be non-NULL and 16-byte aligned");
    if ((uint64_t)ws_bytes < (uint64_t)need) return fail(MLORA_ERR_WORKSPACE, "expert: workspace too small");
  }
  return MLORA_OK;
}

mlora::ExpertArgs base_args(const mlora_expert_shape& s, const int32_t* offsets, const int32_t* order) {
  mlora::ExpertArgs a{};
  a.offsets = offsets;
  a.order = order;
  a.rows = (int32_t)s.rows;
  a.n_experts = s.n_experts;
  return a;
}

}  // namespace

extern "C" {

mlora_status mlora_group_rows_workspace(int64_t rows, int32_t n_groups, int64_t* bytes) {
  if (!bytes) return fail(MLORA_ERR_INVALID_ARG, "group_rows: bytes is NULL");
  if (rows < 0 || rows > kMaxRows) return fail(MLORA_ERR_INVALID_ARG, "group_rows: rows must be in [0, 2^31)");
  if (n_groups < 1 || n_groups > MLORA_MAX_EXPERTS)
    return fail(MLORA_ERR_INVALID_ARG, "group_rows: n_groups must be in [1, 4096]");
  // the most parts any smaller number of rows takes
  const int64_t parts = (rows + mlora::kGroupMinPart - 1) / mlora::kGroupMinPart;
  *bytes = rows <= mlora::kGroupOneLaunch
               ? 0
               : 4 * (int64_t)n_groups * (parts < mlora::kGroupMaxParts ? parts : mlora::kGroupMaxParts);
  return MLORA_OK;
}

mlora_status mlora_group_rows(const int32_t* ids, int64_t rows, int32_t n_groups, int32_t* offsets, int32_t* order,
                              void* workspace, size_t ws_bytes, void* stream) {
  int64_t need = 0;
  const mlora_status st = mlora_group_rows_workspace(rows, n_groups, &need);
  if (st != MLORA_OK) return st;
  if (!offsets || (rows > 0 && (!ids || !order)))
    return fail(MLORA_ERR_INVALID_ARG, "group_rows: ids, offsets and order must be non-NULL");
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4))
    return fail(MLORA_ERR_INVALID_ARG, "group_rows: ids, offsets and order must be 4-byte aligned");
  if (need > 0) {
    if (!workspace || !aligned(workspace, 16))
      return fail(MLORA_ERR_INVALID_ARG, "group_rows: workspace must be non-NULL and 16-byte aligned");
    if ((uint64_t)ws_bytes < (uint64_t)need) return fail(MLORA_ERR_WORKSPACE, "group_rows: workspace too small");
  }
  mlora::launch_group_rows(ids, rows, n_groups, offsets, order, static_cast<int32_t*>(workspace),
                           static_cast<hipStream_t>(stream));
  return launched();
}

mlora_status mlora_expert_workspace(const mlora_expert_shape* shape, int64_t* bytes) {
  if (!shape || !bytes) return fail(MLORA_ERR_INVALID_ARG, "expert: shape and bytes must be non-NULL");
  mlora_status st;
  if (const char* msg = shape_error(*shape, &st)) return fail(st, msg);
  // a weight is quantized (dX only) or has a dW
  const int64_t f = forward_ws(*shape), b = dx_ws(*shape) + dw_ws(*shape);
  *bytes = f > b ? f : b;
  return MLORA_OK;
}

mlora_status mlora_expert_forward_workspace(const mlora_expert_shape* shape, int64_t* bytes) {
  if (!shape || !bytes) return fail(MLORA_ERR_INVALID_ARG, "expert: shape and bytes must be non-NULL");
  mlora_status st;
  if (const char* msg = shape_error(*shape, &st)) return fail(st, msg);
  *bytes = forward_ws(*shape);
  return MLORA_OK;
}

mlora_status mlora_expert_forward(const mlora_expert_shape* shape, const void* X, const void* W,
                                  const int32_t* offsets, const int32_t* order, void* Y, void* workspace,
                                  size_t ws_bytes, void* stream) {
  if (!shape) return fail(MLORA_ERR_INVALID_ARG, "expert: shape is NULL");
  const mlora_expert_shape& s = *shape;
  mlora_status st;
  if (const char* msg = shape_error(s, &st)) return fail(st, msg);
  st = check_call(shape, offsets, order, workspace, ws_bytes, s.rows > 0 ? forward_ws(s) : 0);
  if (st != MLORA_OK) return st;
  if (!W || (s.rows > 0 && (!X || !Y))) return fail(MLORA_ERR_INVALID_ARG, "expert forward: X, W and Y must be non-NULL");
  for (const void* p : {X, W, (const void*)Y})
    if (!aligned(p, 16)) return fail(MLORA_ERR_INVALID_ARG, "expert forward: device pointers must be 16-byte aligned");
  if (s.rows == 0) return MLORA_OK;

  hipStream_t cs = static_cast<hipStream_t>(stream);
  const int64_t esz = s.dtype == MLORA_BF16 ? 2 : 4, wn = s.d_in * s.d_out;
  const mlora::DivBy div = mlora::div_by(s.top_k);
  mlora::ExpertArgs a = base_args(s, offsets, order);
  a.A = static_cast<const uint8_t*>(X);
  a.B = static_cast<const uint8_t*>(W);
  a.C = Y;
  a.lda = s.d_in;
  a.ldc = s.d_out;
  a.ma = {s.x_by_order, div};
  a.mc = {s.y_by_order, {0, 0}};
  a.N = (int32_t)s.d_out;
  a.K = (int32_t)s.d_in;
  const bool nk = s.w_layout == MLORA_W0_NK;
  a.ldb = nk ? s.d_in : s.d_out;
  a.b_expert = wn * esz;
  mlora::ExpertForm form = s.dtype == MLORA_BF16 ? mlora::ExpertForm::kBf16 : mlora::ExpertForm::kF32;
  if (s.w_format == MLORA_W0_MXFP4) {
    a.b_expert = wn / 2;
    a.b_scale = a.B + s.n_experts * (wn / 2);
    form = mlora::ExpertForm::kW4A16;
    if (s.act_format == MLORA_ACT_MXFP4) {
      const int64_t t = s.x_by_order ? s.rows / s.top_k : s.rows;
      uint8_t* codes = static_cast<uint8_t*>(workspace);
      uint8_t* scales = codes + round16(t * s.d_in / 2);
      mlora::launch_quant_mx4(false, false, X, t, s.d_in, s.d_in, codes, scales, nullptr, cs);
      st = launched();
      if (st != MLORA_OK) return st;
      a.A = codes;
      a.a_scale = scales;
      form = mlora::ExpertForm::kW4A4;
    }
  }
  mlora::launch_expert_rows(form, nk, a, cs);
  return launched();
}

mlora_status mlora_expert_backward(const mlora_expert_shape* shape, const void* dY, const void* X, const void* W,
                                   const int32_t* offsets, const int32_t* order, void* dX, float* dW,
                                   void* workspace, size_t ws_bytes, void* stream) {
  if (!shape) return fail(MLORA_ERR_INVALID_ARG, "expert: shape is NULL");
  const mlora_expert_shape& s = *shape;
  mlora_status st;
  if (const char* msg = shape_error(s, &st)) return fail(st, msg);
  const bool w4 = s.w_format == MLORA_W0_MXFP4;
  const bool want_dx = dX != nullptr && s.rows > 0;
  st = check_call(shape, offsets, order, workspace, ws_bytes, (want_dx ? dx_ws(s) : 0) + (dW ? dw_ws(s) : 0));
  if (st != MLORA_OK) return st;
  if (w4 && dW) return fail(MLORA_ERR_UNSUPPORTED, "expert backward: an MXFP4 weight is frozen, dW must be NULL");
  if ((s.rows > 0 && !dY) || (want_dx && !W) || (dW && s.rows > 0 && !X))
    return fail(MLORA_ERR_INVALID_ARG, "expert backward: dY, W (for dX) and X (for dW) must be non-NULL");
  for (const void* p : {dY, X, W, (const void*)dX, (const void*)dW})
    if (!aligned(p, 16)) return fail(MLORA_ERR_INVALID_ARG, "expert backward: device pointers must be 16-byte aligned");

  hipStream_t cs = static_cast<hipStream_t>(stream);
  const bool f32 = s.dtype == MLORA_FP32, nk = s.w_layout == MLORA_W0_NK;
  const int64_t esz = f32 ? 4 : 2, wn = s.d_in * s.d_out;
  const mlora::DivBy div = mlora::div_by(s.top_k);
  if (want_dx) {
    mlora::ExpertArgs a = base_args(s, offsets, order);
    a.A = static_cast<const uint8_t*>(dY);
    a.B = static_cast<const uint8_t*>(W);
    if (w4) {
      // decoded as [n_experts * d_out][d_in]
      const uint8_t* codes = static_cast<const uint8_t*>(W);
      mlora::launch_dequant_mx4(true, codes, codes + s.n_experts * (wn / 2), s.d_in, s.n_experts * s.d_out,
                                static_cast<uint16_t*>(workspace), cs);
      st = launched();
      if (st != MLORA_OK) return st;
      a.B = static_cast<const uint8_t*>(workspace);
    }
    a.C = dX;
    a.lda = s.d_out;
    a.ldc = s.d_in;
    a.ma = {s.y_by_order, {0, 0}};
    a.mc = {s.x_by_order, {0, 0}};
    a.N = (int32_t)s.d_in;
    a.K = (int32_t)s.d_out;
    a.ldb = nk ? s.d_in : s.d_out;
    a.b_expert = wn * esz;
    mlora::launch_expert_rows(f32 ? mlora::ExpertForm::kF32 : mlora::ExpertForm::kBf16, !nk, a, cs);
    st = launched();
    if (st != MLORA_OK) return st;
  }
  if (dW && !(s.rows == 0 && s.grad_accumulate)) {
    mlora::ExpertArgs a = base_args(s, offsets, order);
    const mlora::RowMap mx = {s.x_by_order, div}, my = {s.y_by_order, {0, 0}};
    a.A = static_cast<const uint8_t*>(nk ? dY : X);
    a.B = static_cast<const uint8_t*>(nk ? X : dY);
    a.ma = nk ? my : mx;
    a.mb = nk ? mx : my;
    a.M = (int32_t)(nk ? s.d_out : s.d_in);
    a.N = (int32_t)(nk ? s.d_in : s.d_out);
    a.lda = a.M;
    a.ldb = a.N;
    a.ldc = a.N;
    a.C = dW;
    a.c_expert = wn;
    a.accumulate = s.grad_accumulate;
    a.chunk = (int32_t)mlora::dw_chunk(f32, s.rows, s.n_experts, s.d_in, s.d_out);
    a.part = static_cast<float*>(workspace);
    mlora::launch_expert_dw(f32, a, cs);
    st = launched();
    if (st != MLORA_OK) return st;
  }
  return MLORA_OK;
}

mlora_status mlora_microscale_quantize(const void* X, mlora_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                       int32_t down, void* q, void* values, void* stream) {
  if (dtype != MLORA_BF16 && dtype != MLORA_FP32) return fail(MLORA_ERR_INVALID_ARG, "quantize: unknown dtype");
  if (down != 0 && down != 1) return fail(MLORA_ERR_INVALID_ARG, "quantize: down must be 0 or 1");
  const int64_t unit = dtype == MLORA_BF16 ? 8 : 4;
  if (rows < 0 || cols <= 0 || ld < cols || ld % unit)
    return fail(MLORA_ERR_INVALID_ARG, "quantize: rows >= 0, cols > 0, ld >= cols and a multiple of 8 (bf16) or 4 (fp32)");
  if (down ? (rows % 32 || cols % 8) : cols % 32 != 0)
    return fail(MLORA_ERR_INVALID_ARG,
                "quantize: cols must be a multiple of 32, or with down rows of 32 and cols of 8");
  if (cols > MLORA_MAX_EXPERT_DIM || rows > (kMaxGrid * 256) / (cols / 8))
    return fail(MLORA_ERR_UNSUPPORTED, "quantize: matrix too large for one launch");
  if (rows == 0) return MLORA_OK;
  if (!X || !q) return fail(MLORA_ERR_INVALID_ARG, "quantize: X and q must be non-NULL");
  if (!aligned(X, 16) || !aligned(q, 16) || !aligned(values, 16))
    return fail(MLORA_ERR_INVALID_ARG, "quantize: device pointers must be 16-byte aligned");
  uint8_t* codes = static_cast<uint8_t*>(q);
  mlora::launch_quant_mx4(dtype == MLORA_FP32, down != 0, X, rows, cols, ld, codes, codes + rows * (cols / 2), values,
                          static_cast<hipStream_t>(stream));
  return launched();
}

}  // extern "C"
