// Launch interface of the products with 4-bit codes and group scales (host
// side).  Launchers check nothing: the C interface (api_affine.cpp) validates
// shapes and sizes before calling.
#pragma once

#include "experts.hpp"

namespace mlora {

// Bytes of the codes of a [rows][cols] matrix, and of its groups' parameters
// (a zero point and a scale in bf16 each).
inline int64_t affine_code_bytes(int64_t rows, int64_t cols) { return rows * (cols / 2); }
inline int64_t affine_param_bytes(int64_t rows, int64_t cols, int32_t group) { return rows * (cols / group) * 4; }

// codes [rows][cols / 2], params [rows][cols / group]; values NULL or
// [rows][cols] of X's type.
void launch_affine_quantize(bool f32, const void* X, int64_t rows, int64_t cols, int64_t ld, int32_t group,
                          bool symmetric, uint8_t* codes, uint32_t* params, void* values, hipStream_t s);

// out [rows][cols] bf16: scale (code - zero), rounded.
void launch_affine_decode(const uint8_t* codes, const uint32_t* params, int64_t rows, int64_t cols, int32_t group,
                        uint16_t* out, hipStream_t s);

// Rows form: a.B the codes, a.b_expert their bytes per expert, a.b_scale the
// parameters; one of the tiles that affine_choice.hpp chooses from.
void launch_affine_few(const ExpertArgs& a, int32_t group, int rows, int cols, hipStream_t s);
void launch_affine_tile(const ExpertArgs& a, int32_t group, int rows, int parts, hipStream_t s);
// dX over the same weights (a.N = d_in, a.K = d_out).
void launch_affine_dx(const ExpertArgs& a, int32_t group, int rows, hipStream_t s);

}  // namespace mlora
