// api_rms.cpp -- the C ABI's RMS norm (include/fp8mi.h): argument checks (no
// HIP call is made before they pass) and dispatch to the launchers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "check.hpp"
#include "fp8mi.h"
#include "launch.hpp"

namespace {

using fp8mi::aligned_to;
using fp8mi::check_matrix;
using fp8mi::in_dtype_ok;
using fp8mi::in_size;
using fp8mi::span_ok;

// sizes and types common to all
int check_common(int x_dtype, int w_dtype, int64_t rows, int64_t cols) {
  if (!in_dtype_ok(x_dtype) || !in_dtype_ok(w_dtype)) return FP8MI_ERR_ENUM;
  if (rows < 0 || cols < 1) return FP8MI_ERR_SHAPE;
  if (cols > (1LL << 28)) return FP8MI_ERR_UNSUPPORTED;
  return FP8MI_OK;
}

// x, and the residual with the rows that it and x add up to
int check_inputs(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                 int64_t ld_residual, const void* weight, int w_dtype, const void* total, int64_t ld_total,
                 const float* rstd) {
  const int64_t es = in_size(x_dtype);
  int st;
  if ((st = check_matrix(x, rows, cols, ld_x, es)) != FP8MI_OK) return st;
  if (residual) {
    if ((st = check_matrix(residual, rows, cols, ld_residual, es)) != FP8MI_OK) return st;
    if ((st = check_matrix(total, rows, cols, ld_total, es)) != FP8MI_OK) return st;
  }
  if (!rstd) return FP8MI_ERR_NULL;
  return aligned_to(rstd, 4) && aligned_to(weight, in_size(w_dtype)) ? FP8MI_OK : FP8MI_ERR_ALIGN;
}

fp8mi::RmsParams params(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                        int64_t ld_residual, const void* weight, int w_dtype, float eps, void* total, int64_t ld_total,
                        float* rstd) {
  fp8mi::RmsParams p{};
  p.x_dtype = x_dtype;
  p.w_dtype = w_dtype;
  p.rows = rows;
  p.cols = cols;
  p.x = x;
  p.ld_x = ld_x;
  p.residual = residual;
  p.ld_residual = ld_residual;
  p.weight = weight;
  p.eps = eps;
  p.total = total;
  p.ld_total = ld_total;
  p.rstd = rstd;
  return p;
}

}  // namespace

extern "C" {

int fp8_rms_norm_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                         int64_t ld_residual, const void* weight, int w_dtype, float eps, void* total,
                         int64_t ld_total, void* y, int64_t ld_y, float* rstd, void* stream) {
  int st = check_common(x_dtype, w_dtype, rows, cols);
  if (st != FP8MI_OK) return st;
  if (!(eps >= 0.0f)) return FP8MI_ERR_SHAPE;
  if (rows == 0) return FP8MI_OK;
  if ((st = check_inputs(x, x_dtype, rows, cols, ld_x, residual, ld_residual, weight, w_dtype, total, ld_total,
                         rstd)) != FP8MI_OK)
    return st;
  if ((st = check_matrix(y, rows, cols, ld_y, in_size(x_dtype))) != FP8MI_OK) return st;
  fp8mi::RmsParams p =
      params(x, x_dtype, rows, cols, ld_x, residual, ld_residual, weight, w_dtype, eps, total, ld_total, rstd);
  p.out = y;
  p.ld_out = ld_y;
  return fp8mi::hip_status(fp8mi::launch_rms_forward(p, (hipStream_t)stream));
}

int fp8_rms_norm_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                          int64_t ld_residual, const void* weight, int w_dtype, float eps, void* total,
                          int64_t ld_total, float* rstd, int recipe, int fmt, int orient, int margin, uint8_t* q_row,
                          int64_t ld_q_row, void* s_row, uint8_t* q_col, int64_t ld_q_col, void* s_col,
                          const float* scale, float* amax, int32_t* nonfinite, void* stream) {
  int st = check_common(x_dtype, w_dtype, rows, cols);
  if (st != FP8MI_OK) return st;
  if (recipe < FP8MI_TENSOR_CURRENT || recipe > FP8MI_MX_1x32_OCP) return FP8MI_ERR_ENUM;
  if (fmt != FP8MI_E4M3 && fmt != FP8MI_E5M2) return FP8MI_ERR_ENUM;
  if (orient != FP8MI_ROW && orient != FP8MI_COL && orient != FP8MI_ROW_AND_COL) return FP8MI_ERR_ENUM;
  // scales that are local to a row's or a column's block, or known beforehand
  const bool delayed = recipe == FP8MI_TENSOR_DELAYED;
  if (!delayed && recipe != FP8MI_BLOCK_1x128 && recipe != FP8MI_MX_1x32 && recipe != FP8MI_MX_1x32_OCP)
    return FP8MI_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || margin < 0 || margin > 64) return FP8MI_ERR_SHAPE;
  if (rows == 0) return FP8MI_OK;
  if ((st = check_inputs(x, x_dtype, rows, cols, ld_x, residual, ld_residual, weight, w_dtype, total, ld_total,
                         rstd)) != FP8MI_OK)
    return st;
  const bool row = orient & FP8MI_ROW, col = orient & FP8MI_COL;
  if ((row && !q_row) || (col && !q_col)) return FP8MI_ERR_NULL;
  if (delayed ? !scale || !amax : (row && !s_row) || (col && !s_col)) return FP8MI_ERR_NULL;
  if ((row && (ld_q_row < cols || !span_ok(rows, ld_q_row, 1))) || (col && (ld_q_col < rows || !span_ok(cols, ld_q_col, 1))))
    return FP8MI_ERR_SHAPE;
  const int64_t ss = recipe == FP8MI_BLOCK_1x128 ? 4 : 1;
  if ((row && (!aligned_to(q_row, 16) || ld_q_row % 16 || !aligned_to(s_row, ss))) ||
      (col && (!aligned_to(q_col, 16) || ld_q_col % 16 || !aligned_to(s_col, ss))) || !aligned_to(nonfinite, 4) || !aligned_to(scale, 4) ||
      !aligned_to(amax, 4))
    return FP8MI_ERR_ALIGN;
  fp8mi::RmsParams p =
      params(x, x_dtype, rows, cols, ld_x, residual, ld_residual, weight, w_dtype, eps, total, ld_total, rstd);
  p.q = fp8mi::QuantParams{nullptr, x_dtype, rows, cols, 0, recipe, fmt, orient, margin, q_row, ld_q_row, s_row,
                           q_col, ld_q_col, s_col, const_cast<float*>(scale), nullptr, amax, nonfinite};
  return fp8mi::hip_status(fp8mi::launch_rms_quantize(p, (hipStream_t)stream));
}

int64_t fp8_rms_norm_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return FP8MI_ERR_SHAPE;
  if (cols > (1LL << 28)) return FP8MI_ERR_UNSUPPORTED;
  return fp8mi::rms_partials(rows, cols) * cols * (int64_t)sizeof(float);
}

int fp8_rms_norm_backward(const void* dy, int64_t ld_dy, const void* total, int x_dtype, int64_t rows, int64_t cols,
                          int64_t ld_total, const void* weight, int w_dtype, const float* rstd, const void* dtotal,
                          int64_t ld_dtotal, void* dx, int64_t ld_dx, void* dweight, void* workspace,
                          int64_t workspace_bytes, void* stream) {
  int st = check_common(x_dtype, w_dtype, rows, cols);
  if (st != FP8MI_OK) return st;
  const int64_t es = in_size(x_dtype);
  if (rows > 0) {
    if ((st = check_matrix(dy, rows, cols, ld_dy, es)) != FP8MI_OK) return st;
    if ((st = check_matrix(total, rows, cols, ld_total, es)) != FP8MI_OK) return st;
    if ((st = check_matrix(dx, rows, cols, ld_dx, es)) != FP8MI_OK) return st;
    if (dtotal && (st = check_matrix(dtotal, rows, cols, ld_dtotal, es)) != FP8MI_OK) return st;
    if (!rstd) return FP8MI_ERR_NULL;
    if (!aligned_to(rstd, 4) || !aligned_to(weight, in_size(w_dtype))) return FP8MI_ERR_ALIGN;
  }
  if (dweight) {
    if (!workspace) return FP8MI_ERR_NULL;
    if (workspace_bytes < fp8_rms_norm_workspace(rows, cols)) return FP8MI_ERR_SHAPE;
    if (!aligned_to(workspace, 4) || !aligned_to(dweight, in_size(w_dtype))) return FP8MI_ERR_ALIGN;
  } else if (rows == 0) {
    return FP8MI_OK;
  }
  fp8mi::RmsParams p = params(total, x_dtype, rows, cols, ld_total, dtotal, ld_dtotal, weight, w_dtype, 0.0f, nullptr, 0,
                              const_cast<float*>(rstd));
  p.out = dx;
  p.ld_out = ld_dx;
  p.dy = dy;
  p.ld_dy = ld_dy;
  p.dweight = dweight;
  p.workspace = static_cast<float*>(workspace);
  return fp8mi::hip_status(fp8mi::launch_rms_backward(p, (hipStream_t)stream));
}

}  // extern "C"
