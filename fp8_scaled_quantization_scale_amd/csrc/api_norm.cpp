// api_norm.cpp -- the C ABI's layer norm (include/fp8mi.h): argument checks
// (no HIP call is made before they pass) and dispatch to the launchers.
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

// sizes and types common to both directions
int check_common(int x_dtype, int w_dtype, int64_t rows, int64_t cols) {
  if (!in_dtype_ok(x_dtype) || !in_dtype_ok(w_dtype)) return FP8MI_ERR_ENUM;
  if (rows < 0 || cols < 1) return FP8MI_ERR_SHAPE;
  if (cols > (1LL << 28)) return FP8MI_ERR_UNSUPPORTED;
  return FP8MI_OK;
}

}  // namespace

extern "C" {

int fp8_layer_norm_forward(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* weight,
                           const void* bias, int w_dtype, float eps, void* y, int64_t ld_y, float* mean, float* rstd,
                           void* stream) {
  int st = check_common(x_dtype, w_dtype, rows, cols);
  if (st != FP8MI_OK) return st;
  if (!(eps >= 0.0f)) return FP8MI_ERR_SHAPE;
  if (rows == 0) return FP8MI_OK;
  const int64_t es = in_size(x_dtype);
  if ((st = check_matrix(x, rows, cols, ld_x, es)) != FP8MI_OK) return st;
  if ((st = check_matrix(y, rows, cols, ld_y, es)) != FP8MI_OK) return st;
  if (!mean || !rstd) return FP8MI_ERR_NULL;
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(weight, in_size(w_dtype)) ||
      !aligned_to(bias, in_size(w_dtype)))
    return FP8MI_ERR_ALIGN;
  fp8mi::NormParams p{x,    nullptr, x_dtype, w_dtype, rows, cols,    ld_x,    0,       ld_y,
                      weight, bias,  eps,     mean,    rstd, y, nullptr, nullptr, nullptr};
  return fp8mi::hip_status(fp8mi::launch_norm_forward(p, (hipStream_t)stream));
}

int64_t fp8_layer_norm_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return FP8MI_ERR_SHAPE;
  if (cols > (1LL << 28)) return FP8MI_ERR_UNSUPPORTED;
  return fp8mi::norm_partials(rows) * 2 * cols * (int64_t)sizeof(float);
}

int fp8_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int x_dtype, int64_t rows, int64_t cols,
                            int64_t ld_x, const void* weight, int w_dtype, const float* mean, const float* rstd,
                            void* dx, int64_t ld_dx, void* dweight, void* dbias, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  int st = check_common(x_dtype, w_dtype, rows, cols);
  if (st != FP8MI_OK) return st;
  const int64_t es = in_size(x_dtype);
  if (rows > 0) {
    if ((st = check_matrix(dy, rows, cols, ld_dy, es)) != FP8MI_OK) return st;
    if ((st = check_matrix(x, rows, cols, ld_x, es)) != FP8MI_OK) return st;
    if ((st = check_matrix(dx, rows, cols, ld_dx, es)) != FP8MI_OK) return st;
    if (!mean || !rstd) return FP8MI_ERR_NULL;
    if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(weight, in_size(w_dtype))) return FP8MI_ERR_ALIGN;
  }
  if (dweight || dbias) {
    if (!workspace) return FP8MI_ERR_NULL;
    if (workspace_bytes < fp8_layer_norm_workspace(rows, cols)) return FP8MI_ERR_SHAPE;
    if (!aligned_to(workspace, 4) || !aligned_to(dweight, in_size(w_dtype)) || !aligned_to(dbias, in_size(w_dtype)))
      return FP8MI_ERR_ALIGN;
  } else if (rows == 0) {
    return FP8MI_OK;
  }
  fp8mi::NormParams p{x,      dy,      x_dtype,
                      w_dtype, rows,   cols,
                      ld_x,   ld_dy,   ld_dx,
                      weight, nullptr, 0.0f,
                      const_cast<float*>(mean), const_cast<float*>(rstd), dx,
                      dweight, dbias,  static_cast<float*>(workspace)};
  return fp8mi::hip_status(fp8mi::launch_norm_backward(p, (hipStream_t)stream));
}

}  // extern "C"
