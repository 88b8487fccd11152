// launch.hpp -- internal launchers behind the C ABI (include/fp8mi.h).
// Arguments arrive here already validated by the host-side checks in api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace fp8mi {

// ---- the device a launch runs on, and its size -------------------------
// Work goes to the caller's stream, whose device need not be the current
// one; persistent grids are sized for that device (a partitioned GPU
// exposes devices with fewer compute units).
constexpr int kMaxDevices = 64;

inline int stream_device(hipStream_t st) {
  int dev = -1;
  if (st != nullptr && hipStreamGetDevice(st, &dev) == hipSuccess && dev >= 0 && dev < kMaxDevices) return dev;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) dev = 0;
  return dev;
}

// Compute units of device `dev`, queried once per process and device.  The
// cache is atomic: concurrent first calls store the same value.
inline int cu_count(int dev) {
  static std::atomic<int> cache[kMaxDevices];
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// values mirror the FP8MI_* macros of the public header
constexpr int kInBf16 = 0, kInFp32 = 1;
constexpr int kOutBf16 = 0, kOutFp32 = 1;
constexpr int kRecipeTensorCurrent = 0, kRecipeTensorDelayed = 1, kRecipeBlock1x128 = 2,
              kRecipeBlock128x128 = 3, kRecipeMx1x32 = 4, kRecipeChannel = 5, kRecipeMx1x32Ocp = 6;
constexpr int kGemmTensor = 0, kGemmBlock128x128 = 1, kGemmBlock1x128 = 2, kGemmMx = 3, kGemmBlock2d = 4,
              kGemmChannel = 5;
// internal: BF16 operands, no scales (fp8_bf16_gemm)
constexpr int kGemmBf16 = 16;
// slots of a delayed-scaling amax accumulator (FP8MI_AMAX_SLOTS)
constexpr int kAmaxSlots = 1024;
// experts a sort, a dispatch or a grouped GEMM takes (FP8MI_MAX_EXPERTS), and
// the multiple of rows their segments start on (FP8MI_EXPERT_ALIGN)
constexpr int kMaxExperts = 1024;
constexpr int kExpertAlign = 128;

struct QuantParams {
  const void* x;
  int x_dtype;
  int64_t rows, cols, ld_x;
  int recipe, fmt, orient, margin;
  uint8_t* q_row;
  int64_t ld_q_row;
  void* s_row;
  uint8_t* q_col;
  int64_t ld_q_col;
  void* s_col;
  float* scale;
  float* scale_inv;
  float* amax;
  int32_t* nonfinite;
  // current scaling: where the amax pass leaves its per-workgroup partial
  // maxima (nullptr: amax[1 ..], the caller's array)
  uint32_t* partials = nullptr;
};

struct GemmParams {
  const uint8_t* a;
  int fmt_a;
  const void* s_a;
  int64_t lda;
  const uint8_t* b;
  int fmt_b;
  const void* s_b;
  int64_t ldb;
  int recipe;
  int64_t M, N, K;
  void* c;
  int c_dtype;
  int64_t ldc;
};

// fp8_gemm_grouped (contract: one product per expert over its own rows;
// else each expert's rows times its own B)
struct GroupedGemmParams {
  bool contract;
  const uint8_t* a;
  int fmt_a;
  const void* s_a;
  int64_t lda;
  const uint8_t* b;
  int fmt_b;
  const void* s_b;
  int64_t ldb, stride_b, ld_sb, stride_sb;
  int recipe;
  const int32_t* offsets;
  int64_t experts, R, M, N, K;
  void* c;
  int c_dtype;
  int64_t ldc, stride_c;
};

// fp8_moe_quantize: q.rows is the sorted buffer's row capacity
struct MoeQuantParams {
  QuantParams q;
  const int32_t* offsets;
  const int32_t* row_slot;
  const float* weights;
  int64_t experts, topk, x_rows;
};

struct MoeSortParams {
  const void* expert;
  int idx_dtype;
  int64_t tokens, topk, ld_expert, experts;
  int32_t *offsets, *counts, *row_slot, *slot_row;
  int64_t rows;
  int32_t* workspace;
};

// dispatch, combine and combine's backward pass
struct MoeRowsParams {
  int dtype;
  int64_t tokens, topk, experts, cols, rows;
  const int32_t *offsets, *counts, *slot_row;
  const float* weights;
  const void* token_rows;  // x / dy
  int64_t ld_token;
  const void* expert_rows;  // ys
  int64_t ld_expert;
  void* out;                // dispatch: sorted rows; combine: token rows; backward: sorted rows
  int64_t ld_out;
  float* dweights;
};

struct NormParams {
  const void* x;
  const void* dy;
  int x_dtype, w_dtype;
  int64_t rows, cols, ld_x, ld_dy, ld_out;
  const void* weight;
  const void* bias;
  float eps;
  float *mean, *rstd;
  void* out;  // y / dx
  void *dweight, *dbias;
  float* workspace;
};

// RMS norm: forward (out: y), into codes (q's recipe and outputs), backward (x:
// the rows the forward pass normed, residual: the gradient that reaches them by
// itself, out: dx)
struct RmsParams {
  int x_dtype, w_dtype;
  int64_t rows, cols;
  const void* x;
  int64_t ld_x;
  const void* residual;
  int64_t ld_residual;
  const void* weight;
  float eps;
  void* total;
  int64_t ld_total;
  float* rstd;
  void* out;
  int64_t ld_out;
  const void* dy;
  int64_t ld_dy;
  void* dweight;
  float* workspace;
  QuantParams q;
};

// the router: choices, counts and balance loss of logits (given: of choices
// that the caller made, chosen), and the logits' gradient
struct RouteParams {
  const void* logits;
  int dtype;
  int64_t tokens, experts, ld;
  const uint8_t* mask;
  int64_t topk;
  int normalize;
  int32_t* expert;
  float* weights;
  bool given;
  const void* chosen;
  int idx_dtype;
  int64_t ld_chosen;
  float* loss;
  int32_t* counts;
  float* slope;
  void* workspace;
  // backward
  const float* dweights;
  const float* dloss;
  void* dlogits;
  int64_t ld_dlogits;
};

// FP8MI_OK, or FP8MI_ERR_HIP with the error's text kept for fp8_status_string
int hip_status(hipError_t e);

hipError_t launch_quantize(const QuantParams& p, hipStream_t st);
// fp8_quantize with current scaling's partial maxima in the library's static
// device scratch instead of amax[1 ..] (see quantize.hip)
hipError_t launch_quantize_static_scratch(const QuantParams& p, hipStream_t st);
hipError_t launch_empty_scale(float* amax, float* scale, float* scale_inv, hipStream_t st);
hipError_t launch_history(float* history, int32_t* head, int len, float* amax, int fmt, int margin,
                          float* scale, float* scale_inv, int32_t* nonfinite, hipStream_t st);
hipError_t launch_gemm(const GemmParams& p, hipStream_t st);
// a, b BF16 [M x K], [N x K]; K, lda, ldb in elements
hipError_t launch_gemm_bf16(const GemmParams& p, hipStream_t st);
hipError_t launch_gemm_grouped(const GroupedGemmParams& p, hipStream_t st);
hipError_t launch_moe_quantize(const MoeQuantParams& p, hipStream_t st);
hipError_t launch_moe_sort(const MoeSortParams& p, hipStream_t st);
int64_t moe_sort_blocks(int64_t slots);
hipError_t launch_moe_dispatch(const MoeRowsParams& p, hipStream_t st);
hipError_t launch_moe_combine(const MoeRowsParams& p, hipStream_t st);
hipError_t launch_moe_combine_backward(const MoeRowsParams& p, hipStream_t st);
hipError_t launch_norm_forward(const NormParams& p, hipStream_t st);
hipError_t launch_norm_backward(const NormParams& p, hipStream_t st);
int64_t norm_partials(int64_t rows);
hipError_t launch_rms_forward(const RmsParams& p, hipStream_t st);
hipError_t launch_rms_quantize(const RmsParams& p, hipStream_t st);
hipError_t launch_rms_backward(const RmsParams& p, hipStream_t st);
int64_t rms_partials(int64_t rows, int64_t cols);
hipError_t launch_route(const RouteParams& p, hipStream_t st);
hipError_t launch_route_backward(const RouteParams& p, hipStream_t st);
int64_t route_blocks(int64_t tokens, int64_t experts);
int64_t route_workspace(int64_t tokens, int64_t experts);

}  // namespace fp8mi
