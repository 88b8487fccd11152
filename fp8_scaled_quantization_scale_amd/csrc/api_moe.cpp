// api_moe.cpp -- the C ABI's expert path (include/fp8mi.h): the sort of tokens
// by expert, dispatch, combine and its gradient, and the grouped FP8 GEMM.
// Argument checks (no HIP call is made before they pass) and dispatch to the
// launchers.
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

// tokens, choices and experts that every entry point takes
int check_routing(int64_t tokens, int64_t topk, int64_t experts) {
  if (tokens < 0 || topk < 1 || experts < 1) return FP8MI_ERR_SHAPE;
  if (experts > FP8MI_MAX_EXPERTS || topk > (1 << 20) || tokens > (1LL << 30) || tokens * topk > (1LL << 30))
    return FP8MI_ERR_UNSUPPORTED;
  return FP8MI_OK;
}

int check_rows(int64_t rows) {
  if (rows < 0 || rows % FP8MI_EXPERT_ALIGN) return FP8MI_ERR_SHAPE;
  return rows > 0x7FFFFF00LL ? FP8MI_ERR_UNSUPPORTED : FP8MI_OK;
}

}  // namespace

extern "C" {

int64_t fp8_moe_rows(int64_t tokens, int64_t topk, int64_t experts) {
  const int st = check_routing(tokens, topk, experts);
  if (st != FP8MI_OK) return st;
  const int64_t slots = tokens * topk, held = slots < experts ? slots : experts;
  return (slots + (FP8MI_EXPERT_ALIGN - 1) * held) / FP8MI_EXPERT_ALIGN * FP8MI_EXPERT_ALIGN;
}

int64_t fp8_moe_sort_workspace(int64_t tokens, int64_t topk, int64_t experts) {
  const int st = check_routing(tokens, topk, experts);
  if (st != FP8MI_OK) return st;
  const int64_t blocks = fp8mi::moe_sort_blocks(tokens * topk);
  return blocks > 1 ? blocks * experts * (int64_t)sizeof(int32_t) : 0;
}

int fp8_moe_sort(const void* expert, int idx_dtype, int64_t tokens, int64_t topk, int64_t ld_expert, int64_t experts,
                 int32_t* offsets, int32_t* counts, int32_t* row_slot, int64_t rows, int32_t* slot_row,
                 void* workspace, int64_t workspace_bytes, void* stream) {
  if (idx_dtype != FP8MI_IDX_I32 && idx_dtype != FP8MI_IDX_I64) return FP8MI_ERR_ENUM;
  int st = check_routing(tokens, topk, experts);
  if (st != FP8MI_OK) return st;
  if ((st = check_rows(rows)) != FP8MI_OK) return st;
  if (!offsets || !counts || (rows > 0 && !row_slot)) return FP8MI_ERR_NULL;
  if (tokens > 0 && (!expert || !slot_row)) return FP8MI_ERR_NULL;
  const int64_t es = idx_dtype == FP8MI_IDX_I32 ? 4 : 8;
  if (tokens > 0 && (ld_expert < topk || !span_ok(tokens, ld_expert, es))) return FP8MI_ERR_SHAPE;
  if (rows < fp8_moe_rows(tokens, topk, experts)) return FP8MI_ERR_SHAPE;
  const int64_t need = fp8_moe_sort_workspace(tokens, topk, experts);
  if (need > 0 && !workspace) return FP8MI_ERR_NULL;
  if (workspace_bytes < need) return FP8MI_ERR_SHAPE;
  if (!aligned_to(expert, es) || !aligned_to(offsets, 4) || !aligned_to(counts, 4) || !aligned_to(row_slot, 4) ||
      !aligned_to(slot_row, 4) || !aligned_to(workspace, 4))
    return FP8MI_ERR_ALIGN;
  fp8mi::MoeSortParams p{expert, idx_dtype, tokens, topk, ld_expert, experts, offsets, counts, row_slot, slot_row,
                         rows, static_cast<int32_t*>(workspace)};
  return fp8mi::hip_status(fp8mi::launch_moe_sort(p, (hipStream_t)stream));
}

int fp8_moe_dispatch(const void* x, int dtype, int64_t tokens, int64_t cols, int64_t ld_x, int64_t topk,
                     const float* weights, const int32_t* slot_row, const int32_t* offsets, const int32_t* counts,
                     int64_t experts, void* y, int64_t rows, int64_t ld_y, void* stream) {
  if (!in_dtype_ok(dtype)) return FP8MI_ERR_ENUM;
  int st = check_routing(tokens, topk, experts);
  if (st != FP8MI_OK) return st;
  if ((st = check_rows(rows)) != FP8MI_OK) return st;
  if (cols < 0) return FP8MI_ERR_SHAPE;
  if (tokens == 0 || cols == 0 || rows == 0) return FP8MI_OK;
  if (cols > (1LL << 28) || tokens * ((cols + 1023) / 1024) > (1LL << 31)) return FP8MI_ERR_UNSUPPORTED;
  if (!slot_row || !offsets || !counts) return FP8MI_ERR_NULL;
  if ((st = check_matrix(x, tokens, cols, ld_x, in_size(dtype))) != FP8MI_OK) return st;
  if ((st = check_matrix(y, rows, cols, ld_y, in_size(dtype))) != FP8MI_OK) return st;
  if (!aligned_to(weights, 4) || !aligned_to(slot_row, 4) || !aligned_to(offsets, 4) || !aligned_to(counts, 4))
    return FP8MI_ERR_ALIGN;
  fp8mi::MoeRowsParams p{dtype, tokens, topk, experts, cols, rows, offsets, counts, slot_row, weights,
                         x, ld_x, nullptr, 0, y, ld_y, nullptr};
  return fp8mi::hip_status(fp8mi::launch_moe_dispatch(p, (hipStream_t)stream));
}

int fp8_moe_quantize(const void* x, int x_dtype, int64_t x_rows, int64_t cols, int64_t ld_x, const int32_t* row_slot,
                     int64_t topk, const float* weights, const int32_t* offsets, int64_t experts, int64_t rows,
                     int recipe, int fmt, int orient, int margin, uint8_t* q_row, int64_t ld_q_row, void* s_row,
                     uint8_t* q_col, int64_t ld_q_col, void* s_col, int32_t* nonfinite, void* stream) {
  if (!in_dtype_ok(x_dtype)) return FP8MI_ERR_ENUM;
  if (recipe < FP8MI_TENSOR_CURRENT || recipe > FP8MI_MX_1x32_OCP) return FP8MI_ERR_ENUM;
  if (fmt != FP8MI_E4M3 && fmt != FP8MI_E5M2) return FP8MI_ERR_ENUM;
  if (orient != FP8MI_ROW && orient != FP8MI_COL && orient != FP8MI_ROW_AND_COL) return FP8MI_ERR_ENUM;
  // scales that are local to a row or to a 128-row block only
  if (recipe != FP8MI_BLOCK_1x128 && recipe != FP8MI_MX_1x32 && recipe != FP8MI_MX_1x32_OCP)
    return FP8MI_ERR_UNSUPPORTED;
  if (x_rows < 0 || cols < 0 || margin < 0 || margin > 64) return FP8MI_ERR_SHAPE;
  int st = check_routing(0, row_slot ? topk : 1, experts);
  if (st != FP8MI_OK) return st;
  if ((st = check_rows(rows)) != FP8MI_OK) return st;
  if (!row_slot && (weights || x_rows < rows)) return FP8MI_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP8MI_OK;
  const bool row = orient & FP8MI_ROW, col = orient & FP8MI_COL;
  if (!offsets || (x_rows > 0 && !x)) return FP8MI_ERR_NULL;
  if ((row && (!q_row || !s_row)) || (col && (!q_col || !s_col))) return FP8MI_ERR_NULL;
  const int64_t es = in_size(x_dtype);
  if (ld_x < cols || (row && ld_q_row < cols) || (col && ld_q_col < rows)) return FP8MI_ERR_SHAPE;
  if (!span_ok(x_rows, ld_x, es) || (row && !span_ok(rows, ld_q_row, 1)) || (col && !span_ok(cols, ld_q_col, 1)))
    return FP8MI_ERR_SHAPE;
  if (x_rows > 0x7FFFFFFFLL || (cols + 127) / 128 > 0x7FFFFFFFLL / (rows / 128)) return FP8MI_ERR_UNSUPPORTED;
  if (!aligned_to(x, 16) || ld_x % (16 / es) || (row && (!aligned_to(q_row, 16) || ld_q_row % 16)) ||
      (col && (!aligned_to(q_col, 16) || ld_q_col % 16)) || !aligned_to(offsets, 4) || !aligned_to(row_slot, 4) ||
      !aligned_to(weights, 4))
    return FP8MI_ERR_ALIGN;
  fp8mi::MoeQuantParams p{{x, x_dtype, rows, cols, ld_x, recipe, fmt, orient, margin, q_row, ld_q_row, s_row, q_col,
                           ld_q_col, s_col, nullptr, nullptr, nullptr, nonfinite},
                          offsets, row_slot, weights, experts, row_slot ? topk : 1, x_rows};
  return fp8mi::hip_status(fp8mi::launch_moe_quantize(p, (hipStream_t)stream));
}

int fp8_moe_combine(const void* ys, int dtype, int64_t rows, int64_t cols, int64_t ld_ys, const int32_t* slot_row,
                    int64_t tokens, int64_t topk, const float* weights, void* y, int64_t ld_y, void* stream) {
  if (!in_dtype_ok(dtype)) return FP8MI_ERR_ENUM;
  int st = check_routing(tokens, topk, 1);
  if (st != FP8MI_OK) return st;
  if ((st = check_rows(rows)) != FP8MI_OK) return st;
  if (cols < 0) return FP8MI_ERR_SHAPE;
  if (tokens == 0 || cols == 0) return FP8MI_OK;
  if (cols > (1LL << 28) || tokens * ((cols + 1023) / 1024) > (1LL << 31)) return FP8MI_ERR_UNSUPPORTED;
  if (!slot_row) return FP8MI_ERR_NULL;
  if (rows > 0 && (st = check_matrix(ys, rows, cols, ld_ys, in_size(dtype))) != FP8MI_OK) return st;
  if ((st = check_matrix(y, tokens, cols, ld_y, in_size(dtype))) != FP8MI_OK) return st;
  if (!aligned_to(weights, 4) || !aligned_to(slot_row, 4)) return FP8MI_ERR_ALIGN;
  fp8mi::MoeRowsParams p{dtype, tokens, topk, 0, cols, rows, nullptr, nullptr, slot_row, weights,
                         nullptr, 0, ys, ld_ys, y, ld_y, nullptr};
  return fp8mi::hip_status(fp8mi::launch_moe_combine(p, (hipStream_t)stream));
}

int fp8_moe_combine_backward(const void* dy, int dtype, int64_t tokens, int64_t cols, int64_t ld_dy, const void* ys,
                             int64_t ld_ys, const int32_t* slot_row, const int32_t* offsets, const int32_t* counts,
                             int64_t experts, int64_t topk, const float* weights, void* dys, int64_t rows,
                             int64_t ld_dys, float* dweights, void* stream) {
  if (!in_dtype_ok(dtype)) return FP8MI_ERR_ENUM;
  int st = check_routing(tokens, topk, experts);
  if (st != FP8MI_OK) return st;
  if ((st = check_rows(rows)) != FP8MI_OK) return st;
  if (cols < 0) return FP8MI_ERR_SHAPE;
  if (tokens == 0 || (!dys && !dweights)) return FP8MI_OK;
  if (cols > (1LL << 28)) return FP8MI_ERR_UNSUPPORTED;
  if (!slot_row || (dys && (!offsets || !counts))) return FP8MI_ERR_NULL;
  const int64_t es = in_size(dtype);
  if (cols > 0) {
    if ((st = check_matrix(dy, tokens, cols, ld_dy, es)) != FP8MI_OK) return st;
    if (rows > 0 && dweights && (st = check_matrix(ys, rows, cols, ld_ys, es)) != FP8MI_OK) return st;
    if (rows > 0 && dys && (st = check_matrix(dys, rows, cols, ld_dys, es)) != FP8MI_OK) return st;
  }
  if (!aligned_to(weights, 4) || !aligned_to(slot_row, 4) || !aligned_to(offsets, 4) || !aligned_to(counts, 4) ||
      !aligned_to(dweights, 4))
    return FP8MI_ERR_ALIGN;
  fp8mi::MoeRowsParams p{dtype, tokens, topk, experts, cols, rows, offsets, counts, slot_row, weights,
                         dy, ld_dy, ys, ld_ys, dys, ld_dys, dweights};
  return fp8mi::hip_status(fp8mi::launch_moe_combine_backward(p, (hipStream_t)stream));
}

int fp8_gemm_grouped(const uint8_t* a, int fmt_a, const void* s_a, int64_t lda, const uint8_t* b, int fmt_b,
                     const void* s_b, int64_t ldb, int64_t stride_b, int64_t ld_sb, int64_t stride_sb, int recipe,
                     int group, const int32_t* offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, int64_t K,
                     void* c, int c_dtype, int64_t ldc, int64_t stride_c, void* stream) {
  if (fmt_a != FP8MI_E4M3 && fmt_a != FP8MI_E5M2) return FP8MI_ERR_ENUM;
  if (fmt_b != FP8MI_E4M3 && fmt_b != FP8MI_E5M2) return FP8MI_ERR_ENUM;
  if (recipe < FP8MI_GEMM_TENSOR || recipe > FP8MI_GEMM_CHANNEL) return FP8MI_ERR_ENUM;
  if (group != FP8MI_GROUP_ROWS && group != FP8MI_GROUP_CONTRACT) return FP8MI_ERR_ENUM;
  if (c_dtype != FP8MI_OUT_BF16 && c_dtype != FP8MI_OUT_FP32) return FP8MI_ERR_ENUM;
  const bool contract = group == FP8MI_GROUP_CONTRACT, mx = recipe == FP8MI_GEMM_MX_1x32;
  if (!mx && recipe != (contract ? FP8MI_GEMM_BLOCK_1x128_1x128 : FP8MI_GEMM_BLOCK_1x128_128x128))
    return FP8MI_ERR_UNSUPPORTED;
  int st = check_routing(0, 1, experts);
  if (st != FP8MI_OK) return st;
  if ((st = check_rows(rows)) != FP8MI_OK) return st;
  if (N < 0 || (contract ? M < 0 : K < 0)) return FP8MI_ERR_SHAPE;
  // from here on: M output rows of the largest product, K its contraction
  const int64_t m = contract ? M : rows, k = contract ? rows : K;
  if (m == 0 || N == 0) return FP8MI_OK;
  if (!c || !offsets) return FP8MI_ERR_NULL;
  const int64_t cs = c_dtype == FP8MI_OUT_FP32 ? 4 : 2;
  if (ldc < N || !span_ok(m, ldc, cs)) return FP8MI_ERR_SHAPE;
  if (contract) {
    if (stride_c < 0 || !span_ok(experts, stride_c, cs)) return FP8MI_ERR_SHAPE;
  }
  if (!aligned_to(offsets, 4) || !aligned_to(c, cs)) return FP8MI_ERR_ALIGN;
  if (k > 0) {
    if (!a || !b || !s_a || !s_b) return FP8MI_ERR_NULL;
    if (k % 16 || lda < k || ldb < k) return FP8MI_ERR_SHAPE;
    if (!aligned_to(a, 16) || !aligned_to(b, 16) || lda % 16 || ldb % 16) return FP8MI_ERR_ALIGN;
    if (!aligned_to(s_a, 4) || !aligned_to(s_b, 4)) return FP8MI_ERR_ALIGN;
    // operand panels and scale panels are addressed with 32-bit buffer offsets
    if (lda > (1LL << 22) || ldb > (1LL << 22)) return FP8MI_ERR_UNSUPPORTED;
    if (!contract) {
      const int64_t per_row = mx ? (k + 31) / 32 : (k + 127) / 128;
      if (stride_b < 0 || stride_b % 16 || stride_sb < 0 || ld_sb < per_row) return FP8MI_ERR_SHAPE;
      if (ld_sb > (1LL << 22)) return FP8MI_ERR_UNSUPPORTED;
      if (!span_ok(experts, stride_b, 1) || !span_ok(experts, stride_sb, 4)) return FP8MI_ERR_SHAPE;
    }
  }
  if (m > 0x7FFFFFFFLL || N > 0x7FFFFFFFLL || k > 0x7FFFFFFFLL) return FP8MI_ERR_UNSUPPORTED;
  // the persistent grid numbers all experts' 256 x 256 tiles with 32-bit ints
  const int64_t tm = contract ? (m + 255) / 256 * experts : m / 256 + experts, tn = (N + 255) / 256;
  if (tm > 0x7FFFFFFFLL / tn) return FP8MI_ERR_UNSUPPORTED;
  // no element of C in two experts' products: one after the other, or row by row in turn
  if (contract && experts > 1 && stride_c < (m - 1) * ldc + N && (stride_c < N || (experts - 1) * stride_c + N > ldc))
    return FP8MI_ERR_SHAPE;
  fp8mi::GroupedGemmParams p{contract, a, fmt_a, s_a, lda, b, fmt_b, s_b, ldb, stride_b, ld_sb, stride_sb, recipe,
                             offsets, experts, rows, contract ? M : 0, N, contract ? 0 : K, c, c_dtype, ldc, stride_c};
  return fp8mi::hip_status(fp8mi::launch_gemm_grouped(p, (hipStream_t)stream));
}

}  // extern "C"
