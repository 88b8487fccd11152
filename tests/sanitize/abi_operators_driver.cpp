// Host-only driver for the argument validation of the layer norm's and the
// experts' C entry points (api_norm.cpp, api_moe.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_sanitize_operators.py.  The kernel launchers are replaced by stubs
// that record what reached them; no GPU and no HIP runtime is involved.
#include <stdint.h>
#include <stdio.h>

#include <limits>
#include <vector>

#include "fp8mi.h"
#include "launch.hpp"

namespace {
int g_launches = 0;
int g_failures = 0;
fp8mi::NormParams g_norm;
fp8mi::MoeSortParams g_sort;
fp8mi::MoeRowsParams g_rows;
fp8mi::MoeQuantParams g_quant;
fp8mi::GroupedGemmParams g_gemm;

void expect(int64_t got, int64_t want, const char* what, int line) {
  if (got != want) {
    ++g_failures;
    printf("FAIL line %d: %s -> %lld, expected %lld\n", line, what, (long long)got, (long long)want);
  }
}
#define EXPECT(call, want) expect((int64_t)(call), (want), #call, __LINE__)

// aligned stand-ins for device pointers: neither the validation nor the stubs
// dereference them
alignas(64) unsigned char g_buf[64];
void* const P = g_buf;
float* const F = reinterpret_cast<float*>(g_buf);
int32_t* const I = reinterpret_cast<int32_t*>(g_buf);
uint8_t* const U = g_buf;
constexpr int64_t kMax = std::numeric_limits<int64_t>::max();
constexpr int64_t kMin = std::numeric_limits<int64_t>::min();
}  // namespace

namespace fp8mi {
#define STUB(name, type, to)                    \
  hipError_t name(const type& p, hipStream_t) { \
    ++g_launches;                               \
    to = p;                                     \
    return hipSuccess;                          \
  }
STUB(launch_norm_forward, NormParams, g_norm)
STUB(launch_norm_backward, NormParams, g_norm)
STUB(launch_moe_sort, MoeSortParams, g_sort)
STUB(launch_moe_dispatch, MoeRowsParams, g_rows)
STUB(launch_moe_combine, MoeRowsParams, g_rows)
STUB(launch_moe_combine_backward, MoeRowsParams, g_rows)
STUB(launch_moe_quantize, MoeQuantParams, g_quant)
STUB(launch_gemm_grouped, GroupedGemmParams, g_gemm)
// the most that these say
int64_t norm_partials(int64_t) { return 512; }
int64_t moe_sort_blocks(int64_t slots) { return slots > 2048 ? 256 : 1; }
int hip_status(hipError_t e) { return e == hipSuccess ? FP8MI_OK : FP8MI_ERR_HIP; }
}  // namespace fp8mi

namespace {

using Args = std::vector<int64_t>;

// Every one and every two of the size arguments at the ends of their types:
// each call ends in a status, with no overflow on the way (the sanitizer's
// part), and what reaches a launcher has sizes a launch can have.
template <typename Call, typename Sane>
void extremes(const Args& good, Call call, Sane sane, const char* what) {
  const int64_t odd[] = {kMin, -1, 0, 1, 127, 128, 1LL << 22, (1LL << 30) + 128, 1LL << 31, 1LL << 32, 1LL << 40, 1LL << 61, kMax - 127, kMax};
  auto one = [&](const Args& a) {
    const int before = g_launches;
    const int64_t st = call(a);
    const bool launched = g_launches != before;
    if (st > 0 || st < -8 || (launched && (st != FP8MI_OK || !sane()))) {
      ++g_failures;
      printf("FAIL %s(", what);
      for (int64_t v : a) printf(" %lld", (long long)v);
      printf(") -> %lld, launched %d\n", (long long)st, (int)launched);
    }
  };
  for (size_t i = 0; i < good.size(); ++i)
    for (int64_t v : odd) {
      Args a = good;
      a[i] = v;
      one(a);
      for (size_t j = i + 1; j < good.size(); ++j)
        for (int64_t w : odd) {
          Args b = a;
          b[j] = w;
          one(b);
        }
    }
  for (int64_t v : odd) one(Args(good.size(), v));
}

bool routing_sane(int64_t tokens, int64_t topk, int64_t experts) {
  return tokens >= 0 && topk >= 1 && topk <= (1 << 20) && experts <= FP8MI_MAX_EXPERTS && tokens * topk <= (1LL << 30);
}

int norm_forward(const Args& a) {  // rows, cols, ld_x, ld_y
  return fp8_layer_norm_forward(P, FP8MI_IN_FP32, a[0], a[1], a[2], P, P, FP8MI_IN_BF16, 1e-5f, P, a[3], F, F, nullptr);
}
int norm_backward(const Args& a) {  // rows, cols, ld_dy, ld_x, ld_dx, workspace_bytes
  return fp8_layer_norm_backward(P, a[2], P, FP8MI_IN_BF16, a[0], a[1], a[3], P, FP8MI_IN_FP32, F, F, P, a[4], P, P, P, a[5], nullptr);
}
int sort(const Args& a) {  // tokens, topk, ld_expert, experts, rows, workspace_bytes
  return fp8_moe_sort(P, FP8MI_IDX_I64, a[0], a[1], a[2], a[3], I, I, I, a[4], I, P, a[5], nullptr);
}
int dispatch(const Args& a) {  // tokens, cols, ld_x, topk, experts, rows, ld_y
  return fp8_moe_dispatch(P, FP8MI_IN_FP32, a[0], a[1], a[2], a[3], F, I, I, I, a[4], P, a[5], a[6], nullptr);
}
int combine(const Args& a) {  // rows, cols, ld_ys, tokens, topk, ld_y
  return fp8_moe_combine(P, FP8MI_IN_FP32, a[0], a[1], a[2], I, a[3], a[4], F, P, a[5], nullptr);
}
int combine_backward(const Args& a) {  // tokens, cols, ld_dy, ld_ys, experts, topk, rows, ld_dys
  return fp8_moe_combine_backward(P, FP8MI_IN_FP32, a[0], a[1], a[2], P, a[3], I, I, I, a[4], a[5], F, P, a[6], a[7], F, nullptr);
}
int quantize(const Args& a, int32_t* row_slot, int orient) {  // x_rows, cols, ld_x, topk, experts, rows, ld_q_row, ld_q_col
  return fp8_moe_quantize(P, FP8MI_IN_FP32, a[0], a[1], a[2], row_slot, a[3], nullptr, I, a[4], a[5], FP8MI_BLOCK_1x128, FP8MI_E4M3,
                          orient, 0, U, a[6], P, U, a[7], P, nullptr, nullptr);
}
// lda, ldb, stride_b, ld_sb, stride_sb, experts, rows, M, N, K, ldc, stride_c
int gemm(const Args& a, int group) {
  return fp8_gemm_grouped(U, FP8MI_E4M3, P, a[0], U, FP8MI_E4M3, P, a[1], a[2], a[3], a[4],
                          group == FP8MI_GROUP_ROWS ? FP8MI_GEMM_BLOCK_1x128_128x128 : FP8MI_GEMM_BLOCK_1x128_1x128, group, I, a[5],
                          a[6], a[7], a[8], a[9], P, FP8MI_OUT_FP32, a[10], a[11], nullptr);
}

}  // namespace

int main() {
  // ---- layer norm
  EXPECT(norm_forward({8, 64, 72, 80}), FP8MI_OK);
  EXPECT(g_norm.rows == 8 && g_norm.cols == 64 && g_norm.ld_x == 72 && g_norm.ld_out == 80 && !g_norm.workspace, 1);
  EXPECT(norm_backward({8, 64, 65, 66, 67, 512 * 2 * 64 * 4}), FP8MI_OK);
  EXPECT(g_norm.ld_dy == 65 && g_norm.ld_x == 66 && g_norm.ld_out == 67 && g_norm.workspace == F, 1);
  EXPECT(norm_backward({8, 64, 65, 66, 67, 512 * 2 * 64 * 4 - 1}), FP8MI_ERR_SHAPE);
  EXPECT(norm_backward({1, 1LL << 28, 1LL << 28, 1LL << 28, 1LL << 28, kMax}), FP8MI_OK);
  EXPECT(norm_backward({1, (1LL << 28) + 1, 1LL << 29, 1LL << 29, 1LL << 29, kMax}), FP8MI_ERR_UNSUPPORTED);
  auto norm_sane = [] { return g_norm.rows >= 0 && g_norm.cols >= 1 && g_norm.cols <= (1LL << 28); };
  extremes({8, 64, 64, 64}, norm_forward, norm_sane, "norm_forward");
  extremes({8, 64, 64, 64, 64, 1 << 20}, norm_backward, norm_sane, "norm_backward");
  extremes({8, 64}, [](const Args& a) { return fp8_layer_norm_workspace(a[0], a[1]) < 0 ? -1 : 0; }, [] { return true; }, "workspace");

  // ---- sort
  EXPECT(fp8_moe_rows(100, 2, 8), 1152);
  EXPECT(sort({100, 2, 3, 8, 1152, 0}), FP8MI_OK);
  EXPECT(g_sort.tokens == 100 && g_sort.topk == 2 && g_sort.ld_expert == 3 && g_sort.rows == 1152, 1);
  EXPECT(sort({1LL << 30, 1, 1, 1024, (1LL << 30) + 1024 * 128, 256 * 1024 * 4}), FP8MI_OK);
  EXPECT(sort({1LL << 30, 1, 1, 1024, (1LL << 30) + 1024 * 128, 256 * 1024 * 4 - 1}), FP8MI_ERR_SHAPE);
  EXPECT(sort({(1LL << 30) + 1, 1, 1, 1024, 1LL << 31, kMax}), FP8MI_ERR_UNSUPPORTED);
  extremes({100, 2, 2, 8, 1152, 1 << 20}, sort,
           [] { return routing_sane(g_sort.tokens, g_sort.topk, g_sort.experts) && g_sort.rows <= 0x7FFFFF00; }, "sort");
  extremes({100, 2, 8}, [](const Args& a) { return fp8_moe_rows(a[0], a[1], a[2]) < 0 ? -1 : 0; }, [] { return true; }, "rows");
  extremes({100, 2, 8}, [](const Args& a) { return fp8_moe_sort_workspace(a[0], a[1], a[2]) < 0 ? -1 : 0; }, [] { return true; }, "sort_workspace");

  // ---- rows to and from the sorted buffer
  EXPECT(dispatch({100, 64, 65, 2, 8, 1152, 66}), FP8MI_OK);
  EXPECT(g_rows.tokens == 100 && g_rows.cols == 64 && g_rows.ld_token == 65 && g_rows.ld_out == 66 && g_rows.slot_row == I, 1);
  EXPECT(dispatch({1LL << 30, 1, 1, 1, 1, 1LL << 30, 1}), FP8MI_OK);  // as many tokens as are documented
  EXPECT(dispatch({1LL << 22, 1 << 19, 1 << 19, 1, 1, 1LL << 22, 1 << 19}), FP8MI_OK);
  EXPECT(dispatch({1LL << 22, (1 << 19) + 1, 1 << 20, 1, 1, 1LL << 22, 1 << 20}), FP8MI_ERR_UNSUPPORTED);
  auto rows_sane = [] {
    return routing_sane(g_rows.tokens, g_rows.topk, 1) && g_rows.rows <= 0x7FFFFF00 && g_rows.rows % 128 == 0 && g_rows.cols >= 0 &&
           g_rows.cols <= (1LL << 28);
  };
  extremes({100, 64, 64, 2, 8, 1152, 64}, dispatch, rows_sane, "dispatch");
  EXPECT(combine({1152, 64, 65, 100, 2, 66}), FP8MI_OK);
  EXPECT(g_rows.ld_expert == 65 && g_rows.ld_out == 66 && g_rows.tokens == 100 && !g_rows.offsets, 1);
  extremes({1152, 64, 64, 100, 2, 64}, combine, rows_sane, "combine");
  EXPECT(combine_backward({100, 64, 65, 66, 8, 2, 1152, 67}), FP8MI_OK);
  EXPECT(g_rows.ld_token == 65 && g_rows.ld_expert == 66 && g_rows.ld_out == 67 && g_rows.dweights == F, 1);
  EXPECT(combine_backward({1LL << 30, 8, 8, 8, 1, 1, 1LL << 30, 8}), FP8MI_OK);
  extremes({100, 64, 64, 64, 8, 2, 1152, 64}, combine_backward, rows_sane, "combine_backward");

  // ---- dispatch into codes
  EXPECT(quantize({100, 64, 68, 2, 8, 1152, 80, 1168}, I, FP8MI_ROW_AND_COL), FP8MI_OK);
  EXPECT(g_quant.q.rows == 1152 && g_quant.q.ld_x == 68 && g_quant.x_rows == 100 && g_quant.topk == 2 && g_quant.q.ld_q_col == 1168, 1);
  EXPECT(quantize({1152, 64, 64, 2, 8, 1152, 64, 0}, nullptr, FP8MI_ROW), FP8MI_OK);
  EXPECT(quantize({1151, 64, 64, 2, 8, 1152, 64, 0}, nullptr, FP8MI_ROW), FP8MI_ERR_SHAPE);
  auto quant_sane = [] { return g_quant.q.rows % 128 == 0 && g_quant.x_rows <= 0x7FFFFFFF && g_quant.q.cols > 0 && g_quant.topk >= 1; };
  for (int orient : {FP8MI_ROW, FP8MI_COL, FP8MI_ROW_AND_COL})
    for (int32_t* slots : {I, (int32_t*)nullptr})
      extremes({1152, 64, 64, 2, 8, 1152, 64, 1152}, [=](const Args& a) { return quantize(a, slots, orient); }, quant_sane, "quantize");

  // ---- products
  EXPECT(gemm({256, 272, 256 * 128, 2, 2, 8, 1152, 0, 128, 256, 130, 0}, FP8MI_GROUP_ROWS), FP8MI_OK);
  EXPECT(!g_gemm.contract && g_gemm.R == 1152 && g_gemm.K == 256 && g_gemm.ldb == 272 && g_gemm.ldc == 130, 1);
  EXPECT(gemm({1152, 1168, 0, 0, 0, 8, 1152, 64, 128, 0, 128, 64 * 128}, FP8MI_GROUP_CONTRACT), FP8MI_OK);
  EXPECT(g_gemm.contract && g_gemm.M == 64 && g_gemm.N == 128 && g_gemm.stride_c == 64 * 128, 1);
  EXPECT(gemm({1152, 1152, 0, 0, 0, 8, 1152, 64, 128, 0, 8 * 128, 128}, FP8MI_GROUP_CONTRACT), FP8MI_OK);  // rows in turn
  EXPECT(gemm({1152, 1152, 0, 0, 0, 8, 1152, 64, 128, 0, 8 * 128 - 1, 128}, FP8MI_GROUP_CONTRACT), FP8MI_ERR_SHAPE);
  EXPECT(gemm({0, 0, 0, 0, 0, 8, 0, 64, 128, 0, 128, 64 * 128}, FP8MI_GROUP_CONTRACT), FP8MI_OK);  // no rows: zeros
  auto gemm_sane = [] {
    return g_gemm.R <= 0x7FFFFF00 && g_gemm.M <= 0x7FFFFFFF && g_gemm.N <= 0x7FFFFFFF && g_gemm.K <= 0x7FFFFFFF &&
           (g_gemm.K + g_gemm.R == 0 || (g_gemm.contract && g_gemm.R == 0) || (!g_gemm.contract && g_gemm.K == 0) ||
            (g_gemm.lda <= (1 << 22) && g_gemm.ldb <= (1 << 22)));
  };
  extremes({256, 256, 256 * 128, 2, 2, 8, 1152, 64, 128, 256, 128, 64 * 128},
           [](const Args& a) { return gemm(a, FP8MI_GROUP_ROWS); }, gemm_sane, "gemm rows");
  extremes({1152, 1152, 256 * 128, 2, 2, 8, 1152, 64, 128, 256, 128, 64 * 128},
           [](const Args& a) { return gemm(a, FP8MI_GROUP_CONTRACT); }, gemm_sane, "gemm contract");

  if (g_failures) {
    printf("%d failure(s)\n", g_failures);
    return 1;
  }
  printf("operator validation ok\n");
  return 0;
}
