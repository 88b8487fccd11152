// Host-only driver for the argument validation of the RMS norm's and the
// router's C entry points (api_rms.cpp, api_route.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_sanitize_rms_route.py.  The kernel launchers are replaced by stubs
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
fp8mi::RmsParams g_rms;
fp8mi::RouteParams g_route;

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
STUB(launch_rms_forward, RmsParams, g_rms)
STUB(launch_rms_quantize, RmsParams, g_rms)
STUB(launch_rms_backward, RmsParams, g_rms)
STUB(launch_route, RouteParams, g_route)
STUB(launch_route_backward, RouteParams, g_route)
// the most that these say
int64_t rms_partials(int64_t, int64_t cols) { return cols <= 1024 ? 2048 : 512; }
int64_t route_workspace(int64_t, int64_t experts) { return 4 * (256 * (2 * experts + 1) + 33); }
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
  one(good);
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

int rms_forward(const Args& a) {  // rows, cols, ld_x, ld_residual, ld_total, ld_y
  return fp8_rms_norm_forward(P, FP8MI_IN_FP32, a[0], a[1], a[2], P, a[3], P, FP8MI_IN_BF16, 1e-6f, P, a[4], P, a[5], F, nullptr);
}
int rms_quantize(const Args& a) {  // rows, cols, ld_x, ld_residual, ld_total, ld_q_row, ld_q_col, margin
  return fp8_rms_norm_quantize(P, FP8MI_IN_BF16, a[0], a[1], a[2], P, a[3], P, FP8MI_IN_FP32, 1e-6f, P, a[4], F, FP8MI_MX_1x32,
                               FP8MI_E5M2, FP8MI_ROW_AND_COL, (int)a[7], U, a[5], U, U, a[6], U, nullptr, nullptr, I, nullptr);
}
int rms_backward(const Args& a) {  // rows, cols, ld_dy, ld_total, ld_dtotal, ld_dx, workspace_bytes
  return fp8_rms_norm_backward(P, a[2], P, FP8MI_IN_BF16, a[0], a[1], a[3], P, FP8MI_IN_FP32, F, P, a[4], P, a[5], P, P, a[6], nullptr);
}
bool rms_sane() {
  const auto& p = g_rms;
  return p.rows >= 0 && p.cols >= 1 && p.cols <= (1LL << 28) &&
         (p.rows == 0 || (p.ld_x >= p.cols && p.rows <= kMax / 2 / p.ld_x && (!p.residual || p.ld_residual >= p.cols)));
}
int route(const Args& a) {  // tokens, experts, ld_logits, topk, workspace_bytes
  return fp8_moe_route(P, FP8MI_IN_BF16, a[0], a[1], a[2], U, a[3], 1, I, F, F, I, F, P, a[4], nullptr);
}
int balance(const Args& a) {  // tokens, experts, ld_logits, topk, ld_expert, workspace_bytes
  return fp8_moe_balance(P, FP8MI_IN_FP32, a[0], a[1], a[2], U, P, FP8MI_IDX_I64, a[3], a[4], F, I, F, P, a[5], nullptr);
}
int route_backward(const Args& a) {  // tokens, experts, ld_logits, topk, ld_dlogits
  return fp8_moe_route_backward(P, FP8MI_IN_FP32, a[0], a[1], a[2], U, I, a[3], F, 0, F, F, P, a[4], nullptr);
}
bool route_sane() {
  const auto& p = g_route;
  return p.tokens >= 0 && p.experts >= 1 && p.experts <= FP8MI_MAX_EXPERTS && p.topk >= 1 && p.tokens * p.topk <= (1LL << 30) &&
         (p.tokens == 0 || (p.ld >= p.experts && p.tokens <= kMax / 2 / p.ld));
}

}  // namespace

int main() {
  extremes({100, 64, 64, 64, 64, 64}, rms_forward, rms_sane, "rms_norm_forward");
  extremes({100, 64, 64, 64, 64, 64, 112, 0}, rms_quantize, rms_sane, "rms_norm_quantize");
  extremes({100, 64, 64, 64, 64, 64, 1 << 20}, rms_backward, rms_sane, "rms_norm_backward");
  extremes({100, 8, 8, 2, 1 << 20}, route, route_sane, "moe_route");
  extremes({100, 8, 8, 2, 2, 1 << 20}, balance, route_sane, "moe_balance");
  extremes({100, 8, 8, 2, 8}, route_backward, route_sane, "moe_route_backward");
  const int64_t odd[] = {kMin, -1, 0, 1, 1024, 1025, 1LL << 28, 1LL << 30, 1LL << 31, 1LL << 40, kMax};
  for (int64_t a : odd)
    for (int64_t b : odd) {
      if (fp8_rms_norm_workspace(a, b) < -8 || fp8_moe_route_workspace(a, b) < -8) ++g_failures;
    }
  if (!g_launches || g_failures) {
    printf("%d failures, %d launches\n", g_failures, g_launches);
    return 1;
  }
  printf("rms and route validation ok\n");
  return 0;
}
