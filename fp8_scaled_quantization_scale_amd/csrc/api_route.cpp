// api_route.cpp -- the C ABI's router (include/fp8mi.h): argument checks (no HIP
// call is made before they pass) and dispatch to the launchers.
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

int check_routing(int dtype, int64_t tokens, int64_t experts, int64_t topk) {
  if (!in_dtype_ok(dtype)) return FP8MI_ERR_ENUM;
  if (tokens < 0 || topk < 1 || experts < 1) return FP8MI_ERR_SHAPE;
  if (experts > FP8MI_MAX_EXPERTS || topk > (1 << 20) || tokens > (1LL << 30) || tokens * topk > (1LL << 30))
    return FP8MI_ERR_UNSUPPORTED;
  return FP8MI_OK;
}

int check_sums(int64_t tokens, int64_t experts, const float* loss, const int32_t* counts, const float* slope,
               const void* workspace, int64_t workspace_bytes) {
  const int64_t need = fp8_moe_route_workspace(tokens, experts);
  if (!loss || !counts || !slope || (need > 0 && !workspace)) return FP8MI_ERR_NULL;
  if (workspace_bytes < need) return FP8MI_ERR_SHAPE;
  return aligned_to(loss, 4) && aligned_to(counts, 4) && aligned_to(slope, 4) && aligned_to(workspace, 4)
             ? FP8MI_OK
             : FP8MI_ERR_ALIGN;
}

}  // namespace

extern "C" {

int64_t fp8_moe_route_workspace(int64_t tokens, int64_t experts) {
  const int st = check_routing(FP8MI_IN_FP32, tokens, experts, 1);
  if (st != FP8MI_OK) return st;
  return fp8mi::route_workspace(tokens, experts);
}

int fp8_moe_route(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld_logits,
                  const uint8_t* mask, int64_t topk, int normalize, int32_t* expert, float* weights, float* loss,
                  int32_t* counts, float* slope, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_routing(dtype, tokens, experts, topk);
  if (st != FP8MI_OK) return st;
  if (topk > experts) return FP8MI_ERR_SHAPE;
  if ((st = check_sums(tokens, experts, loss, counts, slope, workspace, workspace_bytes)) != FP8MI_OK) return st;
  if (tokens > 0) {
    if ((st = check_matrix(logits, tokens, experts, ld_logits, in_size(dtype))) != FP8MI_OK) return st;
    if (!expert || !weights) return FP8MI_ERR_NULL;
    if (!aligned_to(expert, 4) || !aligned_to(weights, 4)) return FP8MI_ERR_ALIGN;
  }
  fp8mi::RouteParams p{};
  p.logits = logits;
  p.dtype = dtype;
  p.tokens = tokens;
  p.experts = experts;
  p.ld = ld_logits;
  p.mask = mask;
  p.topk = topk;
  p.normalize = normalize != 0;
  p.expert = expert;
  p.weights = weights;
  p.loss = loss;
  p.counts = counts;
  p.slope = slope;
  p.workspace = workspace;
  return fp8mi::hip_status(fp8mi::launch_route(p, (hipStream_t)stream));
}

int fp8_moe_balance(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld_logits,
                    const uint8_t* mask, const void* expert, int idx_dtype, int64_t topk, int64_t ld_expert,
                    float* loss, int32_t* counts, float* slope, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  int st = check_routing(dtype, tokens, experts, topk);
  if (st != FP8MI_OK) return st;
  if (idx_dtype != FP8MI_IDX_I32 && idx_dtype != FP8MI_IDX_I64) return FP8MI_ERR_ENUM;
  if ((st = check_sums(tokens, experts, loss, counts, slope, workspace, workspace_bytes)) != FP8MI_OK) return st;
  if (tokens > 0) {
    if ((st = check_matrix(logits, tokens, experts, ld_logits, in_size(dtype))) != FP8MI_OK) return st;
    if ((st = check_matrix(expert, tokens, topk, ld_expert, idx_dtype == FP8MI_IDX_I32 ? 4 : 8)) != FP8MI_OK) return st;
  }
  fp8mi::RouteParams p{};
  p.logits = logits;
  p.dtype = dtype;
  p.tokens = tokens;
  p.experts = experts;
  p.ld = ld_logits;
  p.mask = mask;
  p.topk = topk;
  p.given = true;
  p.chosen = expert;
  p.idx_dtype = idx_dtype;
  p.ld_chosen = ld_expert;
  p.loss = loss;
  p.counts = counts;
  p.slope = slope;
  p.workspace = workspace;
  return fp8mi::hip_status(fp8mi::launch_route(p, (hipStream_t)stream));
}

int fp8_moe_route_backward(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld_logits,
                           const uint8_t* mask, const int32_t* expert, int64_t topk, const float* dweights,
                           int normalize, const float* slope, const float* dloss, void* dlogits, int64_t ld_dlogits,
                           void* stream) {
  int st = check_routing(dtype, tokens, experts, topk);
  if (st != FP8MI_OK) return st;
  if (dweights && topk > experts) return FP8MI_ERR_SHAPE;
  if (tokens == 0) return FP8MI_OK;
  if ((st = check_matrix(logits, tokens, experts, ld_logits, in_size(dtype))) != FP8MI_OK) return st;
  if ((st = check_matrix(dlogits, tokens, experts, ld_dlogits, in_size(dtype))) != FP8MI_OK) return st;
  if ((dweights && !expert) || (dloss && !slope)) return FP8MI_ERR_NULL;
  if (!aligned_to(expert, 4) || !aligned_to(dweights, 4) || !aligned_to(slope, 4) || !aligned_to(dloss, 4))
    return FP8MI_ERR_ALIGN;
  fp8mi::RouteParams p{};
  p.logits = logits;
  p.dtype = dtype;
  p.tokens = tokens;
  p.experts = experts;
  p.ld = ld_logits;
  p.mask = mask;
  p.topk = dweights ? topk : 1;
  p.normalize = normalize != 0;
  p.expert = const_cast<int32_t*>(expert);
  p.slope = const_cast<float*>(slope);
  p.dweights = dweights;
  p.dloss = dloss;
  p.dlogits = dlogits;
  p.ld_dlogits = ld_dlogits;
  return fp8mi::hip_status(fp8mi::launch_route_backward(p, (hipStream_t)stream));
}

}  // extern "C"
