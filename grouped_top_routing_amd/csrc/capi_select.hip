// C ABI of routing from logits: argument validation and launches.
// Declarations and contracts are in include/beam_moe.h.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/beam_moe.h"
#include "capi_common.h"
#include "kernels.h"

namespace {

using namespace beam;

// The calls that choose read the groups, the others do not.
int validate_select(const moe_select_config_t* c, bool choose) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->num_tokens < 0 || c->num_experts <= 0 || c->topk <= 0) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SIGMOID && c->score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
  if (c->logits_dtype != MOE_DTYPE_BF16 && c->logits_dtype != MOE_DTYPE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (c->renormalize != 0 && c->renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (choose) {
    if (c->num_groups <= 0 || c->topk_groups <= 0 || c->topk_groups > c->num_groups ||
        c->num_experts % c->num_groups != 0 || (c->group_best != 1 && c->group_best != 2))
      return MOE_ERR_INVALID_ARG;
    if ((int64_t)c->topk > (int64_t)c->topk_groups * (c->num_experts / c->num_groups))
      return MOE_ERR_INVALID_ARG;
    if (c->num_groups > kSelectMaxGroups) return MOE_ERR_UNSUPPORTED;
  }
  if (c->num_experts > kSelectMaxExperts || c->topk > kSelectMaxTopk ||
      c->num_tokens >= (int64_t)1 << 26)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

SelectShape shape_of(const moe_select_config_t* c) {
  return SelectShape{c->num_experts, c->num_groups, c->topk_groups, c->group_best, c->topk,
                     c->score == MOE_SCORE_SOFTMAX, c->renormalize};
}

int64_t logits_bytes(const moe_select_config_t* c) {
  return c->num_tokens * c->num_experts * (c->logits_dtype == MOE_DTYPE_FP32 ? 4 : 2);
}
bool logits_aligned(const moe_select_config_t* c, const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & (c->logits_dtype == MOE_DTYPE_FP32 ? 3u : 1u)) == 0;
}
int64_t slots_bytes(const moe_select_config_t* c) { return c->num_tokens * c->topk * 4; }

}  // namespace

extern "C" {

int moe_select(const moe_select_config_t* cfg, const void* logits, const float* sel_bias,
               int32_t* topk_ids, float* topk_w, void* stream) {
  int st = validate_select(cfg, true);
  if (st) return st;
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!logits_aligned(cfg, logits) || !aligned4(sel_bias) || !aligned4(topk_ids) || !aligned4(topk_w))
    return MOE_ERR_INVALID_ARG;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!apart({{topk_ids, slots_bytes(cfg)}, {topk_w, slots_bytes(cfg)}},
             {{logits, logits_bytes(cfg)}, {sel_bias, (int64_t)cfg->num_experts * 4}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_select_experts(cfg->logits_dtype == MOE_DTYPE_FP32, logits, 1, sel_bias,
                                          topk_ids, topk_w, nullptr, cfg->num_tokens,
                                          shape_of(cfg), static_cast<hipStream_t>(stream)));
}

int moe_route_select(const moe_config_t* cfg, const moe_select_config_t* sel, const uint16_t* x,
                     const float* w_router, const float* sel_bias, int32_t* topk_ids,
                     float* topk_w, float* logits, void* workspace, size_t workspace_bytes,
                     void* stream) {
  // of cfg only the router's own sizes count
  moe_config_t c = cfg ? *cfg : moe_config_t{};
  c.num_groups = c.topk_groups = c.topk = 1;
  int st = validate(cfg ? &c : nullptr, kAnyLayout);
  if (st) return st;
  if ((st = validate_select(sel, true))) return st;
  if (sel->num_tokens != c.num_tokens || sel->num_experts != c.num_experts ||
      sel->logits_dtype != MOE_DTYPE_FP32)
    return MOE_ERR_INVALID_ARG;
  if (!x || !w_router || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned4(sel_bias) || !aligned4(topk_ids) ||
      !aligned4(topk_w) || !aligned4(logits))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ws(workspace, workspace_bytes, route_workspace(&c)))) return st;
  if (c.num_tokens == 0) return MOE_OK;
  if (!apart({{topk_ids, slots_bytes(sel)},
              {topk_w, slots_bytes(sel)},
              {logits, logits_bytes(sel)},
              {workspace, (int64_t)route_workspace(&c)}},
             {{x, c.num_tokens * c.hidden * 2},
              {w_router, (int64_t)c.num_experts * c.hidden * 4},
              {sel_bias, (int64_t)c.num_experts * 4}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const int T = (int)c.num_tokens, splits = router_splits(T, c.hidden);
  if ((st = hip_status(launch_router_logits(x, w_router, part, T, c.hidden, splits, s)))) return st;
  return hip_status(launch_select_experts(true, part, splits, sel_bias, topk_ids, topk_w, logits,
                                          T, shape_of(sel), s));
}

int moe_balance_workspace_bytes(const moe_select_config_t* cfg, size_t* bytes) {
  const int st = validate_select(cfg, false);
  if (st) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = align_up(balance_ws(cfg->num_tokens, cfg->num_experts));
  return MOE_OK;
}

int moe_balance_loss(const moe_select_config_t* cfg, const void* logits, const int32_t* topk_ids,
                     float coef, float* loss, float* load, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int st = validate_select(cfg, false);
  if (st) return st;
  if (!logits || !topk_ids || !loss || !load || !std::isfinite(coef)) return MOE_ERR_INVALID_ARG;
  if (!logits_aligned(cfg, logits) || !aligned4(topk_ids) || !aligned4(loss) || !aligned4(load))
    return MOE_ERR_INVALID_ARG;
  const size_t need = align_up(balance_ws(cfg->num_tokens, cfg->num_experts));
  if ((st = check_ws(workspace, workspace_bytes, need))) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!apart({{loss, 4}, {load, (int64_t)cfg->num_experts * 4}, {workspace, (int64_t)need}},
             {{logits, logits_bytes(cfg)}, {topk_ids, slots_bytes(cfg)}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_balance_loss(cfg->logits_dtype == MOE_DTYPE_FP32, logits, topk_ids,
                                        coef, loss, load, workspace, cfg->num_tokens,
                                        shape_of(cfg), static_cast<hipStream_t>(stream)));
}

int moe_select_backward(const moe_select_config_t* cfg, const void* logits,
                        const int32_t* topk_ids, const float* grad_topk_w, const float* load,
                        const float* grad_loss, void* grad_logits, void* stream) {
  int st = validate_select(cfg, false);
  if (st) return st;
  if (!logits || !topk_ids || !grad_logits || (!grad_topk_w && !load) || (grad_loss && !load))
    return MOE_ERR_INVALID_ARG;
  if (!logits_aligned(cfg, logits) || !logits_aligned(cfg, grad_logits) || !aligned4(topk_ids) ||
      !aligned4(grad_topk_w) || !aligned4(load) || !aligned4(grad_loss))
    return MOE_ERR_INVALID_ARG;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!apart({{grad_logits, logits_bytes(cfg)}},
             {{logits, logits_bytes(cfg)},
              {topk_ids, slots_bytes(cfg)},
              {grad_topk_w, slots_bytes(cfg)},
              {load, (int64_t)cfg->num_experts * 4},
              {grad_loss, 4}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_select_backward(cfg->logits_dtype == MOE_DTYPE_FP32, logits, topk_ids,
                                           grad_topk_w, load, grad_loss, grad_logits,
                                           cfg->num_tokens, shape_of(cfg),
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
