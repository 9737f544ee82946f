// C ABI of the training calls: argument validation, workspace carving and
// launch sequencing.  Declarations and contracts are in include/beam_moe.h.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/beam_moe.h"
#include "capi_common.h"
#include "kernels.h"

namespace beam {

size_t route_backward_ws(const moe_config_t* c) {
  const RouteGradWs w = route_grad_ws(c->num_tokens, c->hidden, c->topk);
  return align_up(w.dz) + align_up(w.plan) + align_up(w.part);
}

}  // namespace beam

namespace {

using namespace beam;

// The row calls read num_tokens, hidden, topk and routed_scaling only.
int validate_rows(const moe_config_t* c, int dtype) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->num_tokens < 0 || c->hidden <= 0 || c->topk <= 0) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->routed_scaling)) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (c->topk > 8 || c->hidden > 1 << 28) return MOE_ERR_UNSUPPORTED;
  if (c->num_tokens >= ((int64_t)1 << 31) || pairs(c) >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Bytes of the row calls' arguments.
struct RowBytes {
  int64_t token_rows, sorted_rows, pairs;
  RowBytes(const moe_config_t* c, int dtype) {
    const int64_t row = (int64_t)c->hidden * (dtype == MOE_DTYPE_FP32 ? 4 : 2);
    token_rows = c->num_tokens * row;
    sorted_rows = beam::pairs(c) * row;
    pairs = beam::pairs(c) * 4;
  }
};

bool rate_ok(double v) { return std::isfinite(v) && v >= 0.0; }
bool beta_ok(double v) { return v >= 0.0 && v < 1.0; }

bool tensor_ok(const moe_adamw_tensor_t& t) {
  if (t.n < 0) return false;
  if (t.param_dtype != MOE_DTYPE_BF16 && t.param_dtype != MOE_DTYPE_FP32) return false;
  if (t.grad_dtype != MOE_DTYPE_BF16 && t.grad_dtype != MOE_DTYPE_FP32) return false;
  if (t.state_bits != 32 && t.state_bits != 8) return false;
  if (t.step < 0 || (reinterpret_cast<uintptr_t>(t.step_dev) & 7u)) return false;
  if (t.n == 0) return true;
  if (!t.param || !t.grad || !t.m || !t.v) return false;
  if ((t.param_dtype == MOE_DTYPE_BF16) != (t.master != nullptr)) return false;
  if (t.state_bits == 8 ? (!t.m_scale || !t.v_scale) : (t.m_scale || t.v_scale)) return false;
  return aligned16(t.param) && aligned16(t.master) && aligned16(t.grad) && aligned16(t.m) &&
         aligned16(t.v);
}

}  // namespace

extern "C" {

int moe_dispatch(const moe_config_t* cfg, int dtype, const void* x, const int32_t* perm_dst,
                 const float* topk_w, void* x_perm, void* stream) {
  int st = validate_rows(cfg, dtype);
  if (st) return st;
  if (!x || !perm_dst || !x_perm) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(x_perm) || !aligned4(perm_dst) || !aligned4(topk_w))
    return MOE_ERR_INVALID_ARG;
  if (cfg->num_tokens == 0) return MOE_OK;
  const RowBytes b(cfg, dtype);
  if (!apart({{x_perm, b.sorted_rows}},
             {{x, b.token_rows}, {perm_dst, b.pairs}, {topk_w, b.pairs}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_dispatch(dtype == MOE_DTYPE_FP32, x, perm_dst, topk_w, x_perm,
                                    cfg->num_tokens, cfg->hidden, cfg->topk,
                                    static_cast<hipStream_t>(stream)));
}

int moe_dispatch_backward(const moe_config_t* cfg, int dtype, const void* grad_x_perm,
                          const int32_t* perm_dst, const float* topk_w, const void* x,
                          void* grad_x, float* grad_topk_w, void* stream) {
  int st = validate_rows(cfg, dtype);
  if (st) return st;
  if (!grad_x_perm || !perm_dst || !grad_x) return MOE_ERR_INVALID_ARG;
  if ((x != nullptr) != (grad_topk_w != nullptr) || (x && !topk_w)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(grad_x_perm) || !aligned16(grad_x) || !aligned16(x) || !aligned4(perm_dst) ||
      !aligned4(topk_w) || !aligned4(grad_topk_w))
    return MOE_ERR_INVALID_ARG;
  if (cfg->num_tokens == 0) return MOE_OK;
  const RowBytes b(cfg, dtype);
  if (!apart({{grad_x, b.token_rows}, {grad_topk_w, b.pairs}},
             {{grad_x_perm, b.sorted_rows}, {perm_dst, b.pairs}, {topk_w, b.pairs},
              {x, b.token_rows}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_dispatch_backward(dtype == MOE_DTYPE_FP32, grad_x_perm, perm_dst,
                                             topk_w, x, grad_x, grad_topk_w, cfg->num_tokens,
                                             cfg->hidden, cfg->topk,
                                             static_cast<hipStream_t>(stream)));
}

int moe_combine_rows(const moe_config_t* cfg, int dtype, const void* y_perm,
                     const int32_t* perm_dst, const float* topk_w, void* out, void* stream) {
  int st = validate_rows(cfg, dtype);
  if (st) return st;
  if (!y_perm || !perm_dst || !topk_w || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y_perm) || !aligned16(out) || !aligned4(perm_dst) || !aligned4(topk_w))
    return MOE_ERR_INVALID_ARG;
  if (cfg->num_tokens == 0) return MOE_OK;
  const RowBytes b(cfg, dtype);
  if (!apart({{out, b.token_rows}},
             {{y_perm, b.sorted_rows}, {perm_dst, b.pairs}, {topk_w, b.pairs}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_combine_rows(dtype == MOE_DTYPE_FP32, y_perm, perm_dst, topk_w, out,
                                        cfg->num_tokens, cfg->hidden, cfg->topk,
                                        cfg->routed_scaling, static_cast<hipStream_t>(stream)));
}

int moe_combine_backward(const moe_config_t* cfg, int dtype, const void* grad_out,
                         const void* y_perm, const int32_t* perm_dst, const float* topk_w,
                         void* grad_y_perm, float* grad_topk_w, void* stream) {
  int st = validate_rows(cfg, dtype);
  if (st) return st;
  if (!grad_out || !perm_dst || (!grad_y_perm && !grad_topk_w)) return MOE_ERR_INVALID_ARG;
  if ((grad_topk_w && !y_perm) || (grad_y_perm && !topk_w)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(grad_out) || !aligned16(y_perm) || !aligned16(grad_y_perm) ||
      !aligned4(perm_dst) || !aligned4(topk_w) || !aligned4(grad_topk_w))
    return MOE_ERR_INVALID_ARG;
  if (cfg->num_tokens == 0) return MOE_OK;
  const RowBytes b(cfg, dtype);
  if (!apart({{grad_y_perm, b.sorted_rows}, {grad_topk_w, b.pairs}},
             {{grad_out, b.token_rows}, {y_perm, b.sorted_rows}, {perm_dst, b.pairs},
              {topk_w, b.pairs}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  return hip_status(launch_combine_backward(dtype == MOE_DTYPE_FP32, grad_out, y_perm, perm_dst,
                                            topk_w, grad_y_perm, grad_topk_w, cfg->num_tokens,
                                            cfg->hidden, cfg->topk, cfg->routed_scaling,
                                            static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                       const int32_t* topk_ids, const float* topk_logits,
                       const float* grad_topk_w, const int32_t* perm_src, const int32_t* offsets,
                       const uint16_t* grad_x_add, int accumulate, float* grad_w_router,
                       uint16_t* grad_x, void* workspace, size_t workspace_bytes, void* stream) {
  int st = validate(cfg, kAnyLayout);
  if (st) return st;
  if (!x || !w_router || !topk_ids || !topk_logits || !grad_topk_w || !perm_src || !offsets ||
      !grad_w_router || (grad_x_add && !grad_x) || (accumulate != 0 && accumulate != 1))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(grad_w_router) || !aligned16(grad_x) ||
      !aligned16(grad_x_add) || !aligned4(topk_ids) || !aligned4(topk_logits) ||
      !aligned4(grad_topk_w) || !aligned4(perm_src) || !aligned4(offsets))
    return MOE_ERR_INVALID_ARG;
  if (!route_grad_fits(cfg->num_tokens, cfg->hidden, cfg->topk, grad_x != nullptr))
    return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(workspace, workspace_bytes, route_backward_ws(cfg)))) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  const RowBytes b(cfg, MOE_DTYPE_BF16);
  const int64_t weights = (int64_t)cfg->num_experts * cfg->hidden * 4;
  if (!apart({{grad_w_router, weights}, {grad_x, b.token_rows},
              {workspace, (int64_t)route_backward_ws(cfg)}},
             {{x, b.token_rows}, {w_router, weights}, {topk_ids, b.pairs}, {topk_logits, b.pairs},
              {grad_topk_w, b.pairs}, {perm_src, b.pairs}, {offsets, (cfg->num_experts + 1) * 4},
              {grad_x_add == grad_x ? nullptr : grad_x_add, b.token_rows}}))
    return MOE_ERR_INVALID_ARG;
  if ((st = device_ready())) return st;
  const RouteGradWs w = route_grad_ws(cfg->num_tokens, cfg->hidden, cfg->topk);
  char* ws = static_cast<char*>(workspace);
  void* dz = ws;
  int32_t* plan = reinterpret_cast<int32_t*>(ws + align_up(w.dz));
  float* part = reinterpret_cast<float*>(ws + align_up(w.dz) + align_up(w.plan));
  return hip_status(launch_route_backward(
      x, w_router, topk_ids, topk_logits, grad_topk_w, perm_src, offsets, grad_x_add,
      grad_w_router, accumulate, grad_x, cfg->num_tokens, cfg->hidden, cfg->topk,
      cfg->renormalize, dz, plan, part, static_cast<hipStream_t>(stream)));
}

int moe_adamw_step(const moe_adamw_t* opt, const moe_adamw_tensor_t* tensors, int num_tensors,
                   void* stream) {
  if (!opt || num_tensors < 0 || (num_tensors > 0 && !tensors)) return MOE_ERR_INVALID_ARG;
  if (!rate_ok(opt->lr) || !beta_ok(opt->beta1) || !beta_ok(opt->beta2) || !rate_ok(opt->eps) ||
      !rate_ok(opt->weight_decay) || !std::isfinite(opt->grad_scale) ||
      (!opt->step_dev && opt->step < 1))
    return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(opt->step_dev) & 7u) || !aligned4(opt->lr_dev) ||
      !aligned4(opt->grad_scale_dev))
    return MOE_ERR_INVALID_ARG;
  bool any = false;
  for (int i = 0; i < num_tensors; ++i) {
    if (!tensor_ok(tensors[i])) return MOE_ERR_INVALID_ARG;
    if (tensors[i].n >= (int64_t)1 << 34) return MOE_ERR_UNSUPPORTED;
    any = any || tensors[i].n > 0;
  }
  if (!any) return MOE_OK;
  int st = device_ready();
  if (st) return st;
  AdamArgs a{};
  a.lr = opt->lr;
  a.beta1 = opt->beta1;
  a.beta2 = opt->beta2;
  a.eps = opt->eps;
  a.weight_decay = opt->weight_decay;
  a.grad_scale = opt->grad_scale;
  a.lr_dev = opt->lr_dev;
  a.grad_scale_dev = opt->grad_scale_dev;
  a.seed = opt->seed;
  // a launch ends where its list is full or its grid nears 2^32 threads (a
  // tensor of 2^34 elements alone stays below that)
  constexpr int64_t kMostBlocks = (int64_t)1 << 23;
  int64_t blocks = 0;
  for (int i = 0; i <= num_tensors; ++i) {
    const int64_t mine = i < num_tensors ? adamw_blocks(tensors[i].n) : 0;
    if (a.count > 0 &&
        (i == num_tensors || a.count == kAdamTensors || blocks + mine > kMostBlocks)) {
      adamw_factors(a);
      if ((st = hip_status(launch_adamw(a, blocks, static_cast<hipStream_t>(stream))))) return st;
      a.count = 0;
      blocks = 0;
    }
    if (mine == 0) continue;
    const moe_adamw_tensor_t& t = tensors[i];
    AdamTensor& d = a.tensor[a.count];
    d.param = t.param;
    d.master = t.master;
    d.grad = t.grad;
    d.m = t.m;
    d.v = t.v;
    d.m_scale = t.m_scale;
    d.v_scale = t.v_scale;
    d.n = t.n;
    d.kind = (t.param_dtype == MOE_DTYPE_FP32 ? 1 : 0) | (t.grad_dtype == MOE_DTYPE_FP32 ? 2 : 0) |
             (t.state_bits == 32 ? 4 : 0);
    if (const int64_t* counter = t.step_dev ? t.step_dev : t.step > 0 ? nullptr : opt->step_dev) {
      d.step_dev = counter;
      d.kind |= 8;
    } else {
      d.step = t.step > 0 ? t.step : opt->step;
    }
    d.place = i;
    a.first[a.count++] = blocks;
    blocks += mine;
  }
  return MOE_OK;
}

}  // extern "C"
