// Host-side helpers shared by the C ABI's translation units: argument
// validation, alignment, workspace checks, status codes.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "../../include/beam_moe.h"

namespace beam {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Weight layouts an entry point accepts (bit i = layout i).
constexpr int kBf16Layouts = (1 << MOE_LAYOUT_ROW_MAJOR) | (1 << MOE_LAYOUT_PACKED);
constexpr int kFp8Layouts = 1 << MOE_LAYOUT_FP8_PACKED;
constexpr int kFp4Layouts = 1 << MOE_LAYOUT_FP4_PACKED;
constexpr int kAnyLayout = kBf16Layouts | kFp8Layouts | kFp4Layouts;

inline int validate(const moe_config_t* c, int layouts = kBf16Layouts) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->num_tokens < 0 || c->hidden <= 0 || c->intermediate <= 0 || c->num_experts <= 0 ||
      c->num_groups <= 0 || c->topk_groups <= 0 || c->topk <= 0)
    return MOE_ERR_INVALID_ARG;
  if (c->renormalize != 0 && c->renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->routed_scaling)) return MOE_ERR_INVALID_ARG;
  if (c->num_experts % c->num_groups != 0) return MOE_ERR_INVALID_ARG;
  if (c->weight_layout < 0 || c->weight_layout > MOE_LAYOUT_FP4_PACKED ||
      !((layouts >> c->weight_layout) & 1))
    return MOE_ERR_INVALID_ARG;
  if (c->topk_groups > c->num_groups) return MOE_ERR_INVALID_ARG;
  if ((int64_t)c->topk > (int64_t)c->topk_groups * (c->num_experts / c->num_groups))
    return MOE_ERR_INVALID_ARG;
  // shapes the gfx950 kernels are built for
  if (c->num_experts != 256) return MOE_ERR_UNSUPPORTED;
  if (c->num_groups > 64 || (c->num_groups & (c->num_groups - 1)) != 0) return MOE_ERR_UNSUPPORTED;
  if (c->topk > 8) return MOE_ERR_UNSUPPORTED;
  if (c->hidden % 256 != 0 || c->intermediate % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (c->num_tokens * (int64_t)c->topk >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

inline int64_t pairs(const moe_config_t* c) { return c->num_tokens * (int64_t)c->topk; }

inline int check_ws(void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws || have < need) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Whether no output overlaps an input or another output (null: not given).
// The kernels read and write them in no order.
struct Span {
  const void* at;
  int64_t bytes;
  bool meets(const Span& o) const {
    const uintptr_t a = reinterpret_cast<uintptr_t>(at), b = reinterpret_cast<uintptr_t>(o.at);
    return at && o.at && (a < b ? b - a < (uint64_t)bytes : a - b < (uint64_t)o.bytes);
  }
};
inline bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (o->meets(i)) return false;
    for (const Span* p = outs.begin(); p != o; ++p)
      if (o->meets(*p)) return false;
  }
  return true;
}

// Workspace of moe_route and its kin (capi.hip).
size_t route_workspace(const moe_config_t* c);

// Workspace of moe_route_backward (capi_train.hip).
size_t route_backward_ws(const moe_config_t* c);

inline int device_ready() {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace beam
