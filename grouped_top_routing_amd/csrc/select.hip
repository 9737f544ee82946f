// Routing to experts from the router's logits, its gradient, and the loss that
// balances the experts' load, on gfx950.
//
// With z the logits of one token, s its scores (sigmoid of z, or softmax over
// the experts) and b a selection bias:
//   select    v_e = s_e + b_e; a group scores the sum of its one or two best v;
//             the best groups are kept, the best experts in them chosen; their
//             weights are s, or s over the sum of the chosen s
//   backward  dz from the gradient of those weights and of the balance loss
//   balance   coef * sum_e f_e P_e, f the experts' share of the pairs, P their
//             mean (normalised) score
//
// One wavefront handles one token: lane l holds experts l, l + 64, ...
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

constexpr int kWaves = 4;  // tokens per workgroup

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }

// A logit as the formulas take it: +inf counts as the largest finite number
// (NaN stays NaN, -inf masks its expert).
__device__ __forceinline__ float finite_top(float z) { return z > 3.4028234e38f ? 3.4028234e38f : z; }

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
template <class T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const T o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  return v;
}

// Logits of a token: the sum of `parts` arrays of `stride` elements (the
// router's partial sums, in their order), or one array.
template <class Z>
__device__ __forceinline__ float gather_logit(const Z* z, int parts, int64_t stride, int64_t at) {
  float v = load_logit(z + at);
  for (int p = 1; p < parts; ++p) v += load_logit(z + p * stride + at);
  return v;
}

// log of the sigmoid, without cancellation or overflow
__device__ __forceinline__ double log_sigmoid(double z) {
  return (z < 0.0 ? z : 0.0) - log1p(exp(-fabs(z)));
}
__device__ __forceinline__ float log_sigmoid(float z) {
  return fminf(z, 0.f) - log1pf(expf(-fabsf(z)));
}

// What a token's normalised scores are proportional to, with top its largest
// logit: exp(z - top) for the softmax; for the sigmoid itself, or where all of a
// row's sigmoids are so small that fp32 loses them, exp(z - top) again (sigmoid(z)
// = exp(z) to 2^-57 below z = -40).
__device__ __forceinline__ float share_of(float z, float top, int softmax) {
  if (softmax || top < -40.f) return z > -INFINITY ? expf(z - top) : 0.f;
  return sigmoidf_(z);
}

}  // namespace

// Selection.  Scores and selection values are taken in 64 bits: two experts
// whose values differ by less than an fp32 rounding are ordered by the values,
// not by the roundings.  Without a bias experts are ordered by their logits.
template <class Z, int V>
__global__ __launch_bounds__(64 * kWaves) void select_experts_kernel(
    const Z* __restrict__ logits, int parts, const float* __restrict__ bias,
    int32_t* __restrict__ ids, float* __restrict__ wout, float* __restrict__ zout, int64_t T,
    SelectShape c) {
  __shared__ double values[kWaves][V * 64];
  __shared__ double totals[kWaves][64];
  __shared__ uint8_t kept[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  const bool live = t < T;
  const int E = c.experts;

  float z[V];
  bool nan = false;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    z[i] = -INFINITY;
    if (live && e < E) {
      z[i] = gather_logit(logits, parts, T * E, t * E + e);
      if (zout) zout[t * E + e] = z[i];
      z[i] = finite_top(z[i]);
    }
    if (z[i] != z[i]) {
      nan = true;
      z[i] = -INFINITY;
    }
    top = fmaxf(top, z[i]);
  }
  nan = __any(nan);
  top = wave_max(top);
  double s[V], total = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const double d = z[i];
    if (c.softmax) s[i] = z[i] > -INFINITY ? exp(d - top) : 0.0;
    else s[i] = 1.0 / (1.0 + exp(-d));
    total += s[i];
  }
  if (c.softmax) {
    total = wave_sum(total);
    if (total > 0.0) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] /= total;
    }
  }
  double v[V], order[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    v[i] = s[i];
    if (bias && e < E) v[i] += (double)bias[e];
    if (!(z[i] > -INFINITY) || v[i] != v[i]) v[i] = -INFINITY;
    order[i] = bias ? v[i] : (double)z[i];
  }

  if (c.topk_groups < c.groups) {
    const int size = E / c.groups;
#pragma unroll
    for (int i = 0; i < V; ++i) values[wave][lane + 64 * i] = v[i];
    __syncthreads();
    double mine = -INFINITY;
    if (lane < c.groups) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int j = 0; j < size; ++j) {
        const double x = values[wave][lane * size + j];
        m2 = fmax(m2, fmin(m1, x));
        m1 = fmax(m1, x);
      }
      mine = c.group_best == 2 && m2 > -INFINITY ? m1 + m2 : m1;
    }
    totals[wave][lane] = mine;
    __syncthreads();
    int rank = 0;
    for (int g = 0; g < c.groups; ++g) {
      const double o = totals[wave][g];
      rank += o > mine || (o == mine && g < lane) ? 1 : 0;
    }
    kept[wave][lane] = rank < c.topk_groups;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !kept[wave][e / size]) order[i] = -INFINITY;
    }
  }

  int my_id = -1;
  float my_z = -INFINITY;
  double my_s = 0.0;
  for (int j = 0; j < c.topk; ++j) {
    double best = order[0];
    int at = lane;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (order[i] > best) {
        best = order[i];
        at = lane + 64 * i;
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const double ob = __shfl_xor(best, off);
      const int oa = __shfl_xor(at, off);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (!(best > -INFINITY)) break;  // the same in every lane
    const int owner = at & 63;
    double sw = 0.0;
    float zw = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at >> 6 == i) {
        sw = s[i];
        zw = z[i];
        if (lane == owner) order[i] = -INFINITY;
      }
    sw = __shfl(sw, owner);
    zw = __shfl(zw, owner);
    if (lane == j) {
      my_id = at;
      my_s = sw;
      my_z = zw;
    }
  }
  if (c.renormalize) {
    // by logarithms: scores that underflow still have a ratio
    double l = -INFINITY;
    if (my_id >= 0) l = c.softmax ? (double)my_z : log_sigmoid((double)my_z);
    const double m = wave_max(l);
    my_s = my_id >= 0 ? exp(l - m) : 0.0;
    const double sum = wave_sum(my_s);
    if (sum > 0.0) my_s /= sum;
  }
  if (live && lane < c.topk) {
    ids[t * c.topk + lane] = my_id;
    wout[t * c.topk + lane] = nan ? __builtin_nanf("") : (float)my_s;
  }
}

// Gradient of the weights (g) and of the balance loss (gl * load) with respect
// to every logit of a token; with C the slots that name an expert,
//   sigmoid:              dz_e = sum_{j of e} g_j s_e (1 - s_e)
//   ... renormalised:     dz_e = sum_{j of e} w_j (1 - s_e) (g_j - sum_C g_i w_i)
//   softmax:              dz_e = p_e (sum_{j of e} g_j - sum_C g_i p_i)
//   ... renormalised:     dz_e = sum_{j of e} w_j (g_j - sum_C g_i w_i)
//   balance:              + gl q_e (load_e - sum_i load_i q_i) [(1 - s_e) for the sigmoid]
// in rows with a slot in C; other rows get zeros.
template <class Z, int V>
__global__ __launch_bounds__(64 * kWaves) void select_backward_kernel(
    const Z* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ grad,
    const float* __restrict__ load, const float* __restrict__ grad_loss, Z* __restrict__ out,
    int64_t T, SelectShape c) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= T) return;  // the whole wave
  const int E = c.experts;
  float z[V], p[V], dz[V];
  bool nan = false;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    z[i] = e < E ? finite_top(load_logit(logits + t * E + e)) : -INFINITY;
    if (z[i] != z[i]) {
      nan = true;
      z[i] = -INFINITY;
    }
    top = fmaxf(top, z[i]);
    dz[i] = 0.f;
  }
  nan = __any(nan);
  top = wave_max(top);

  int id = -1;
  float g = 0.f, zc = -INFINITY;
  if (lane < c.topk) {
    id = ids[t * c.topk + lane];
    if (id >= 0 && id < E) {
      g = grad ? grad[t * c.topk + lane] : 0.f;
      zc = finite_top(load_logit(logits + t * E + id));
    } else {
      id = -1;
    }
  }
  const bool real = __any(id >= 0);

  // q: the scores over their sum; p: the scores
  float q[V], total = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    q[i] = share_of(z[i], top, c.softmax);
    total += q[i];
  }
  total = wave_sum(total);
  const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    q[i] *= inv;
    p[i] = c.softmax ? q[i] : sigmoidf_(z[i]);
  }

  if (grad) {
    float w = 0.f;
    if (id >= 0) {
      if (c.renormalize) w = c.softmax ? zc : log_sigmoid(zc);
      else if (c.softmax) w = zc > -INFINITY ? expf(zc - top) * inv : 0.f;
    }
    if (c.renormalize) {
      const float m = wave_max(id >= 0 ? w : -INFINITY);
      w = id >= 0 && m > -INFINITY ? expf(w - m) : 0.f;
      const float sum = wave_sum(w);
      if (sum > 0.f) w /= sum;
    }
    const float dot = c.renormalize || c.softmax ? wave_sum(id >= 0 ? g * w : 0.f) : 0.f;
    const float each = c.renormalize ? w * (g - dot) : g;
    for (int j = 0; j < c.topk; ++j) {
      const int e = __shfl(id, j);
      const float a = __shfl(each, j);
      if (e < 0) continue;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e == lane + 64 * i) dz[i] += a;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!c.renormalize) dz[i] = c.softmax ? p[i] * (dz[i] - dot) : p[i] * dz[i];
      if (!c.softmax) dz[i] *= sigmoidf_(-z[i]);
    }
  }
  if (load && real) {
    const float gl = grad_loss ? *grad_loss : 1.f;
    float l[V], mean = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      l[i] = e < E ? load[e] : 0.f;
      mean += q[i] * l[i];
    }
    mean = wave_sum(mean);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float d = gl * q[i] * (l[i] - mean);
      if (!c.softmax) d *= sigmoidf_(-z[i]);
      dz[i] += d;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    if (e < E) store_logit(out + t * E + e, !real ? 0.f : nan ? __builtin_nanf("") : dz[i]);
  }
}

// Balance loss, first pass: a workgroup sums the normalised scores of its
// tokens by expert (registers, then LDS, in a fixed order) and counts their
// pairs (integer atomics in LDS).  part: [blocks][E] sums, [blocks][E] counts,
// [blocks] rows with an expert.
template <class Z, int V>
__global__ __launch_bounds__(64 * kWaves) void balance_part_kernel(
    const Z* __restrict__ logits, const int32_t* __restrict__ ids, float* __restrict__ part,
    int64_t T, int per, SelectShape c) {
  __shared__ float sums[kWaves][V * 64];
  __shared__ int counts[V * 64];
  __shared__ int rows[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = c.experts;
  for (int e = threadIdx.x; e < V * 64; e += 64 * kWaves) counts[e] = 0;
  __syncthreads();
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  int mine = 0;
  const int64_t first = (int64_t)blockIdx.x * per;
  for (int64_t t = first + wave; t < first + per && t < T; t += kWaves) {
    int id = -1;
    if (lane < c.topk) {
      id = ids[t * c.topk + lane];
      if (id < 0 || id >= E) id = -1;
      else atomicAdd(&counts[id], 1);
    }
    if (!__any(id >= 0)) continue;
    ++mine;
    float z[V], p[V], top = -INFINITY, total = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      z[i] = e < E ? finite_top(load_logit(logits + t * E + e)) : -INFINITY;
      nan = nan || z[i] != z[i];
      top = fmaxf(top, z[i]);
    }
    nan = __any(nan);
    top = wave_max(top);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = share_of(z[i], top, c.softmax);
      total += p[i];
    }
    total = wave_sum(total);
    const float inv = nan ? __builtin_nanf("") : total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += p[i] * inv;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[wave][lane + 64 * i] = sum[i];
  if (lane == 0) rows[wave] = mine;
  __syncthreads();
  const int64_t B = gridDim.x;
  int32_t* pc = reinterpret_cast<int32_t*>(part) + B * E;
  int32_t* pr = pc + B * E;
  for (int e = threadIdx.x; e < E; e += 64 * kWaves) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += sums[w][e];
    part[(int64_t)blockIdx.x * E + e] = v;
    pc[(int64_t)blockIdx.x * E + e] = counts[e];
  }
  if (threadIdx.x == 0) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) n += rows[w];
    pr[blockIdx.x] = n;
  }
}

// Second pass, one workgroup: the sums over the first pass's workgroups, the
// load vector and the loss (64 bits).
__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ part, int B,
                                                            int E, float coef,
                                                            float* __restrict__ loss,
                                                            float* __restrict__ load) {
  __shared__ double dsum[16];
  __shared__ int64_t isum[16];
  __shared__ int64_t rsum[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t* pc = reinterpret_cast<const int32_t*>(part) + (int64_t)B * E;
  const int32_t* pr = pc + (int64_t)B * E;
  double p = 0.0;
  int64_t n = 0, r = 0;
  const int e = threadIdx.x;
  if (e < E)
    for (int b = 0; b < B; ++b) {
      p += (double)part[(int64_t)b * E + e];
      n += pc[(int64_t)b * E + e];
    }
  for (int b = threadIdx.x; b < B; b += 1024) r += pr[b];
  int64_t ns = wave_sum(n);
  r = wave_sum(r);
  if (lane == 0) {
    isum[wave] = ns;
    rsum[wave] = r;
  }
  __syncthreads();
  int64_t pairs = 0, rows = 0;
  for (int w = 0; w < 16; ++w) {
    pairs += isum[w];
    rows += rsum[w];
  }
  const double f = pairs > 0 ? (double)E * (double)n / (double)pairs : 0.0;
  const double l = rows > 0 ? (double)coef * f / (double)rows : 0.0;
  if (e < E) load[e] = (float)l;
  double d = wave_sum(e < E && rows > 0 ? l * p : 0.0);
  if (lane == 0) dsum[wave] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < 16; ++w) v += dsum[w];
    *loss = (float)v;
  }
}

// ---------------------------------------------------------------------------
namespace {
// Calls f with the number of experts per lane as a constant.
template <class F>
hipError_t by_experts(int E, F f) {
  if (E <= 64) return f(std::integral_constant<int, 1>{});
  if (E <= 128) return f(std::integral_constant<int, 2>{});
  if (E <= 256) return f(std::integral_constant<int, 4>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}
unsigned token_blocks(int64_t T) { return (unsigned)((T + kWaves - 1) / kWaves); }
}  // namespace

hipError_t launch_select_experts(bool fp32, const void* logits, int parts, const float* bias,
                                 int32_t* ids, float* w, float* zout, int64_t T,
                                 const SelectShape& c, hipStream_t stream) {
  return by_experts(c.experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (fp32)
      hipLaunchKernelGGL((select_experts_kernel<float, V>), dim3(token_blocks(T)),
                         dim3(64 * kWaves), 0, stream, static_cast<const float*>(logits), parts,
                         bias, ids, w, zout, T, c);
    else
      hipLaunchKernelGGL((select_experts_kernel<uint16_t, V>), dim3(token_blocks(T)),
                         dim3(64 * kWaves), 0, stream, static_cast<const uint16_t*>(logits), parts,
                         bias, ids, w, zout, T, c);
    return hipGetLastError();
  });
}

hipError_t launch_select_backward(bool fp32, const void* logits, const int32_t* ids,
                                  const float* grad, const float* load, const float* grad_loss,
                                  void* out, int64_t T, const SelectShape& c, hipStream_t stream) {
  return by_experts(c.experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (fp32)
      hipLaunchKernelGGL((select_backward_kernel<float, V>), dim3(token_blocks(T)),
                         dim3(64 * kWaves), 0, stream, static_cast<const float*>(logits), ids,
                         grad, load, grad_loss, static_cast<float*>(out), T, c);
    else
      hipLaunchKernelGGL((select_backward_kernel<uint16_t, V>), dim3(token_blocks(T)),
                         dim3(64 * kWaves), 0, stream, static_cast<const uint16_t*>(logits), ids,
                         grad, load, grad_loss, static_cast<uint16_t*>(out), T, c);
    return hipGetLastError();
  });
}

// Workgroups of the first pass, and the tokens of each.
static int64_t balance_per(int64_t T) {
  const int64_t per = (T + 255) / 256;
  return (per + kWaves - 1) / kWaves * kWaves;
}
static int64_t balance_blocks(int64_t T) { return T > 0 ? (T + balance_per(T) - 1) / balance_per(T) : 0; }

size_t balance_ws(int64_t T, int E) {
  const int64_t B = balance_blocks(T);
  return (size_t)(B * E * 8 + B * 4);
}

hipError_t launch_balance_loss(bool fp32, const void* logits, const int32_t* ids, float coef,
                               float* loss, float* load, void* ws, int64_t T, const SelectShape& c,
                               hipStream_t stream) {
  const int64_t B = balance_blocks(T);
  float* part = static_cast<float*>(ws);
  const hipError_t err = by_experts(c.experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (fp32)
      hipLaunchKernelGGL((balance_part_kernel<float, V>), dim3((unsigned)B), dim3(64 * kWaves), 0,
                         stream, static_cast<const float*>(logits), ids, part, T,
                         (int)balance_per(T), c);
    else
      hipLaunchKernelGGL((balance_part_kernel<uint16_t, V>), dim3((unsigned)B), dim3(64 * kWaves),
                         0, stream, static_cast<const uint16_t*>(logits), ids, part, T,
                         (int)balance_per(T), c);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(1024), 0, stream, part, (int)B, c.experts,
                     coef, loss, load);
  return hipGetLastError();
}

}  // namespace beam
