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
// One wavefront handles one token: lane l holds experts l, l + 64, ... (V of
// them), so that rows of any length and alignment are read in whole lines.
// Sums and maxima over the token run on DPP moves and end in scalar registers
// (by shuffles, and with all ordering in 64 bits, the selection of 16384 tokens took
// 41 us instead of 14.4); an arg-max is the maximum, then the first lane of a ballot that holds it.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

constexpr int kWaves = 4;         // tokens per workgroup
constexpr int kBalanceWaves = 16;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16(v); }

// A logit as the formulas take it: +inf counts as the largest finite number
// (NaN stays NaN, -inf masks its expert).
__device__ __forceinline__ float finite_top(float z) { return z > 3.4028234e38f ? 3.4028234e38f : z; }

// One DPP move of a value of one or two registers; lanes without a source (or in
// rows outside ROWS) get `none`.
template <int CTRL, int ROWS, class T>
__device__ __forceinline__ T dpp(T none, T v) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                             __builtin_bit_cast(int, v), CTRL,
                                                             ROWS, 0xf, false));
  } else {
    struct Two { int lo, hi; };
    const Two n = __builtin_bit_cast(Two, none), x = __builtin_bit_cast(Two, v);
    const Two o = {__builtin_amdgcn_update_dpp(n.lo, x.lo, CTRL, ROWS, 0xf, false),
                   __builtin_amdgcn_update_dpp(n.hi, x.hi, CTRL, ROWS, 0xf, false)};
    return __builtin_bit_cast(T, o);
  }
}
template <class T>
__device__ __forceinline__ T lane_value(T v, int lane) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  } else {
    struct Two { int lo, hi; };
    const Two x = __builtin_bit_cast(Two, v);
    const Two o = {__builtin_amdgcn_readlane(x.lo, lane), __builtin_amdgcn_readlane(x.hi, lane)};
    return __builtin_bit_cast(T, o);
  }
}
// Reduction over the wave, by rows of 16 lanes (row_shr 1, 2, 4, 8), then across
// them (row_bcast 15, 31); lane 63 ends with it.
template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, T none, F f) {
  v = f(v, dpp<0x111, 0xf>(none, v));
  v = f(v, dpp<0x112, 0xf>(none, v));
  v = f(v, dpp<0x114, 0xf>(none, v));
  v = f(v, dpp<0x118, 0xf>(none, v));
  v = f(v, dpp<0x142, 0xa>(none, v));
  v = f(v, dpp<0x143, 0xc>(none, v));
  return lane_value(v, 63);
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  return wave_reduce(v, T(0), [](T a, T b) { return a + b; });
}
// Keys that order as unsigned numbers like the floats they stand for, 0 below all
// of them (-inf is 0x7fffff; -0 counts as 0): a maximum of keys is one DPP
// instruction per step.
__device__ __forceinline__ uint32_t key_of(float v) {
  const int u = __float_as_int(v + 0.f);
  return (uint32_t)(u ^ (u >> 31 | (int)0x80000000));
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((int)k < 0 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint32_t wave_max_key(uint32_t k) {
  return wave_reduce(k, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float top_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double top_of(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float wave_max(float v) { return of_key(wave_max_key(key_of(v))); }
__device__ __forceinline__ double wave_max(double v) {
  return wave_reduce(v, (double)-INFINITY, [](double a, double b) { return fmax(a, b); });
}

// Logits of a token: the sum of `parts` arrays of `stride` elements (the
// router's partial sums, in their order), or one array.
template <class Z>
__device__ __forceinline__ float gather_logit(const Z* z, int parts, int64_t stride, int64_t at) {
  float v = load_logit(z + at);
#pragma unroll 4
  for (int p = 1; p < parts; ++p) v += load_logit(z + p * stride + at);
  return v;
}

// log of the sigmoid, without cancellation or overflow
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

// Scores in 32 or 64 bits, 0 for a masked expert.
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
template <int V, class T>
__device__ __forceinline__ void scores(const float (&z)[V], float top, int softmax, T (&s)[V]) {
  T total = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (softmax) s[i] = z[i] > -INFINITY ? exp_of((T)z[i] - (T)top) : (T)0;
    else s[i] = (T)1 / ((T)1 + exp_of(-(T)z[i]));
    total += s[i];
  }
  if (softmax) {
    total = wave_sum(total);
    if (total > (T)0) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] /= total;
    }
  }
}

// The kept groups of a token, one bit per group at bit g * sub, from its values
// in `values` (LDS of this wave, masked experts at -inf).  Lanes in `sub`s share
// a group; T is float or double, and `near` is set where two groups at the border
// are no further apart than `slack`.
template <class T>
__device__ __forceinline__ uint64_t kept_groups(const T* values, const SelectShape& c, int sub,
                                                int lane, T slack, bool& near) {
  const int size = c.experts / c.groups, mine = lane / sub;
  T m1 = -INFINITY, m2 = -INFINITY;
  if (mine < c.groups)
    for (int j = lane % sub; j < size; j += sub) {
      const T x = values[mine * size + j];
      m2 = top_of(m2, x < m1 ? x : m1);
      m1 = top_of(m1, x);
    }
  for (int off = 1; off < sub; off <<= 1) {
    const T a = __shfl_xor(m1, off), b = __shfl_xor(m2, off);
    m2 = top_of(a < m1 ? a : m1, top_of(m2, b));
    m1 = top_of(m1, a);
  }
  const T total = c.group_best == 2 && m2 > -INFINITY ? m1 + m2 : m1;
  int rank = 0;
  for (int g = 0; g < c.groups; ++g) {
    const T o = lane_value(total, g * sub);
    rank += o > total || (o == total && g < mine) ? 1 : 0;
  }
  const bool live = mine < c.groups, keep = live && rank < c.topk_groups;
  const T worst = -wave_max(keep ? -total : (T)-INFINITY);
  const T next = wave_max(live && !keep ? total : (T)-INFINITY);
  near = near || (next > -INFINITY && !(worst - next > slack));
  return __ballot(keep && lane % sub == 0);
}

// What choose() works on: fp32 values as keys, fp64 values as they are.
__device__ __forceinline__ uint32_t handle_of(float v) { return v > -INFINITY ? key_of(v) : 0u; }
__device__ __forceinline__ double handle_of(double v) { return v; }
__device__ __forceinline__ bool handles_one(uint32_t h) { return h != 0; }
__device__ __forceinline__ bool handles_one(double h) { return h > -INFINITY; }
__device__ __forceinline__ uint32_t wave_max_handle(uint32_t h) { return wave_max_key(h); }
__device__ __forceinline__ double wave_max_handle(double h) { return wave_max(h); }
__device__ __forceinline__ uint32_t top_of(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The topk experts with the largest `order`, one after the other (the lower index
// of equals): lane j gets the j-th's index, or -1.  `near` is set where two
// neighbours in the order, the first that is left out among them, are no further
// apart than `slack` (negative: not asked; fp32 only).
template <int V, class T>
__device__ __forceinline__ int choose(const T (&order)[V], int topk, int lane, float slack,
                                      bool& near) {
  using H = decltype(handle_of(T(0)));
  H h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = handle_of(order[i]);
  const H none = handle_of((T)-INFINITY);
  int id = -1;
  float before = INFINITY;
  for (int j = 0; j <= topk; ++j) {
    if (j == topk && slack < 0.f) break;
    H best = h[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = top_of(best, h[i]);
    best = wave_max_handle(best);
    if (!handles_one(best)) break;
    if constexpr (sizeof(T) == 4) {
      if (slack >= 0.f) {
        const float v = of_key(best);
        near = near || !(before - v > slack);
        before = v;
      }
    }
    if (j == topk) break;
    int at = -1;  // the lowest index of those that hold it
#pragma unroll
    for (int i = V - 1; i >= 0; --i) {
      const uint64_t held = __ballot(h[i] == best);
      at = held ? __builtin_ctzll(held) + 64 * i : at;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = lane + 64 * i == at ? none : h[i];
    id = lane == j ? at : id;
  }
  return id;
}

}  // namespace

// Selection.  Two experts (or groups) whose values differ by less than an fp32
// rounding are ordered by the values, not by the roundings: values are compared
// in fp32, and a token whose order has a gap within their errors is done again in
// 64 bits.  Without a bias experts are ordered by their logits, and only groups need
// scores.
//
// How many are done again goes by the logits.  Of normal ones over 256 experts in 8
// groups, 4 kept, 8 chosen, at standard deviations of 1.5 / 3 / 5: sigmoids with a
// bias of deviation 0.3 0.1 % / 0.2 % / 0.2 % of the tokens, without one 0.04 / 0.3 /
// 6, with a bias of zeros 0.7 / 8 / 93 (saturated scores lie close together, and the
// bound is that of the row's largest score); softmax 0.02-0.2 / 0.02-0.5 / 0.5-5.
// Equal logits under equal biases count as near too: bf16 logits and a bias of zeros
// 30-37 % from 1.5 on.  16384 tokens take 26-29 us where few are, 48 where all are;
// 32 tokens 8.0 and 11.5 (calls from Python).
//
// Bound by the instructions of topk dependent rounds: 16384 tokens of 256 experts,
// 8 chosen, take 13.6 us (12.4 the fastest; their bytes would take 3.4).  Keys are integers
// because a float maximum takes two instructions per DPP step (14.4 us a call, 12.7 with
// keys).  32 tokens are one chain of latencies, 6.6 us at the fastest with sigmoids, bias
// and groups, 10.8 where the GPU idles between.
//
// Bound: with s_max the row's largest score, a score carries at most 48 U s_max
// (U = 2^-24; exponential 2 U, its argument's rounding U |d| at exp(-|d|), a sum
// over the experts 22 U and its arguments' mean 7 U, a quotient; 1e-36 where
// scores leave fp32's range), v one rounding more; two of them differ by twice
// that, sums of two by twice again.
template <class Z, int V>
__global__ __launch_bounds__(64 * kWaves) void select_experts_kernel(
    const Z* __restrict__ logits, int parts, const float* __restrict__ bias,
    int32_t* __restrict__ ids, float* __restrict__ wout, float* __restrict__ zout, int64_t T,
    SelectShape c) {
  __shared__ double mem[kWaves][V * 64];  // values of one token per wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= T) return;  // the whole wave; waves share nothing
  const int E = c.experts;

  float z[V], top = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    z[i] = e < E ? gather_logit(logits, parts, T * E, t * E + e) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    if (zout && e < E) zout[t * E + e] = z[i];
    nan = nan || z[i] != z[i];
    z[i] = z[i] != z[i] ? -INFINITY : finite_top(z[i]);
    top = fmaxf(top, z[i]);
  }
  nan = __any(nan);
  const bool raw = c.softmax && !c.renormalize;

  const bool grouped = c.topk_groups < c.groups;
  int sub = 64;  // lanes per group
  while (sub > 1 && (64 / sub) < c.groups) sub >>= 1;
  const uint32_t by_size = ((1u << 20) + E / c.groups - 1) / (E / c.groups);  // e / size, e < 1024

  float s[V];
  if (bias || grouped || raw) top = wave_max(top);
  if (bias || grouped) scores(z, top, c.softmax, s);
  int id = -1;
  // T is float, or double where float cannot tell
  auto pick = [&](auto zero, float slack, bool& near) {
    using T = decltype(zero);
    T v[V], order[V];
    if (bias || grouped) {
      if constexpr (sizeof(T) == 8) scores(z, top, c.softmax, v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        if constexpr (sizeof(T) == 4) v[i] = s[i];
        if (bias) v[i] += e < E ? (T)bias[e] : (T)0;
        if (!(z[i] > -INFINITY) || v[i] != v[i]) v[i] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) order[i] = bias ? v[i] : (T)z[i];
    if (grouped) {
      T* values = reinterpret_cast<T*>(mem[wave]);
#pragma unroll
      for (int i = 0; i < V; ++i) values[lane + 64 * i] = v[i];
      compiler_fence();  // a wave's LDS accesses are done in order
      const uint64_t kept = kept_groups(values, c, sub, lane, (T)(2.f * slack), near);
      compiler_fence();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t e = lane + 64 * i, g = (e * by_size) >> 20;
        if (!((kept >> ((g * sub) & 63)) & 1)) order[i] = -INFINITY;
      }
    }
    id = choose(order, c.topk, lane, bias && sizeof(T) == 4 ? slack : -1.f, near);
  };
  bool near = false;
  if (!bias && !grouped) {
    pick(0.f, 0.f, near);
  } else {
    float s_max = 0.f, v_max = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      const float b = bias && e < E ? bias[e] : 0.f;
      s_max = fmaxf(s_max, s[i]);
      if (fabsf(b) < INFINITY) v_max = fmaxf(v_max, s[i] + fabsf(b));
    }
    const float slack =
        2.f * 5.9604645e-8f * (48.f * wave_max(s_max) + 2.f * wave_max(v_max)) + 1e-36f;
    pick(0.f, slack, near);
    if (near) {
      near = false;
      pick(0.0, 0.f, near);
    }
  }

  // the chosen logits, then the weights (by logarithms: scores that underflow
  // still have a ratio)
  float w = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float zi = __shfl(z[i], id & 63);
    w = id >> 6 == i ? zi : w;
  }
  if (c.renormalize) {
    if (!c.softmax) w = log_sigmoid(w);
    const float m = wave_max(id >= 0 ? w : -INFINITY);
    w = id >= 0 ? expf(w - m) : 0.f;
    const float sum = wave_sum(w);
    if (sum > 0.f) w /= sum;
  } else if (!raw) {
    w = id >= 0 ? sigmoidf_(w) : 0.f;
  } else {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) total += z[i] > -INFINITY ? expf(z[i] - top) : 0.f;
    total = wave_sum(total);
    w = id >= 0 ? expf(w - top) / total : 0.f;
  }
  if (lane < c.topk) {
    ids[t * c.topk + lane] = id;
    wout[t * c.topk + lane] = nan ? __builtin_nanf("") : w;
  }
}

// Gradient of the weights (g) and of the balance loss (gl * load) with respect
// to every logit of a token; with C the slots that name an expert,
//   sigmoid:              dz_e = sum_{j of e} g_j s_e (1 - s_e)
//   ... renormalised:     dz_e = sum_{j of e} w_j (1 - s_e) (g_j - sum_C g_i w_i)
//   softmax:              dz_e = p_e (sum_{j of e} g_j - sum_C g_i p_i)
//   ... renormalised:     dz_e = sum_{j of e} w_j (g_j - sum_C g_i w_i)
//   balance:              + gl q_e (load_e - sum_i load_i q_i) [(1 - s_e) for the sigmoid]
// in rows with a slot in C; other rows get zeros.  One read of the logits, one write;
// 4096 tokens of 256 experts with the balance loss take 6.6 us (1.3 TB/s), 509 of 60
// experts 3.6: the latencies of a wave's loads (logits, ids, the chosen logits) and
// sums.
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
      const int e = lane_value(id, j);
      const float a = lane_value(each, j);
      if (e < 0) continue;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e >> 6 == i) dz[i] += lane == (e & 63) ? a : 0.f;
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
// tokens by expert (a wave's tokens in registers, then the waves in LDS, in a
// fixed order) and counts their pairs (integer atomics in LDS).  A wave's sum is
// one of up to 32768 tokens: in 64 bits, and rounded to 32 once, since 32 bits
// would drift by up to half a step per token where a router's scores are alike
// (5e-5 of the loss at 4096 tokens a wave).  part: [blocks][E]
// sums, [blocks][E] counts, [blocks] rows with an expert.  At most 128 workgroups,
// so that the second pass stays short: 4096 tokens of 256 experts take 5.7 us here and
// 6.3 there, both latencies of dependent loads rather than their bytes (4.3 MB).
template <class Z, int V>
__global__ __launch_bounds__(64 * kBalanceWaves) void balance_part_kernel(
    const Z* __restrict__ logits, const int32_t* __restrict__ ids, float* __restrict__ part,
    int64_t T, int64_t per, SelectShape c) {
  __shared__ float sums[kBalanceWaves][V * 64];
  __shared__ int counts[V * 64];
  __shared__ int rows[kBalanceWaves];
  constexpr int kThreads = 64 * kBalanceWaves;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = c.experts;
  for (int e = threadIdx.x; e < V * 64; e += kThreads) counts[e] = 0;
  __syncthreads();
  double sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.0;
  int mine = 0;
  const int64_t first = (int64_t)blockIdx.x * per, last = first + per < T ? first + per : T;
  auto load = [&](int64_t t, float (&z)[V], int& id) {  // of a token, if there is one
    if (t >= last) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      z[i] = e < E ? load_logit(logits + t * E + e) : -INFINITY;
    }
    id = lane < c.topk ? ids[t * c.topk + lane] : -1;
  };
  auto add = [&](float (&z)[V], int id) {
    const bool on = id >= 0 && id < E;
    if (on) atomicAdd(&counts[id], 1);
    if (!__any(on)) return;
    ++mine;
    float p[V], top = -INFINITY, total = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[i] = finite_top(z[i]);
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
    for (int i = 0; i < V; ++i) sum[i] += (double)(p[i] * inv);
  };
  // the next token's logits are on their way while one is added
  float za[V], zb[V];
  int ia = -1, ib = -1;
  int64_t t = first + wave;
  load(t, za, ia);
  for (; t < last; t += 2 * kBalanceWaves) {
    load(t + kBalanceWaves, zb, ib);
    add(za, ia);
    load(t + 2 * kBalanceWaves, za, ia);
    if (t + kBalanceWaves < last) add(zb, ib);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[wave][lane + 64 * i] = (float)sum[i];
  if (lane == 0) rows[wave] = mine;
  __syncthreads();
  const int64_t B = gridDim.x;
  int32_t* pc = reinterpret_cast<int32_t*>(part) + B * E;
  int32_t* pr = pc + B * E;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kBalanceWaves; ++w) v += sums[w][e];
    part[(int64_t)blockIdx.x * E + e] = v;
    pc[(int64_t)blockIdx.x * E + e] = counts[e];
  }
  if (threadIdx.x == 0) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kBalanceWaves; ++w) n += rows[w];
    pr[blockIdx.x] = n;
  }
}

// Second pass, one workgroup: the sums over the first pass's workgroups in 64
// bits (1024 / E threads per expert take every so-many-th of them, and are added
// in order), the load vector and the loss.
__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ part, int B,
                                                            int E, float coef,
                                                            float* __restrict__ loss,
                                                            float* __restrict__ load) {
  __shared__ double psum[1024];
  __shared__ int64_t nsum[1024];
  __shared__ double dsum[16];
  __shared__ int64_t isum[16], rsum[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t* pc = reinterpret_cast<const int32_t*>(part) + (int64_t)B * E;
  const int32_t* pr = pc + (int64_t)B * E;
  const int ways = 1024 / E, way = threadIdx.x / E, e = threadIdx.x - way * E;
  double p = 0.0;
  int64_t n = 0, r = 0;
  if (way < ways) {
#pragma unroll 8
    for (int b = way; b < B; b += ways) {
      p += (double)part[(int64_t)b * E + e];
      n += pc[(int64_t)b * E + e];
    }
  }
  psum[threadIdx.x] = p;
  nsum[threadIdx.x] = n;
  for (int b = threadIdx.x; b < B; b += 1024) r += pr[b];
  __syncthreads();
  const bool owner = (int)threadIdx.x < E;
  p = 0.0;
  n = 0;
  if (owner)
    for (int w = 0; w < ways; ++w) {
      p += psum[w * E + threadIdx.x];
      n += nsum[w * E + threadIdx.x];
    }
  const int64_t ns = wave_sum(n);
  r = wave_sum(r);
  if (lane == 0) {
    isum[wave] = ns;
    rsum[wave] = r;
  }
  __syncthreads();
  int64_t pairs = 0, rows = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    pairs += isum[w];
    rows += rsum[w];
  }
  const double f = pairs > 0 ? (double)E * (double)n / (double)pairs : 0.0;
  const double l = rows > 0 ? (double)coef * f / (double)rows : 0.0;
  if (owner) load[threadIdx.x] = (float)l;
  const double d = wave_sum(owner && rows > 0 ? l * p : 0.0);
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

// Workgroups of the first pass (at most 128: the second one adds them up), and
// the tokens of each.
static int64_t balance_per(int64_t T) {
  const int64_t per = (T + 127) / 128;
  return per < kBalanceWaves ? kBalanceWaves : per;
}
static int64_t balance_blocks(int64_t T) { return (T + balance_per(T) - 1) / balance_per(T); }

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
      hipLaunchKernelGGL((balance_part_kernel<float, V>), dim3((unsigned)B),
                         dim3(64 * kBalanceWaves), 0, stream, static_cast<const float*>(logits),
                         ids, part, T, balance_per(T), c);
    else
      hipLaunchKernelGGL((balance_part_kernel<uint16_t, V>), dim3((unsigned)B),
                         dim3(64 * kBalanceWaves), 0, stream,
                         static_cast<const uint16_t*>(logits), ids, part, T, balance_per(T), c);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(1024), 0, stream, part, (int)B, c.experts,
                     coef, loss, load);
  return hipGetLastError();
}

}  // namespace beam
