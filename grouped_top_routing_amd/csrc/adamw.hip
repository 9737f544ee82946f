// AdamW over a list of tensors (gfx950).
//
// Step t of one tensor, with g' = gs * g:
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p - lr wd p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32.  p is the parameter (fp32), or the fp32 master of a bf16 one, which
// is then rounded to nearest into the parameter.  t is the tensor's own: one
// that gets a gradient now and then has made fewer steps than its list, and its
// moments are corrected for those.
//
// States in 8 bits: blocks of 32 consecutive elements, an E4M3 code per element
// and one E8M0 scale (a power of two, so scaling is exact) per block.  Kept are
// m and sqrt(v), whose exponent range is half of v's.  Both are rounded
// stochastically: with b2 = 0.999 one step moves sqrt(v) by 0.05 %, and half a
// code step is 6 %, so rounding to nearest would freeze it; rounding up with
// the probability of the remainder keeps its mean.  The random bits are a hash
// of (seed, step, tensor, element), so a step is reproducible and does not
// depend on the launch.  The update uses m and v before they are rounded.
//
// Bound by HBM: 28 bytes per element with 32-bit states, 16.1 with 8-bit ones
// (bf16 parameter and gradient, fp32 master).  Every thread owns 8 consecutive
// elements (16-byte accesses, 8 for codes); four neighbouring lanes share a
// scale block.  The list travels in the kernel's arguments (no table in memory
// to keep or to copy), kAdamTensors tensors to a launch; a workgroup takes one
// span of 2048 elements (four spans: 415 -> 432 us, and the factors of a step
// are worked out on the host unless they are on the device).  Measured on 73.4
// M elements (one layer's rank-16 adapters): 377 us with 32-bit states (5.5
// TB/s), 213 with 8-bit ones (5.5 TB/s; conversions that are not the hardware's
// take 307).  With the step, the rate or the gradients' factor on the device
// every workgroup works the factors out before it can use its loads: 381 and 233
// us.  Stores are non-temporal (plain ones took 415 instead of 378 and 224
// instead of 208 us, and 10.6 instead of 9.5 on 1.3 M elements that stay in the
// caches); loads are not (393, 213 and 10.3 with them).
#include <cfloat>

#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

constexpr int kPer = 8;                    // elements per thread
constexpr int kSpan = 256 * kPer;          // elements per workgroup

// Scrambles 32 bits (two rounds of xor-shift and odd multiply).
__device__ __forceinline__ uint32_t mix32(uint32_t z) {
  z = (z ^ (z >> 16)) * 0x7A3D5E4Bu;
  z = (z ^ (z >> 15)) * 0xB5297A4Du;
  return z ^ (z >> 16);
}

// E8M0 code of the least power of two by which `most` (finite, >= 0) is at
// most 448, the largest E4M3 value; at least 2^-126.
__device__ __forceinline__ uint32_t scale_code(float most) {
  const uint32_t u = __float_as_uint(most);
  const int c = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(c, 1);
}

// 1 - b^t for t >= 1, by repeated squaring in 64 bits.
__host__ __device__ inline double one_minus_power(double b, int64_t t) {
  double r = 1.0, s = b;
  for (uint64_t u = (uint64_t)t; u; u >>= 1) {
    if (u & 1) r *= s;
    s *= s;
  }
  return 1.0 - r;
}

// Decay lr wd from which it goes by the factor 1 - lr wd: that factor's
// rounding, up to 2^-25, is then at most 2^-13 of the decay.  Below, where it
// would be a tenth of it (2e-5 * 0.01: 1.79e-7 instead of 2e-7) or all of it
// (below 2^-25 the factor is 1), decay joins the update before the one
// subtraction from p, which keeps its mean over many steps and elements.  (Same
// time either way: the kernel is bound by HBM.)
constexpr double kKeepFrom = 0x1p-12;

__host__ __device__ inline AdamFactors factors_of(const AdamArgs& a, int64_t t, double lr,
                                                  float gs) {
  AdamFactors f;
  f.b1 = (float)a.beta1;
  f.b2 = (float)a.beta2;
  f.omb1 = (float)(1.0 - a.beta1);
  f.omb2 = (float)(1.0 - a.beta2);
  f.eps = (float)a.eps;
  const double decay = lr * a.weight_decay;
  f.keep = decay < kKeepFrom ? 1.f : (float)(1.0 - decay);
  f.decay = decay < kKeepFrom ? (float)decay : 0.f;
  f.rate = (float)(lr / one_minus_power(a.beta1, t));
  f.root = (float)(1.0 / __builtin_sqrt(one_minus_power(a.beta2, t)));
  f.gs = gs;
  return f;
}

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float (&f)[kPer]) {
  if (n == kPer) {
    if constexpr (F32) {
      const float4 a = *reinterpret_cast<const float4*>((const float*)p + i);
      const float4 b = *reinterpret_cast<const float4*>((const float*)p + i + 4);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
      const uint4 q = ld16((const uint16_t*)p + i);
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f[2 * c] = bf16_to_f32(u[c] & 0xffffu);
        f[2 * c + 1] = __uint_as_float(u[c] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      f[c] = 0.f;
      if (c < n) f[c] = F32 ? ((const float*)p)[i + c] : bf16_to_f32(((const uint16_t*)p)[i + c]);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float (&f)[kPer]) {
  if (n == kPer) {
    if constexpr (F32) {
      __builtin_nontemporal_store(f32x4_t{f[0], f[1], f[2], f[3]},
                                  reinterpret_cast<f32x4_t*>((float*)p + i));
      __builtin_nontemporal_store(f32x4_t{f[4], f[5], f[6], f[7]},
                                  reinterpret_cast<f32x4_t*>((float*)p + i + 4));
    } else {
      __builtin_nontemporal_store(u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])},
                                  reinterpret_cast<u32x4_t*>((uint16_t*)p + i));
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (c < n) {
        if constexpr (F32) ((float*)p)[i + c] = f[c];
        else ((uint16_t*)p)[i + c] = (uint16_t)pack_bf16x2(f[c], 0.f);
      }
  }
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t i, int n, float scale,
                                           float (&f)[kPer]) {
  uint32_t w[2] = {0u, 0u};
  if (n == kPer) {
    const uint2 q = *reinterpret_cast<const uint2*>(p + i);
    w[0] = q.x;
    w[1] = q.y;
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (c < n) w[c >> 2] |= (uint32_t)p[i + c] << (8 * (c & 3));
  }
#pragma unroll
  for (int c = 0; c < kPer; c += 2) {
    const auto v = (c & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(w[c >> 2], true)
                           : __builtin_amdgcn_cvt_pk_f32_fp8(w[c >> 2], false);
    f[c] = v[0] * scale;
    f[c + 1] = v[1] * scale;
  }
}

// The largest over the four lanes of a quad.
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0xb1, 0xf, 0xf, true)));
  return fmaxf(v, __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0x4e, 0xf, 0xf, true)));
}

// The codes of f, their scale into `scales` (the four lanes of a block agree
// on it; values that are not finite do not count for it).  The hardware's
// stochastic conversion adds the seed's high bits below the kept mantissa and
// truncates: with 16 random bits on top and zeros behind, code = floor(x / step
// + random / 65536) steps exactly, subnormals included (checked against that
// formula on 2^26 values); infinities and NaN become NaN codes.  LOW: a value
// above zero does not become zero (sqrt(v) = 0 beside m != 0 would divide by
// eps alone).
template <bool LOW>
__device__ __forceinline__ void store_codes(uint8_t* p, uint8_t* scales, int64_t i, int n,
                                            const float (&f)[kPer], const uint32_t (&random)[kPer]) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) most = fmaxf(most, fabsf(f[c]));
  if (!(most < INFINITY)) {
    most = 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) most = fmaxf(most, fabsf(f[c]) < INFINITY ? fabsf(f[c]) : 0.f);
  }
  const uint32_t code = scale_code(quad_max(most));
  const float inv = __uint_as_float((254u - code) << 23);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    float x = f[c] * inv;
    if (LOW && x > 0.f) x = fmaxf(x, 0x1p-9f);
    const uint32_t seed = LOW ? random[c] & 0xffff0000u : random[c] << 16;
    uint32_t& o = w[c >> 2];
    switch (c & 3) {
      case 0: o = __builtin_amdgcn_cvt_sr_fp8_f32(x, seed, o, 0); break;
      case 1: o = __builtin_amdgcn_cvt_sr_fp8_f32(x, seed, o, 1); break;
      case 2: o = __builtin_amdgcn_cvt_sr_fp8_f32(x, seed, o, 2); break;
      default: o = __builtin_amdgcn_cvt_sr_fp8_f32(x, seed, o, 3); break;
    }
  }
  if (n == kPer) {
    __builtin_nontemporal_store(u32x2_t{w[0], w[1]}, reinterpret_cast<u32x2_t*>(p + i));
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c)
      if (c < n) p[i + c] = (uint8_t)(w[c >> 2] >> (8 * (c & 3)));
  }
  if (n > 0 && i % 32 == 0) scales[i / 32] = (uint8_t)code;
}

// 8 elements at i of one tensor (n of them exist; lanes past the end still
// take part in their block's scale).
template <bool P32, bool G32, bool S32>
__device__ __forceinline__ void update8(const AdamTensor& t, const AdamFactors& k, uint32_t key,
                                        int64_t i, int n) {
  // m and v are specified as separately rounded products and sums, so that
  // their 8-bit codes are the same wherever they are computed
#pragma clang fp contract(off)
  void* master = P32 ? t.param : (void*)t.master;
  float p[kPer], g[kPer], m[kPer], v[kPer];
  load8<G32>(t.grad, i, n, g);
  load8<true>(master, i, n, p);
  if constexpr (S32) {
    load8<true>(t.m, i, n, m);
    load8<true>(t.v, i, n, v);
  } else {
    const float ms = n > 0 ? __uint_as_float((uint32_t)t.m_scale[i / 32] << 23) : 0.f;
    const float vs = n > 0 ? __uint_as_float((uint32_t)t.v_scale[i / 32] << 23) : 0.f;
    load_codes((const uint8_t*)t.m, i, n, ms, m);
    load_codes((const uint8_t*)t.v, i, n, vs, v);
#pragma unroll
    for (int c = 0; c < kPer; ++c) v[c] = v[c] * v[c];
  }
  float root[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float gs = g[c] * k.gs;
    m[c] = m[c] * k.b1 + gs * k.omb1;
    v[c] = v[c] * k.b2 + (gs * gs) * k.omb2;
    root[c] = sqrtf(v[c]);
    // an infinite p stays infinite whatever the decay
    const float near = fminf(fmaxf(p[c], -FLT_MAX), FLT_MAX);
    p[c] = p[c] * k.keep - (k.decay * near + m[c] / (root[c] * k.root + k.eps) * k.rate);
  }
  store8<true>(master, i, n, p);
  if constexpr (!P32) store8<false>(t.param, i, n, p);
  if constexpr (S32) {
    store8<true>(t.m, i, n, m);
    store8<true>(t.v, i, n, v);
  } else {
    uint32_t random[kPer];
    const uint32_t lo = (uint32_t)i * 0x9E3779B1u + (uint32_t)(i >> 32) * 0x7F4A7C15u;
#pragma unroll
    for (int c = 0; c < kPer; ++c) random[c] = mix32((lo + (uint32_t)c * 0x9E3779B1u) ^ key);
    store_codes<false>((uint8_t*)t.m, t.m_scale, i, n, m, random);
    store_codes<true>((uint8_t*)t.v, t.v_scale, i, n, root, random);
  }
}

// *p by a scalar load (p is the same in every lane, and nothing in the kernel
// writes there).  Through vector registers the step takes its hash there too,
// also in steps that have it from the list: 227 against 213 us for the 8-bit
// states of 73.4 M elements.
__device__ __forceinline__ int64_t scalar_load(const int64_t* p) {
  typedef const __attribute__((address_space(4))) int64_t* scalar_ptr;
  return *(scalar_ptr)(uintptr_t)p;
}

__global__ __launch_bounds__(256) void adamw_kernel(const AdamArgs a) {
  // the tensor of this workgroup: the last whose first workgroup is not
  // behind it
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.first[mid] <= (int64_t)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamTensor& t = a.tensor[lo];
  AdamFactors k = a.factors;
  k.rate = t.rate;
  k.root = t.root;
  const bool counted = t.kind & 8;
  const int64_t step = counted ? scalar_load(t.step_dev) : t.step;
  if (counted || a.lr_dev || a.grad_scale_dev) {
    __shared__ AdamFactors shared;
    if (threadIdx.x == 0)
      shared = factors_of(a, step, a.lr_dev ? (double)*a.lr_dev : a.lr,
                          (float)a.grad_scale * (a.grad_scale_dev ? *a.grad_scale_dev : 1.f));
    __syncthreads();
    k = shared;
  }
  const uint32_t key = mix32(a.seed * 0x9E3779B9u + (uint32_t)step * 0x85157AF5u +
                             (uint32_t)t.place * 0x632BE5ABu);
  const int64_t i = ((int64_t)blockIdx.x - a.first[lo]) * kSpan + threadIdx.x * kPer;
  const int64_t left = t.n - i;
  const int n = left >= kPer ? kPer : left > 0 ? (int)left : 0;
  switch (t.kind & 7) {
    case 0: update8<false, false, false>(t, k, key, i, n); break;
    case 1: update8<true, false, false>(t, k, key, i, n); break;
    case 2: update8<false, true, false>(t, k, key, i, n); break;
    case 3: update8<true, true, false>(t, k, key, i, n); break;
    case 4: update8<false, false, true>(t, k, key, i, n); break;
    case 5: update8<true, false, true>(t, k, key, i, n); break;
    case 6: update8<false, true, true>(t, k, key, i, n); break;
    default: update8<true, true, true>(t, k, key, i, n); break;
  }
}

}  // namespace

int64_t adamw_blocks(int64_t n) { return (n + kSpan - 1) / kSpan; }

void adamw_factors(AdamArgs& a) {
  // of the tensors whose step is known here; most lists have one step
  int64_t last = 0;
  for (int i = 0; i < a.count; ++i) {
    AdamTensor& t = a.tensor[i];
    if (t.kind & 8) continue;
    if (t.step != last) a.factors = factors_of(a, t.step, a.lr, (float)a.grad_scale);
    last = t.step;
    t.rate = a.factors.rate;
    t.root = a.factors.root;
  }
}

hipError_t launch_adamw(const AdamArgs& a, int64_t blocks, hipStream_t stream) {
  hipLaunchKernelGGL(adamw_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace beam
