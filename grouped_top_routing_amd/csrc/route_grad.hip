// Gradient of the router (gfx950).
//
// Forward, for token t with hidden state x and the chosen experts e_j:
//   z_j = x . W_{e_j},  s_j = sigmoid(z_j),  w_j = s_j / S with S = sum_i s_i
//   (or w_j = s_j without renormalisation).
// Given g_j = dL/dw_j:
//   renormalised  dz_j = w_j (1 - s_j) (g_j - sum_i g_i w_i)
//   otherwise     dz_j = s_j (1 - s_j) g_j
//   dL/dW_e = sum over the pairs of expert e of dz * x_t
//   dL/dx_t = sum_j dz_j W_{e_j}
// The selection itself has no gradient.  1 - s is taken as sigmoid(-z), and
// w from the log-sigmoids, so neither cancels nor underflows at large |z|.
//
// dz is sparse (topk of 256 experts per token), so both products are sums of
// rows: 4 topk T H operations instead of the dense 4*256 T H, no matrix cores
// needed, and fp32 throughout.  What bounds them is how often the rows are
// read: each x row by topk experts and each W row by all its tokens.  Both
// kernels therefore work on slabs of 256 columns, and consecutive workgroups
// of one XCD stay on one slab: the W slab (256 KB) and the x slab (512 B per
// token) stay in that XCD's L2.
#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

constexpr int kE = 256;            // experts
constexpr int kSlab = 256;         // columns per workgroup
constexpr int kTokensPerWave = 4;  // of the grad x part

// The plan (int32): per chunk (expert, first row, rows), then for every
// expert its first chunk (kE + 1 entries).  Every expert has at least one
// chunk, so the ones without rows get their zeros written too.
struct Plan {
  int32_t* chunk;
  int32_t* first;
};
__host__ __device__ inline Plan plan_of(int32_t* p, int64_t chunks) { return {p, p + 3 * chunks}; }

__device__ __forceinline__ float log_sigmoid(float z) {
  return fminf(z, 0.f) - log1pf(expf(-fabsf(z)));
}

// Workgroups 0 .. gridDim.x - 2: dz of 256 tokens.  The last one: the plan.
__global__ __launch_bounds__(256) void route_dz_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ logits,
    const float* __restrict__ grad_w, float* __restrict__ dz, const int32_t* __restrict__ offsets,
    int32_t* __restrict__ plan, int64_t chunks, int64_t T, int topk, int renormalize) {
  if (blockIdx.x == gridDim.x - 1) {
    __shared__ int sum[kE];
    const int e = threadIdx.x;
    const int n = (int)(T * topk);
    const int lo = min(max(offsets[e], 0), n), hi = min(max(offsets[e + 1], lo), n);
    const int mine = max(1, (hi - lo + kRouteChunk - 1) / kRouteChunk);
    sum[e] = mine;
    __syncthreads();
    for (int off = 1; off < kE; off <<= 1) {
      const int v = e >= off ? sum[e - off] : 0;
      __syncthreads();
      sum[e] += v;
      __syncthreads();
    }
    const Plan pl = plan_of(plan, chunks);
    // offsets that overlap could ask for more chunks than there are
    const int end = (int)min((int64_t)sum[e], chunks);
    const int begin = min(sum[e] - mine, end);
    pl.first[e] = begin;
    if (e == kE - 1) pl.first[kE] = end;
    for (int c = begin; c < end; ++c) {
      const int r0 = lo + (c - begin) * kRouteChunk;
      pl.chunk[3 * c] = e;
      pl.chunk[3 * c + 1] = r0;
      pl.chunk[3 * c + 2] = min(kRouteChunk, hi - r0);
    }
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= T) return;
  float z[8], g[8], w[8];
  bool on[8];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    on[j] = false;
    z[j] = g[j] = w[j] = 0.f;
    if (j < topk) {
      const int e = ids[t * topk + j];
      on[j] = e >= 0 && e < kE;
      if (on[j]) {
        z[j] = logits[t * topk + j];
        g[j] = grad_w[t * topk + j];
        w[j] = log_sigmoid(z[j]);
        top = fmaxf(top, w[j]);
      }
    }
  }
  float mean = 0.f;  // sum_i g_i w_i
  if (renormalize) {
    // w_j = s_j / S as exp(log s_j - max): scores that all underflow (every
    // logit -infinity) weigh nothing, and nothing flows back
    float total = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = on[j] && top > -INFINITY ? expf(w[j] - top) : 0.f;
      total += w[j];
    }
    const float inv = total != 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] *= inv;
      if (on[j]) mean += g[j] * w[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = sigmoidf_(z[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < topk)
      dz[t * topk + j] = on[j] ? w[j] * sigmoidf_(-z[j]) * (g[j] - mean) : 0.f;
}

// One (chunk, slab) of grad W: 4 waves, each two rows at a time (32 lanes of
// 8 columns each), summed in LDS.  An expert of one chunk is finished here;
// of several, each chunk leaves a partial sum for route_dw_reduce_kernel.
__device__ __forceinline__ void dw_item(const uint16_t* __restrict__ x,
                                        const int32_t* __restrict__ perm_src,
                                        const float* __restrict__ dz, const Plan pl, int chunk,
                                        int slab, float* __restrict__ grad, int accumulate,
                                        float* __restrict__ part, int64_t n, int H, int topk,
                                        float (*lds)[kSlab]) {
  const int e = pl.chunk[3 * chunk], r0 = pl.chunk[3 * chunk + 1], rows = pl.chunk[3 * chunk + 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = slab * kSlab + (lane & 31) * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i = 2 * wave + (lane >> 5); i < rows; i += 8) {
    const int64_t p = perm_src[r0 + i];
    if (p < 0 || p >= n) continue;
    const float d = dz[p];
    const uint4 q = ld16(x + (int64_t)((uint32_t)p / (uint32_t)topk) * H + col);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      acc[2 * c] += d * bf16_to_f32(u[c] & 0xffffu);
      acc[2 * c + 1] += d * __uint_as_float(u[c] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] += __shfl_xor(acc[c], 32);
  if (lane < 32)
#pragma unroll
    for (int c = 0; c < 8; ++c) lds[wave][lane * 8 + c] = acc[c];
  __syncthreads();
  const int c = threadIdx.x;
  float s = ((lds[0][c] + lds[1][c]) + lds[2][c]) + lds[3][c];
  const bool whole = pl.first[e + 1] - pl.first[e] == 1;
  if (whole) {
    float* o = grad + (size_t)e * H + slab * kSlab + c;
    *o = accumulate ? *o + s : s;
  } else {
    part[(size_t)chunk * H + slab * kSlab + c] = s;
  }
}

// kTokensPerWave tokens of one slab of grad x per wave.
__device__ __forceinline__ void dx_item(const float* __restrict__ wr,
                                        const int32_t* __restrict__ ids,
                                        const float* __restrict__ dz,
                                        const uint16_t* __restrict__ add,
                                        uint16_t* __restrict__ grad_x, int64_t group, int slab,
                                        int64_t T, int H, int topk) {
  const int lane = threadIdx.x & 63;
  const int col = slab * kSlab + lane * 4;
  for (int i = 0; i < kTokensPerWave; ++i) {
    const int64_t t = __builtin_amdgcn_readfirstlane(
        (int)((group * 4 + (threadIdx.x >> 6)) * kTokensPerWave + i));
    if (t >= T) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (add) {
      const uint2 a = *reinterpret_cast<const uint2*>(add + t * H + col);
      acc = make_float4(bf16_to_f32(a.x & 0xffffu), __uint_as_float(a.x & 0xffff0000u),
                        bf16_to_f32(a.y & 0xffffu), __uint_as_float(a.y & 0xffff0000u));
    }
    float4 q[8];
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = j < topk ? ids[t * topk + j] : -1;
      const bool on = e >= 0 && e < kE;
      d[j] = on ? dz[t * topk + j] : 0.f;
      q[j] = on ? *reinterpret_cast<const float4*>(wr + (size_t)e * H + col)
                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc.x += d[j] * q[j].x; acc.y += d[j] * q[j].y;
      acc.z += d[j] * q[j].z; acc.w += d[j] * q[j].w;
    }
    *reinterpret_cast<uint2*>(grad_x + t * H + col) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  }
}

// Both products in one launch (they are independent): the first dw_items
// workgroups take (slab, chunk), the rest (slab, 16 tokens).  Within each part
// XCD b mod 8 walks a contiguous eighth of the slab-major items.
__global__ __launch_bounds__(256) void route_grad_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ wr, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ perm_src, const float* __restrict__ dz, int32_t* plan,
    int64_t chunks, const uint16_t* __restrict__ add, float* __restrict__ grad_w, int accumulate,
    float* __restrict__ part, uint16_t* __restrict__ grad_x, int64_t T, int H, int topk,
    int64_t dw_blocks) {
  __shared__ float lds[4][kSlab];
  const int slabs = H / kSlab;
  int64_t b = blockIdx.x;
  if (b < dw_blocks) {
    const int64_t per = dw_blocks / 8, item = (b & 7) * per + (b >> 3);
    const int slab = (int)(item / chunks), chunk = (int)(item - slab * chunks);
    const Plan pl = plan_of(plan, chunks);
    if (slab >= slabs || chunk >= pl.first[kE]) return;
    dw_item(x, perm_src, dz, pl, chunk, slab, grad_w, accumulate, part, T * topk, H, topk, lds);
  } else {
    b -= dw_blocks;
    const int64_t per = (gridDim.x - dw_blocks) / 8, item = (b & 7) * per + (b >> 3);
    const int64_t groups = (T + 4 * kTokensPerWave - 1) / (4 * kTokensPerWave);
    const int slab = (int)(item / groups);
    if (slab >= slabs) return;
    dx_item(wr, ids, dz, add, grad_x, item - slab * groups, slab, T, H, topk);
  }
}

// grad W of the experts with several chunks: their partial sums in chunk order.
__global__ __launch_bounds__(256) void route_dw_reduce_kernel(int32_t* plan, int64_t chunks,
                                                              const float* __restrict__ part,
                                                              float* __restrict__ grad, int H,
                                                              int accumulate) {
  const Plan pl = plan_of(plan, chunks);
  const int e = blockIdx.x, c = blockIdx.y * 256 + threadIdx.x;
  const int c0 = pl.first[e], c1 = pl.first[e + 1];
  if (c1 - c0 < 2) return;
  float s = 0.f;
#pragma unroll 4
  for (int i = c0; i < c1; ++i) s += part[(size_t)i * H + c];
  float* o = grad + (size_t)e * H + c;
  *o = accumulate ? *o + s : s;
}

int64_t chunks_of(int64_t n) { return kE + n / kRouteChunk; }
int64_t groups_of(int64_t T) { return (T + 4 * kTokensPerWave - 1) / (4 * kTokensPerWave); }

}  // namespace

RouteGradWs route_grad_ws(int64_t T, int H, int topk) {
  const int64_t n = T * topk, chunks = chunks_of(n);
  RouteGradWs w;
  w.dz = (size_t)n * sizeof(float);
  w.plan = (size_t)(3 * chunks + kE + 1) * sizeof(int32_t);
  w.part = n > kRouteChunk ? (size_t)chunks * H * sizeof(float) : 0;
  return w;
}

bool route_grad_fits(int64_t T, int H, int topk) {
  const int64_t blocks = (chunks_of(T * topk) + groups_of(T)) * (H / kSlab) + 16;
  return blocks * 256 < (int64_t)1 << 32;
}

hipError_t launch_route_backward(const uint16_t* x, const float* wr, const int32_t* ids,
                                 const float* logits, const float* grad_topk_w,
                                 const int32_t* perm_src, const int32_t* offsets,
                                 const uint16_t* add, float* grad_w, int accumulate,
                                 uint16_t* grad_x, int64_t T, int H, int topk, int renormalize,
                                 float* dz, int32_t* plan, float* part, hipStream_t stream) {
  const int64_t n = T * topk, chunks = chunks_of(n), slabs = H / kSlab;
  hipLaunchKernelGGL(route_dz_kernel, dim3((unsigned)((T + 255) / 256 + 1)), dim3(256), 0, stream,
                     ids, logits, grad_topk_w, dz, offsets, plan, chunks, T, topk, renormalize);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t dw = (chunks * slabs + 7) / 8 * 8;
  const int64_t dx = grad_x ? (groups_of(T) * slabs + 7) / 8 * 8 : 0;
  hipLaunchKernelGGL(route_grad_kernel, dim3((unsigned)(dw + dx)), dim3(256), 0, stream, x, wr,
                     ids, perm_src, dz, plan, chunks, add, grad_w, accumulate, part, grad_x, T, H,
                     topk, dw);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (n <= kRouteChunk) return hipSuccess;  // no expert has a second chunk
  hipLaunchKernelGGL(route_dw_reduce_kernel, dim3(kE, (unsigned)slabs), dim3(256), 0, stream, plan,
                     chunks, part, grad_w, H, accumulate);
  return hipGetLastError();
}

}  // namespace beam
