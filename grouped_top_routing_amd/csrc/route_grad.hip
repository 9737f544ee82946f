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
// read: each x row by topk experts (420 MB from L2 at 5120 tokens of 5120
// columns) and each W row by all its tokens (840 MB).  Workgroups therefore take
// slabs of columns, and consecutive workgroups of one XCD stay on one slab, so
// that an x slab (256 columns, 512 B per token) and a W slab (1 MB) stay in that
// XCD's L2 (token by token instead, grad x of 5120 tokens takes 74 against 62
// us of the whole call); large batches read W from LDS.  With 5120 tokens of
// 5120 columns and `add` the call takes 62 us, 75 with the tokens on few experts:
// grad W 37 (its 420 MB of row reads at 11 TB/s), grad x 32, dz and the plan 4,
// the partial sums 5.
#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

constexpr int kE = 256;            // experts
constexpr int kSlab = 256;         // columns per workgroup of the grad W part
constexpr int kDxCols = 1024;      // columns per workgroup of the grad x part
// Batches from which grad x reads the weights from LDS instead of L2.  The whole
// call, LDS against L2, with `add` and without: 5120 columns, 2048 tokens 35.1
// against 33.8 us and 33.4 against 32.1, 4096 tokens 53.1 against 54.0 and 50.7
// against 50.9, 5120 tokens 62 against 76 and 59 against 61, 16384 tokens 235
// against 309 and 220 against 238; 1280 columns, 2048 tokens 19.8 against 17.2
// and 19.1 against 16.1, 4096 tokens 24.6 against 24.5 and 23.4 against 22.9,
// 5120 tokens 26.8 against 28.7 and 25.6 against 27.0.
constexpr int64_t kLdsFrom = 4096;

// The plan (int32): per chunk (expert, first row, rows), then for every
// expert its first chunk (kE + 1 entries).  Every expert has at least one
// chunk, so the ones without rows get their zeros written too.
struct Plan {
  int32_t* chunk;
  int32_t* first;
};
__host__ __device__ inline Plan plan_of(int32_t* p, int64_t chunks) { return {p, p + 3 * chunks}; }

// What a slot adds: its expert (kE for none) and dz.  Every token has 8 of
// them, whatever topk is, so that they come in one scalar load of 64 bytes.
struct Slot {
  int expert;
  float dz;
};

__device__ __forceinline__ float log_sigmoid(float z) {
  return fminf(z, 0.f) - log1pf(expf(-fabsf(z)));
}

// Sum, maximum over the 8 lanes of a token.
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}

// Slot j of token t; the 8 lanes of a token call it together (t >= T: empty).
__device__ __forceinline__ Slot slot_of(const int32_t* __restrict__ ids,
                                        const float* __restrict__ logits,
                                        const float* __restrict__ grad_w, int64_t t, int j,
                                        int64_t T, int topk, int renormalize) {
  const bool slot = t < T && j < topk;
  const int64_t p = t * topk + j;
  const int e = slot ? ids[p] : -1;
  const float z = slot ? logits[p] : 0.f, gr = slot ? grad_w[p] : 0.f;
  const bool on = e >= 0 && e < kE;
  const float g = on ? gr : 0.f;
  float w, mean = 0.f;  // mean = sum_i g_i w_i
  if (renormalize) {
    // w_j = s_j / S as exp(log s_j - max): scores that all underflow keep
    // their ratios; with every logit -infinity nothing flows back
    const float ls = log_sigmoid(z);
    const float top = max8(on ? ls : -INFINITY);
    w = on && top > -INFINITY ? expf(ls - top) : 0.f;
    const float total = sum8(w);
    w = total != 0.f ? w / total : 0.f;
    mean = sum8(g * w);
  } else {
    w = sigmoidf_(z);
  }
  return {on ? e : kE, on ? w * sigmoidf_(-z) * (g - mean) : 0.f};
}

// Workgroups 0 .. gridDim.x - 2: dz of 32 tokens, a lane per slot (a lane per
// token took 8.7 instead of 3.8 us at 5120 tokens: the exponentials of 8 slots
// one after another).  The last one: the plan.
__global__ __launch_bounds__(256) void route_dz_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ logits,
    const float* __restrict__ grad_w, Slot* __restrict__ slots, const int32_t* __restrict__ offsets,
    int32_t* __restrict__ plan, int64_t chunks, int64_t T, int topk, int renormalize) {
  if (blockIdx.x == gridDim.x - 1) {
    __shared__ int wave_sum[kE / kWave];
    const int e = threadIdx.x, lane = e % kWave, wave = e / kWave;
    const int n = (int)(T * topk);
    const int lo = min(max(offsets[e], 0), n), hi = min(max(offsets[e + 1], lo), n);
    const int mine = max(1, (hi - lo + kRouteChunk - 1) / kRouteChunk);
    int sum = mine;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int v = __shfl_up(sum, off);
      if (lane >= off) sum += v;
    }
    if (lane == kWave - 1) wave_sum[wave] = sum;
    __syncthreads();
    for (int i = 0; i < wave; ++i) sum += wave_sum[i];
    const Plan pl = plan_of(plan, chunks);
    // offsets that overlap could ask for more chunks than there are
    const int end = (int)min((int64_t)sum, chunks);
    const int begin = min(sum - mine, end);
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
  const int64_t t = (int64_t)blockIdx.x * 32 + threadIdx.x / 8;
  const Slot s = slot_of(ids, logits, grad_w, t, threadIdx.x % 8, T, topk, renormalize);
  if (t < T) slots[t * 8 + threadIdx.x % 8] = s;
}

// One (chunk, slab) of grad W: 4 waves, each two rows at a time (32 lanes of
// 8 columns each), summed in LDS.  The chunk's tokens and dz are brought into
// LDS first, so that the row loads depend on nothing and run 4 deep.  An
// expert of one chunk is finished here; of several, each chunk leaves a
// partial sum for route_dw_reduce_kernel.
struct DwShared {
  float dz[kRouteChunk];
  int token[kRouteChunk];
  float part[4][kSlab];
};
__device__ __forceinline__ void dw_item(const uint16_t* __restrict__ x,
                                        const int32_t* __restrict__ perm_src,
                                        const Slot* __restrict__ slots, const Plan pl, int chunk,
                                        int slab, float* __restrict__ grad, int accumulate,
                                        float* __restrict__ part, int64_t n, int H, int topk,
                                        DwShared& sh) {
  const int e = pl.chunk[3 * chunk], r0 = pl.chunk[3 * chunk + 1], rows = pl.chunk[3 * chunk + 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool whole = pl.first[e + 1] - pl.first[e] == 1;
  static_assert(kRouteChunk == 256, "a thread per row of the chunk");
  {
    const int i = threadIdx.x;
    const int64_t p = i < rows ? perm_src[r0 + i] : -1;
    const bool ok = p >= 0 && p < n;
    const uint32_t t = (uint32_t)p / (uint32_t)topk;
    sh.dz[i] = ok ? slots[(int64_t)t * 8 + ((uint32_t)p - t * topk)].dz : 0.f;
    sh.token[i] = ok ? (int)t : -1;
  }
  __syncthreads();
  const int col = slab * kSlab + (lane & 31) * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i0 = 2 * wave + (lane >> 5); i0 < rows; i0 += 32) {
    uint4 q[4];
    float d[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 8 * u;  // at most 255: rows past the chunk's hold no token
      const int t = sh.token[i];
      d[u] = sh.dz[i];
      q[u] = t >= 0 ? ld16(x + (int64_t)t * H + col) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[2 * c] += d[u] * bf16_to_f32(w[c] & 0xffffu);
        acc[2 * c + 1] += d[u] * __uint_as_float(w[c] & 0xffff0000u);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] += __shfl_xor(acc[c], 32);
  if (lane < 32)
#pragma unroll
    for (int c = 0; c < 8; ++c) sh.part[wave][lane * 8 + c] = acc[c];
  __syncthreads();
  const int c = threadIdx.x;
  const float s = ((sh.part[0][c] + sh.part[1][c]) + sh.part[2][c]) + sh.part[3][c];
  if (whole) {
    float* o = grad + (size_t)e * H + slab * kSlab + c;
    *o = accumulate ? *o + s : s;
  } else {
    part[(size_t)chunk * H + slab * kSlab + c] = s;
  }
}

// kDxCols columns of one token of grad x, 256 per wave.  `add` may be grad_x.
__device__ __forceinline__ void dx_item(const float* __restrict__ wr,
                                        const Slot* __restrict__ slots, const uint16_t* add,
                                        uint16_t* grad_x, int64_t t, int slab, int H) {
  const int col = slab * kDxCols + 4 * threadIdx.x;
  if (col >= H) return;
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
    const Slot s = slots[t * 8 + j];
    d[j] = s.dz;
    q[j] = s.expert < kE ? *reinterpret_cast<const float4*>(wr + (size_t)s.expert * H + col)
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

// Both products in one launch (they are independent): the first dw_items
// workgroups take (slab, chunk), the rest (slab, token).  Within each part
// XCD b mod 8 walks a contiguous eighth of the slab-major items.
__global__ __launch_bounds__(256) void route_grad_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ wr,
    const int32_t* __restrict__ perm_src, const Slot* __restrict__ slots, int32_t* plan,
    int64_t chunks, const uint16_t* add, float* __restrict__ grad_w, int accumulate,
    float* __restrict__ part, uint16_t* grad_x, int64_t T, int H, int topk,
    uint32_t dw_end) {
  __shared__ DwShared sh;
  const int slabs = H / kSlab;
  // fewer than 2^24 workgroups: 32-bit arithmetic
  uint32_t b = blockIdx.x;
  if (b < dw_end) {
    const uint32_t item = (b & 7) * (dw_end / 8) + (b >> 3);
    const int slab = item / (uint32_t)chunks, chunk = item - slab * (uint32_t)chunks;
    const Plan pl = plan_of(plan, chunks);
    if (slab >= slabs || chunk >= pl.first[kE]) return;
    dw_item(x, perm_src, slots, pl, chunk, slab, grad_w, accumulate, part, T * topk, H, topk, sh);
  } else {
    b -= dw_end;
    const uint32_t item = (b & 7) * ((gridDim.x - dw_end) / 8) + (b >> 3);
    const int slab = item / (uint32_t)T;
    if (slab * kDxCols >= H) return;
    dx_item(wr, slots, add, grad_x, item - slab * (uint32_t)T, slab, H);
  }
}

// Batches of at most kSmallTokens tokens in one launch.  Their few pairs have
// few rows per expert, so a workgroup of the grad W part takes one expert and
// 2048 columns (a thread 8 of them, over all the expert's rows), and works out
// the dz of the whole batch by itself; one of the grad x part takes a token and
// 1024 columns, and works out its 8 slots.  The launches, not the work, are
// what such a batch costs (128 tokens of 5120 columns: 13.4 against 19.9 us for
// a call, 14.2 with the tokens on few experts; 256 tokens would take 18.7 and,
// on few experts, 24.9 against 19.6).
constexpr int kSmallTokens = 128, kSmallCols = 256 * 8;
__global__ __launch_bounds__(256) void route_grad_small_kernel(
    const uint16_t* __restrict__ x, const float* __restrict__ wr, const int32_t* __restrict__ ids,
    const float* __restrict__ logits, const float* __restrict__ grad_topk_w,
    const int32_t* __restrict__ perm_src, const int32_t* __restrict__ offsets,
    const uint16_t* add, float* __restrict__ grad_w, int accumulate, uint16_t* grad_x, int T,
    int H, int topk, int renormalize, int dw_end) {
  const int lane = threadIdx.x % kWave;
  if ((int)blockIdx.x >= dw_end) {
    const int b = blockIdx.x - dw_end, t = b % T, col = b / T * kDxCols + 4 * threadIdx.x;
    const Slot s = slot_of(ids, logits, grad_topk_w, t, lane % 8, T, topk, renormalize);
    if (col >= H) return;
    const int64_t at = (int64_t)t * H + col;
    u32x2_t a = {0u, 0u};
    if (add) a = *reinterpret_cast<const u32x2_t*>(add + at);
    float4 q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = __builtin_amdgcn_readlane(s.expert, j);
      q[j] = e < kE ? *reinterpret_cast<const float4*>(wr + (size_t)e * H + col)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float4 acc = make_float4(bf16_to_f32(a[0] & 0xffffu), __uint_as_float(a[0] & 0xffff0000u),
                             bf16_to_f32(a[1] & 0xffffu), __uint_as_float(a[1] & 0xffff0000u));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s.dz), j));
      acc.x += d * q[j].x; acc.y += d * q[j].y;
      acc.z += d * q[j].z; acc.w += d * q[j].w;
    }
    *reinterpret_cast<u32x2_t*>(grad_x + at) =
        u32x2_t{pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w)};
    return;
  }
  __shared__ float batch_dz[kSmallTokens * 8], dz[kSmallTokens * 8];
  __shared__ int token[kSmallTokens * 8], kept;
  const int e = blockIdx.x % kE, col = (int)(blockIdx.x / kE) * kSmallCols + 8 * threadIdx.x;
  const int n = T * topk;
  const int lo = min(max(offsets[e], 0), n);
  int rows = min(max(offsets[e + 1], lo), n) - lo;
  if (rows > 0) {  // the same for the whole workgroup
    if (threadIdx.x == 0) kept = rows;
    for (int i = threadIdx.x; i < kSmallTokens * 8; i += 256)
      batch_dz[i] = slot_of(ids, logits, grad_topk_w, i / 8, i % 8, T, topk, renormalize).dz;
    __syncthreads();
    for (int i = threadIdx.x; i < rows; i += 256) {
      const int p = perm_src[lo + i];
      const bool ok = p >= 0 && p < n;
      const int t = ok ? p / topk : 0;
      token[i] = ok ? t : -1;
      dz[i] = ok ? batch_dz[t * 8 + (p - t * topk)] : 0.f;
      if (!ok) kept = -1;
    }
    __syncthreads();
    // pairs outside the batch have no row to add: they leave the list, in the
    // rare case by one thread, so that the loop below has nothing to check
    // (checked per row, 128 tokens on few experts took 16.5 instead of 15.3 us)
    if (__builtin_amdgcn_readfirstlane(kept) < 0) {
      __syncthreads();  // everyone has read it
      if (threadIdx.x == 0) {
        int k = 0;
        for (int i = 0; i < rows; ++i) {
          if (token[i] < 0) continue;
          token[k] = token[i];
          dz[k++] = dz[i];
        }
        kept = k;
      }
      __syncthreads();
      rows = __builtin_amdgcn_readfirstlane(kept);
    }
  }
  if (col >= H) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < rows; ++i) {
    const uint4 q = ld16(x + (int64_t)token[i] * H + col);
    const float d = dz[i];
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      acc[2 * c] += d * bf16_to_f32(u[c] & 0xffffu);
      acc[2 * c + 1] += d * __uint_as_float(u[c] & 0xffff0000u);
    }
  }
  float4* o = reinterpret_cast<float4*>(grad_w + (size_t)e * H + col);
  if (accumulate) {
    const float4 a = o[0], b = o[1];
    acc[0] = a.x + acc[0]; acc[1] = a.y + acc[1]; acc[2] = a.z + acc[2]; acc[3] = a.w + acc[3];
    acc[4] = b.x + acc[4]; acc[5] = b.y + acc[5]; acc[6] = b.z + acc[6]; acc[7] = b.w + acc[7];
  }
  o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// grad x of large batches: a workgroup holds 128 columns of all 256 experts'
// weights in LDS (128 KB, read at twice the rate of L1) and walks its share of
// the tokens, 8 per wave at a time; the next 8 tokens' slots and `add` are on
// their way meanwhile.  `add` may be grad_x.
constexpr int kLdsCols = 128, kLdsWaves = 16, kLdsTokens = 8;
__global__ __launch_bounds__(kLdsWaves * 64) void route_dx_kernel(
    const float* __restrict__ wr, const Slot* __restrict__ slots, const uint16_t* add,
    uint16_t* grad_x, int64_t T, int H, int64_t share) {
  __shared__ float4 w4[(kE + 1) * kLdsCols / 4];  // the last row, of an empty slot, is zero
  const int slabs = H / kLdsCols;
  const int slab = blockIdx.x % slabs;
  const int64_t part = blockIdx.x / slabs;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int64_t end = min(T, (part + 1) * share);
  const int col = slab * kLdsCols + 2 * lane;
  constexpr int kStep = kLdsWaves * kLdsTokens;
  int64_t t0 = part * share + wave * kLdsTokens;
  // lane 8u + j holds slot j of token t0 + u
  const auto load = [&](int64_t t, Slot& s, uint32_t (&a)[kLdsTokens]) {
    s = slots[min(t * 8 + lane, end * 8 - 1)];
#pragma unroll
    for (int u = 0; u < kLdsTokens; ++u)
      a[u] = add ? *reinterpret_cast<const uint32_t*>(add + min(t + u, end - 1) * H + col) : 0u;
  };
  Slot next;
  uint32_t next_a[kLdsTokens];
  load(t0, next, next_a);
#pragma unroll
  for (int i = threadIdx.x; i < kE * kLdsCols / 4; i += kLdsWaves * 64) {
    const int e = i / (kLdsCols / 4), c = i % (kLdsCols / 4);
    w4[i] = *reinterpret_cast<const float4*>(wr + (size_t)e * H + slab * kLdsCols + 4 * c);
  }
  if (threadIdx.x < kLdsCols / 4)
    w4[kE * kLdsCols / 4 + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  const float2* w2 = reinterpret_cast<const float2*>(w4) + lane;  // row stride kLdsCols / 2
  for (; t0 < end; t0 += kStep) {
    const Slot now = next;
    uint32_t a[kLdsTokens];
#pragma unroll
    for (int u = 0; u < kLdsTokens; ++u) a[u] = next_a[u];
    if (t0 + kStep < end) load(t0 + kStep, next, next_a);
#pragma unroll
    for (int u = 0; u < kLdsTokens; ++u) {
      float2 q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        q[j] = w2[__builtin_amdgcn_readlane(now.expert, 8 * u + j) * (kLdsCols / 2)];
      float ax = bf16_to_f32(a[u] & 0xffffu), ay = __uint_as_float(a[u] & 0xffff0000u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = __uint_as_float(
            __builtin_amdgcn_readlane(__float_as_uint(now.dz), 8 * u + j));
        ax += d * q[j].x;
        ay += d * q[j].y;
      }
      if (t0 + u < end)
        __builtin_nontemporal_store(pack_bf16x2(ax, ay),
                                    reinterpret_cast<uint32_t*>(grad_x + (t0 + u) * H + col));
    }
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
int64_t dw_blocks(int64_t T, int H, int topk) {
  return (chunks_of(T * topk) * (H / kSlab) + 7) / 8 * 8;
}
int64_t dx_blocks(int64_t T, int64_t H) {
  return (T * ((H + kDxCols - 1) / kDxCols) + 7) / 8 * 8;
}
// whether grad x, where wanted, is route_grad_kernel's (else route_dx_kernel's)
bool dx_beside_dw(int64_t T) { return T < kLdsFrom; }

}  // namespace

RouteGradWs route_grad_ws(int64_t T, int H, int topk) {
  if (T <= kSmallTokens) return {0, 0, 0};
  const int64_t n = T * topk, chunks = chunks_of(n);
  RouteGradWs w;
  w.dz = (size_t)T * 8 * sizeof(Slot);
  w.plan = (size_t)(3 * chunks + kE + 1) * sizeof(int32_t);
  w.part = n > kRouteChunk ? (size_t)chunks * H * sizeof(float) : 0;
  return w;
}

bool route_grad_fits(int64_t T, int H, int topk, bool grad_x) {
  // a grid holds fewer than 2^32 threads.  The other launches' are smaller than
  // this one's, but for the one of 8 threads per token.
  const int64_t blocks =
      dw_blocks(T, H, topk) + (grad_x && dx_beside_dw(T) ? dx_blocks(T, H) : 0);
  return blocks < (int64_t)1 << 24 && (T / 32 + 2) * 256 < (int64_t)1 << 32;
}

hipError_t launch_route_backward(const uint16_t* x, const float* wr, const int32_t* ids,
                                 const float* logits, const float* grad_topk_w,
                                 const int32_t* perm_src, const int32_t* offsets,
                                 const uint16_t* add, float* grad_w, int accumulate,
                                 uint16_t* grad_x, int64_t T, int H, int topk, int renormalize,
                                 void* dz, int32_t* plan, float* part, hipStream_t stream) {
  if (T <= kSmallTokens) {
    const int dw = kE * ((H + kSmallCols - 1) / kSmallCols);
    const int dx = grad_x ? (int)T * ((H + kDxCols - 1) / kDxCols) : 0;
    hipLaunchKernelGGL(route_grad_small_kernel, dim3(dw + dx), dim3(256), 0, stream, x, wr, ids,
                       logits, grad_topk_w, perm_src, offsets, add, grad_w, accumulate, grad_x,
                       (int)T, H, topk, renormalize, dw);
    return hipGetLastError();
  }
  Slot* slots = static_cast<Slot*>(dz);
  const int64_t n = T * topk, chunks = chunks_of(n), slabs = H / kSlab;
  hipLaunchKernelGGL(route_dz_kernel, dim3((unsigned)((T + 31) / 32 + 1)), dim3(256), 0, stream,
                     ids, logits, grad_topk_w, slots, offsets, plan, chunks, T, topk, renormalize);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool lds_dx = grad_x && !dx_beside_dw(T);
  const int64_t dw = dw_blocks(T, H, topk), dx = grad_x && !lds_dx ? dx_blocks(T, H) : 0;
  hipLaunchKernelGGL(route_grad_kernel, dim3((unsigned)(dw + dx)), dim3(256), 0, stream, x, wr,
                     perm_src, slots, plan, chunks, add, grad_w, accumulate, part, grad_x, T, H,
                     topk, (uint32_t)dw);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (lds_dx) {
    // as many workgroups as there are CUs, each with an equal share of tokens
    const int cols = H / kLdsCols;
    int64_t parts = cols < 256 ? 256 / cols : 1;
    const int64_t share = (T + parts - 1) / parts;
    parts = (T + share - 1) / share;
    hipLaunchKernelGGL(route_dx_kernel, dim3((unsigned)(cols * parts)), dim3(kLdsWaves * 64), 0,
                       stream, wr, slots, add, grad_x, T, H, share);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (n <= kRouteChunk) return hipSuccess;  // no expert has a second chunk
  hipLaunchKernelGGL(route_dw_reduce_kernel, dim3(kE, (unsigned)slabs), dim3(256), 0, stream, plan,
                     chunks, part, grad_w, H, accumulate);
  return hipGetLastError();
}

}  // namespace beam
