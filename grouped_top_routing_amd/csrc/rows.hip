// Rows moved between token order and expert-major order, and the gradients of
// both directions (gfx950).
//
// Pair p = t*topk + j (slot j of token t) has row r = perm_dst[p] of the
// sorted order; a perm_dst outside [0, T*topk) (-1 from the permutation) names
// no row and the pair is dropped.  With a the token rows, b the sorted rows:
//   dispatch            b[r] = w[p] * a[t]                 (w = 1 without weights)
//   dispatch, backward  grad a[t] = sum_j w[p] * grad b[r],  grad w[p] = <a[t], grad b[r]>
//   combine             out[t] = c * sum_j w[p] * b[r]
//   combine, backward   grad b[r] = c * w[p] * grad out[t],  grad w[p] = c * <grad out[t], b[r]>
// (c the routed scaling).  bf16 rows of a multiple of 256 elements are combined
// by combine.hip; the combine here takes fp32 rows and other widths.
//
// All of it is bound by HBM: per token one row of the token order and topk
// rows of the sorted order move once.  Both kernels are therefore laid out by
// token: the token's row is read once and held in registers while its topk
// rows are written (or read), and the indices are wave-uniform scalar loads.
// Sums are fp32 in slot order, each result is rounded once, and there are no
// atomics: a row of the sorted order has one writer.
#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

// 16 bytes at any element's alignment: gfx950 reads and writes unaligned
// global memory in one instruction, so rows of odd length take the same path.
typedef unsigned v4u_t __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 ld16u(const void* p) {
  const v4u_t v = *static_cast<const v4u_t*>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint4 ld16u_nt(const void* p) {
  const v4u_t v = __builtin_nontemporal_load(static_cast<const v4u_t*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool NT>
__device__ __forceinline__ void st16u(void* p, uint4 v) {
  const v4u_t q = {v.x, v.y, v.z, v.w};
  if constexpr (NT) __builtin_nontemporal_store(q, static_cast<v4u_t*>(p));
  else *static_cast<v4u_t*>(p) = q;
}

// Cache policy.  Sorted rows are read once: non-temporal loads (dispatch then
// its gradient, 5120 bf16 columns: 169 -> 122 us at 4096 tokens, no difference
// at 512).  Sorted rows that are written are read next, by the experts or
// their gradient: up to twice the 256 MB last-level cache a plain store leaves
// enough of them there (same chain, plain against non-temporal stores: 58
// against 69 us at 2048 tokens, 122 against 131 at 4096 with 335 MB), past it
// only displaces what is still to be read (275 against 255 us at 8192 tokens,
// 577 against 502 at 16384).  Token rows, an eighth of that, are written
// non-temporally (the gradient of dispatch and a kernel that reads it, 4096
// tokens: 88 -> 86 us, 16384: 360 -> 337).
constexpr int64_t kCachedBytes = (int64_t)512 << 20;

// The row types: storage S, elements per 16 bytes, conversions.
struct Bf16Rows {
  using S = uint16_t;
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(uint4 q, float (&f)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      f[2 * c] = bf16_to_f32(u[c] & 0xffffu);
      f[2 * c + 1] = __uint_as_float(u[c] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 round(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float get(const S* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void put(S* p, float v) { *p = (S)(pack_bf16x2(v, 0.f)); }
};
struct F32Rows {
  using S = float;
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(uint4 q, float (&f)[4]) {
    f[0] = __uint_as_float(q.x); f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z); f[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 round(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float get(const S* p) { return *p; }
  static __device__ __forceinline__ void put(S* p, float v) { *p = v; }
};

// A row's pieces of 16 bytes.  Where N does not divide H the last one starts
// at H - N and repeats the end of the one before it (the same values are
// written twice; a dot product leaves the repeated elements out): a lane that
// took the odd elements one by one would hold up its wave (777 bf16 columns,
// 4000 tokens: gradient of dispatch 21.1 -> 16.4 us, of combine 29.4 -> 24.1).
// Rows shorter than a piece are one piece, taken element by element.
__host__ __device__ constexpr int pieces(int H, int N) { return (H + N - 1) / N; }

// Rows of the token's slots, -1 where a slot names none.
template <int K>
__device__ __forceinline__ void slot_rows(const int32_t* __restrict__ perm_dst, int64_t t,
                                          int topk, int64_t n, int64_t (&rows)[K]) {
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t r = j < topk ? perm_dst[t * topk + j] : -1;
    rows[j] = r >= 0 && r < n ? r : -1;
  }
}

// ---------------------------------------------------------------------------
// dispatch: thread (x, y) of a workgroup handles one piece of item
// blockIdx.x * blockDim.y + y, an item being (token, slice of blockDim.x
// pieces).  Where blockDim.x is a multiple of 64 a wave has one token and its
// indices are scalars; NARROW rows (at most 32 pieces) share a wave.
template <class R, bool WEIGHTED, bool NT, bool NARROW>
__global__ __launch_bounds__(256) void dispatch_kernel(
    const typename R::S* __restrict__ x, const int32_t* __restrict__ perm_dst,
    const float* __restrict__ w, typename R::S* __restrict__ out, int64_t T, int64_t n, int H,
    int topk, int slices) {
  constexpr int N = R::N;
  // a launch has at most 2^31 threads: 32-bit items
  const uint32_t item = blockIdx.x * blockDim.y + threadIdx.y;
  const uint32_t it = NARROW ? item : item / (uint32_t)slices;
  const int64_t t = NARROW ? (int)it : __builtin_amdgcn_readfirstlane((int)it);
  const int v = (int)(NARROW ? 0 : item - it * slices) * blockDim.x + threadIdx.x;
  if (t >= T || v * N >= H) return;
  int64_t rows[8];
  slot_rows(perm_dst, t, topk, n, rows);
  if (H >= N) {
    const int at = min(v * N, H - N);
    const uint4 q = ld16u(x + t * H + at);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (rows[j] < 0) continue;
      uint4 o = q;
      if constexpr (WEIGHTED) {
        const float wt = w[t * topk + j];
        float f[N];
        R::widen(q, f);
#pragma unroll
        for (int c = 0; c < N; ++c) f[c] *= wt;
        o = R::round(f);
      }
      st16u<NT>(out + rows[j] * H + at, o);
    }
  } else {
    for (int c = 0; c < H; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (rows[j] < 0) continue;
        if constexpr (WEIGHTED)
          R::put(out + rows[j] * H + c, w[t * topk + j] * R::get(x + t * H + c));
        else
          out[rows[j] * H + c] = x[t * H + c];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// SCATTER: b[r] = (c*w) * a[t] (the combine's gradient); otherwise a[t] =
// c * sum_j w * b[r] (the dispatch's gradient with c = 1, and the combine).
// DOT: grad w[p] = c * <a[t], b[r]>.
// Threads (.., y) of a workgroup share one token; for DOT blockDim.x threads
// cover the whole row and its waves' sums meet in LDS.  NARROW rows (at most 32
// pieces, one each of blockDim.x = 8, 16 or 32 threads) share a wave.
template <class R, bool SCATTER, bool DOT, bool WRITE, bool NT, bool NARROW>
__global__ __launch_bounds__(NARROW ? 256 : 1024) void row_grad_kernel(
    const typename R::S* __restrict__ a, const typename R::S* __restrict__ b,
    const int32_t* __restrict__ perm_dst, const float* __restrict__ w,
    typename R::S* __restrict__ out, float* __restrict__ grad_w, int64_t T, int64_t n, int H,
    int topk, float scale) {
  constexpr int N = R::N;
  const int token = (int)(blockIdx.x * (int64_t)blockDim.y + threadIdx.y);
  const int64_t t = NARROW ? token : __builtin_amdgcn_readfirstlane(token);
  int64_t rows[8];
  float wt[8], dot[8];
  if (t < T) slot_rows(perm_dst, t, topk, n, rows);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (t >= T) rows[j] = -1;
    wt[j] = w && j < topk && t < T ? (SCATTER ? scale * w[t * topk + j] : w[t * topk + j]) : 1.f;
    dot[j] = 0.f;
  }
  const int nv = t < T ? pieces(H, N) : 0;
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    if (H >= N) {
      const int start = min(v * N, H - N), twice = v * N - start;
      uint4 qb[8];
      if constexpr (DOT || !SCATTER) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          qb[j] = rows[j] >= 0 ? ld16u_nt(b + rows[j] * H + start) : make_uint4(0u, 0u, 0u, 0u);
      }
      float fa[N];
      if constexpr (DOT || SCATTER) R::widen(ld16u_nt(a + t * H + start), fa);
      float acc[N];
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (rows[j] < 0) continue;
        if constexpr (DOT || !SCATTER) {
          float fb[N];
          R::widen(qb[j], fb);
          if constexpr (DOT) {
            if (twice == 0) {  // every piece but the last of an odd row
#pragma unroll
              for (int c = 0; c < N; ++c) dot[j] += fa[c] * fb[c];
            } else {
#pragma unroll
              for (int c = 0; c < N; ++c)
                if (c >= twice) dot[j] += fa[c] * fb[c];
            }
          }
          if constexpr (!SCATTER)
#pragma unroll
            for (int c = 0; c < N; ++c) acc[c] += wt[j] * fb[c];
        }
        if constexpr (SCATTER && WRITE) {
          float o[N];
#pragma unroll
          for (int c = 0; c < N; ++c) o[c] = wt[j] * fa[c];
          st16u<NT>(out + rows[j] * H + start, R::round(o));
        }
      }
      if constexpr (!SCATTER) {
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] *= scale;
        st16u<true>(out + t * H + start, R::round(acc));
      }
    } else {
      for (int c = 0; c < H; ++c) {
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (rows[j] < 0) continue;
          const int64_t bt = rows[j] * H + c;
          if constexpr (DOT) dot[j] += R::get(a + t * H + c) * R::get(b + bt);
          if constexpr (!SCATTER) acc += wt[j] * R::get(b + bt);
          if constexpr (SCATTER && WRITE) R::put(out + bt, wt[j] * R::get(a + t * H + c));
        }
        if constexpr (!SCATTER) R::put(out + t * H + c, scale * acc);
      }
    }
  }
  if constexpr (DOT && NARROW) {
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      for (int off = blockDim.x / 2; off >= 1; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
      if ((int)threadIdx.x == j) mine = dot[j];
    }
    if (t < T && (int)threadIdx.x < topk) grad_w[t * topk + threadIdx.x] = scale * mine;
  } else if constexpr (DOT) {
    __shared__ float part[16][8];  // 16 waves of at most 1024 threads
    const int waves = blockDim.x / kWave;  // of one token
    const int wave = (threadIdx.y * blockDim.x + threadIdx.x) / kWave;
    // the 8 sums across a wave in 10 exchanges: at each of the first three
    // a lane hands half of its sums over and keeps the other half, so that
    // lanes 8j .. 8j + 7 end up with the parts of sum j
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
      const bool up = lane & (8 * half);
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const float keep = up ? dot[j + half] : dot[j], give = up ? dot[j] : dot[j + half];
        dot[j] = keep + __shfl_xor(give, 8 * half);
      }
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) dot[0] += __shfl_xor(dot[0], off);
    if (lane % 8 == 0) part[wave][lane / 8] = dot[0];
    __syncthreads();
    if (t < T && (int)threadIdx.x < topk) {
      float s = 0.f;
      for (int i = 0; i < waves; ++i) s += part[threadIdx.y * waves + i][threadIdx.x];
      grad_w[t * topk + threadIdx.x] = scale * s;
    }
  }
}

// Threads of a narrow row: 8, 16 or 32, as many as it has pieces or more; 0 for
// a wider row.  (16000 tokens of 64 bf16 columns, 8 slots, a wave per token
// against 8: dispatch 9.9 -> 6.5 us, its gradient 16.4 -> 7.8.)
int narrow_threads(int nv) { return nv <= 8 ? 8 : nv <= 16 ? 16 : nv <= 32 ? 32 : 0; }

// A grid holds fewer than 2^32 threads: batches past half of that go in
// several launches over ranges of tokens.
constexpr int64_t kLaunchThreads = (int64_t)1 << 31;

template <class R>
hipError_t dispatch(const void* x, const int32_t* perm_dst, const float* w, void* out, int64_t T,
                    int H, int topk, hipStream_t stream) {
  using S = typename R::S;
  const int nv = pieces(H, R::N);
  // threads per item: of 256, 128 and 64, the one with the fewest idle lanes
  const int few = narrow_threads(nv);
  int tx = few ? few : 64;
  for (int c = 128; !few && c <= 256; c *= 2)
    if ((nv + c - 1) / c * c <= (nv + tx - 1) / tx * tx) tx = c;
  const int slices = (nv + tx - 1) / tx, ty = 256 / tx;
  const int64_t n = T * topk;
  const bool nt_out = n * H * (int64_t)sizeof(S) > kCachedBytes;
  int64_t most = kLaunchThreads / ((int64_t)slices * tx);
  if (most < 1) most = 1;
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    const int64_t nt = T - t0 < most ? T - t0 : most;
    const dim3 grid((unsigned)((nt * slices + ty - 1) / ty)), block(tx, ty);
#define BEAM_PICK(W, NT) (few ? dispatch_kernel<R, W, NT, true> : dispatch_kernel<R, W, NT, false>)
    const auto kernel = w ? (nt_out ? BEAM_PICK(true, true) : BEAM_PICK(true, false))
                          : (nt_out ? BEAM_PICK(false, true) : BEAM_PICK(false, false));
#undef BEAM_PICK
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, static_cast<const S*>(x) + t0 * H,
                       perm_dst + t0 * topk, w ? w + t0 * topk : nullptr, static_cast<S*>(out), nt,
                       n, H, topk, slices);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <class R, bool SCATTER, bool DOT, bool WRITE>
hipError_t row_grad(const void* a, const void* b, const int32_t* perm_dst, const float* w,
                    void* out, float* grad_w, int64_t T, int H, int topk, float scale,
                    hipStream_t stream) {
  using S = typename R::S;
  const int nv = pieces(H, R::N), few = narrow_threads(nv), waves = (nv + kWave - 1) / kWave;
  // one round of at most 1024 threads over the row, or equal rounds
  const int rounds = (waves + 15) / 16;
  const int tx = few ? few : kWave * ((waves + rounds - 1) / rounds);
  const int ty = tx >= 256 ? 1 : 256 / tx;
  const int64_t n = T * topk, most = kLaunchThreads / tx;
  constexpr bool writes_sorted = SCATTER && WRITE;
  const bool nt_out = !writes_sorted || n * H * (int64_t)sizeof(S) > kCachedBytes;
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    const int64_t nt = T - t0 < most ? T - t0 : most;
    const S* as = static_cast<const S*>(a);
    S* o = static_cast<S*>(out);
#define BEAM_PICK(NT)                                          \
  (few ? row_grad_kernel<R, SCATTER, DOT, WRITE, NT, true>     \
       : row_grad_kernel<R, SCATTER, DOT, WRITE, NT, false>)
    const auto kernel = nt_out ? BEAM_PICK(true) : BEAM_PICK(!writes_sorted);
#undef BEAM_PICK
    hipLaunchKernelGGL(kernel, dim3((unsigned)((nt + ty - 1) / ty)), dim3(tx, ty), 0, stream,
                       as ? as + t0 * H : nullptr, static_cast<const S*>(b),
                       perm_dst + t0 * topk, w ? w + t0 * topk : nullptr,
                       SCATTER ? o : o + t0 * H, grad_w ? grad_w + t0 * topk : nullptr, nt, n, H,
                       topk, scale);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_dispatch(bool fp32, const void* x, const int32_t* perm_dst, const float* w,
                           void* out, int64_t T, int H, int topk, hipStream_t stream) {
  return fp32 ? dispatch<F32Rows>(x, perm_dst, w, out, T, H, topk, stream)
              : dispatch<Bf16Rows>(x, perm_dst, w, out, T, H, topk, stream);
}

hipError_t launch_dispatch_backward(bool fp32, const void* grad, const int32_t* perm_dst,
                                    const float* w, const void* x, void* grad_x, float* grad_w,
                                    int64_t T, int H, int topk, hipStream_t stream) {
#define BEAM_GRAD(R, DOT)                                                                     \
  row_grad<R, false, DOT, true>(x, grad, perm_dst, w, grad_x, grad_w, T, H, topk, 1.f, stream)
  if (fp32) return grad_w ? BEAM_GRAD(F32Rows, true) : BEAM_GRAD(F32Rows, false);
  return grad_w ? BEAM_GRAD(Bf16Rows, true) : BEAM_GRAD(Bf16Rows, false);
#undef BEAM_GRAD
}

hipError_t launch_combine_rows(bool fp32, const void* y, const int32_t* perm_dst, const float* w,
                               void* out, int64_t T, int H, int topk, float scale,
                               hipStream_t stream) {
  return fp32 ? row_grad<F32Rows, false, false, true>(nullptr, y, perm_dst, w, out, nullptr, T, H,
                                                      topk, scale, stream)
              : row_grad<Bf16Rows, false, false, true>(nullptr, y, perm_dst, w, out, nullptr, T,
                                                       H, topk, scale, stream);
}

hipError_t launch_combine_backward(bool fp32, const void* grad_out, const void* y,
                                   const int32_t* perm_dst, const float* w, void* grad_y,
                                   float* grad_w, int64_t T, int H, int topk, float scale,
                                   hipStream_t stream) {
#define BEAM_GRAD(R, DOT, WRITE)                                                             \
  row_grad<R, true, DOT, WRITE>(grad_out, y, perm_dst, w, grad_y, grad_w, T, H, topk, scale, \
                                stream)
  if (fp32) {
    if (!grad_y) return BEAM_GRAD(F32Rows, true, false);
    return grad_w ? BEAM_GRAD(F32Rows, true, true) : BEAM_GRAD(F32Rows, false, true);
  }
  if (!grad_y) return BEAM_GRAD(Bf16Rows, true, false);
  return grad_w ? BEAM_GRAD(Bf16Rows, true, true) : BEAM_GRAD(Bf16Rows, false, true);
#undef BEAM_GRAD
}

}  // namespace beam
