// Expert SwiGLU MLPs with 4-bit weights and group scales on gfx950.
//
// Each expert matrix row n holds E2M1 codes q[n, k] (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives) and one E8M0 scale per 32 consecutive k:
//   w[n, k] = 2^(s[n, k / 32] - 127) * q[n, k]
// Activations stay bf16.  A code times a power of two is a bf16 value (two
// mantissa bits), so v_cvt_scalef32_pk_bf16_fp4 widens two codes and applies
// their scale without a rounding, the products are exact in the fp32
// accumulator of v_mfma_f32_16x16x32_bf16, and a group of 32 k is one MFMA
// step.
//
// Packed layout (moe_quantize_fp4, moe_pack_fp4): each expert's [N, K] matrix
// is stored as [N/16][K/128] fragments.  A code fragment is [64 lanes][4][4
// bytes]: lane l, word s holds the 8 codes of row 16b + l%16 at k = 128 st +
// 32 s + 8 (l/16) .. +7 (lower k in lower bits), so that one 16-byte read per
// lane brings its operands of four MFMA steps.  A scale fragment is [16 rows]
// [4 bytes], one byte per 32 k.
#include "common.h"
#include "kernels.h"

namespace beam {

namespace {

constexpr int kStageK = 128;    // k per fragment
constexpr int kCodeB = 1024;    // bytes of a code fragment (16 rows x 128 k)
constexpr int kScaleB = 64;     // bytes of its scales

// E2M1 code of |v| <= 7, to the nearest, ties to the even code.
__device__ __forceinline__ uint32_t e2m1_rne(float v) {
  const float a = fabsf(v);
  const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                     (a >= 3.5f) + (a > 5.0f);
  return c | (v < 0.f ? 8u : 0u);
}

// E8M0 code of the least power of two, at least 2^-126, by which `most` is at
// most 7 (7 rounds to 6: at most half a step away, as everywhere else).  Code
// 255 (NaN) where `most` is not finite.
__device__ __forceinline__ uint32_t e8m0_of(float most) {
  const uint32_t u = __float_as_uint(most);
  if (u >= 0x7f800000u) return 255u;
  const int c = (int)(u >> 23) - 2 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(c < 1 ? 1 : c);
}

__device__ __forceinline__ float e8m0_value(uint32_t code) { return __uint_as_float(code << 23); }

}  // namespace

// One thread per 32 consecutive weights of a row.
__global__ __launch_bounds__(256) void quantize_fp4_kernel(const uint16_t* __restrict__ w,
                                                           uint8_t* __restrict__ q,
                                                           uint8_t* __restrict__ s, int K,
                                                           int64_t groups) {
  const int per = K / 32;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;  // of all experts: N is a multiple of 16
    const int g = (int)(i - row * per);
    const uint16_t* src = w + row * K + g * 32;
    float v[32], most = 0.f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 u = ld16(src + 8 * c);
      const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * c + 2 * j] = bf16_to_f32(p[j] & 0xffffu);
        v[8 * c + 2 * j + 1] = bf16_to_f32(p[j] >> 16);
      }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      bad = bad || !(fabsf(v[j]) <= 3.4028234e38f);
      most = fmaxf(most, fabsf(v[j]));
    }
    const uint32_t code = bad ? 255u : e8m0_of(most);
    // 1 / scale: exact, 2^(127 - code), code in [1, 253]
    const float inv = __uint_as_float((254u - (bad ? 127u : code)) << 23);
    const int st = g >> 2, step = g & 3, r = (int)(row & 15);
    const int64_t frag = (row >> 4) * (K / kStageK) + st;
    s[frag * kScaleB + r * 4 + step] = (uint8_t)code;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) word |= e2m1_rne(v[8 * c + j] * inv) << (4 * j);
      *reinterpret_cast<uint32_t*>(q + frag * kCodeB + (c * 16 + r) * 16 + step * 4) = word;
    }
  }
}

// Row-major codes (two per byte, the lower k in the low half) and scales into
// fragments: one thread per lane of a fragment.
__global__ __launch_bounds__(256) void pack_fp4_kernel(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales,
                                                       uint8_t* __restrict__ q,
                                                       uint8_t* __restrict__ s, int K,
                                                       int64_t lanes) {
  const int per = K / kStageK;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < lanes;
       i += (int64_t)gridDim.x * 256) {
    const int l = (int)(i & 63), r = l & 15, c = l >> 4;
    const int64_t frag = i >> 6;
    const int64_t block = frag / per;
    const int st = (int)(frag - block * per);
    const int64_t row = block * 16 + r;
    const uint8_t* src = codes + row * (K / 2) + st * 64 + 4 * c;
    uint4 v;
    v.x = *reinterpret_cast<const uint32_t*>(src);
    v.y = *reinterpret_cast<const uint32_t*>(src + 16);
    v.z = *reinterpret_cast<const uint32_t*>(src + 32);
    v.w = *reinterpret_cast<const uint32_t*>(src + 48);
    st16(q + i * 16, v);
    if (c == 0)
      *reinterpret_cast<uint32_t*>(s + frag * kScaleB + r * 4) =
          *reinterpret_cast<const uint32_t*>(scales + row * (K / 32) + st * 4);
  }
}

// ---------------------------------------------------------------------------
// A work item is an m-tile of up to 64 rows of one expert times 256 of its
// weight rows (gate/up: 128 gate rows and the matching up rows).  Wave w of
// four takes column blocks 4w .. 4w + 3 (gate/up: gate blocks 2w, 2w + 1 and
// their up blocks).  Operands go straight from global memory to registers.
constexpr int kRowBlocks = 4;
constexpr int kColBlocks = 4;  // per wave

template <bool SWIGLU>
__global__ __launch_bounds__(256) void gemm_fp4_kernel(
    const uint16_t* __restrict__ A, const int32_t* __restrict__ gather, int topk,
    const uint8_t* __restrict__ Q, const uint8_t* __restrict__ S, uint16_t* __restrict__ C,
    const int32_t* __restrict__ plan, int max_tiles, int K, int n_out, int up_row0,
    GemmBounds bounds) {
  (void)bounds;
  constexpr int HALF = SWIGLU ? kColBlocks / 2 : kColBlocks;
  constexpr int WCOLS = 4 * HALF * 16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int* plan_expert = plan + 4;
  const int* plan_row0 = plan_expert + max_tiles;
  const int* plan_rows = plan_row0 + max_tiles;
  const int nt_n = n_out / WCOLS;
  const int total = plan[0] * nt_n;
  const int nst = K / kStageK;
  const int64_t wrows = SWIGLU ? 2 * (int64_t)n_out : n_out;
  for (int q = blockIdx.x; q < total; q += gridDim.x) {
    const int tile = q / nt_n, ntile = q - tile * nt_n;
    const int e = BEAM_CLAMP(plan_expert[tile], 0, bounds.n_experts - 1, kCheckPlanRows);
    const int row0 = plan_row0[tile], nrows = plan_rows[tile];
    const int nrb = (nrows + 15) >> 4;
    const uint16_t* arow[kRowBlocks];
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i) {
      const int row = row0 + min(16 * i + r, nrows - 1);
      const int src = gather
          ? gather[BEAM_CLAMP(row, 0, bounds.n_rows - 1, kCheckGatherIndex)] / topk : row;
      arow[i] = A + (size_t)BEAM_CLAMP(src, 0, bounds.n_src - 1, kCheckTokenIndex) * K + 8 * g;
    }
    // column block j of this wave: its first weight row
    int64_t frag[kColBlocks];
#pragma unroll
    for (int j = 0; j < kColBlocks; ++j) {
      const int col = ntile * WCOLS + (wave * HALF + j % HALF) * 16 + (j >= HALF ? up_row0 : 0);
      frag[j] = ((int64_t)e * (wrows / 16) + BEAM_CLAMP(col / 16, 0, wrows / 16 - 1,
                                                         kCheckWeightOffset)) * nst;
    }
    f32x4_t acc[kRowBlocks][kColBlocks];
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i)
#pragma unroll
      for (int j = 0; j < kColBlocks; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int st = 0; st < nst; ++st) {
      uint4 code[kColBlocks];
      uint32_t scale[kColBlocks];
#pragma unroll
      for (int j = 0; j < kColBlocks; ++j) {
        code[j] = ld16(Q + (frag[j] + st) * kCodeB + 16 * lane);
        scale[j] = *reinterpret_cast<const uint32_t*>(S + (frag[j] + st) * kScaleB + 4 * r);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8_t b[kColBlocks];
#pragma unroll
        for (int j = 0; j < kColBlocks; ++j) {
          const uint32_t w = s == 0 ? code[j].x : s == 1 ? code[j].y : s == 2 ? code[j].z : code[j].w;
          b[j] = widen_fp4(w, e8m0_value((scale[j] >> (8 * s)) & 255u));
        }
#pragma unroll
        for (int i = 0; i < kRowBlocks; ++i)
          if (i < nrb) {
            const bf16x8_t a = as_bf16x8(ld16(arow[i] + st * kStageK + 32 * s));
#pragma unroll
            for (int j = 0; j < kColBlocks; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a, acc[i][j], 0, 0, 0);
          }
      }
    }
    // The weights are the first operand: lane (r, g) holds output columns
    // 4g .. 4g + 3 of row r.
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i) {
      const int row = 16 * i + r;
      if (row >= nrows) continue;
#pragma unroll
      for (int j = 0; j < HALF; ++j) {
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
          o[v] = SWIGLU ? silu_mul(acc[i][j][v], acc[i][j + (SWIGLU ? HALF : 0)][v]) : acc[i][j][v];
        const int col = ntile * WCOLS + (wave * HALF + j) * 16 + 4 * g;
        *reinterpret_cast<uint2*>(C + (size_t)(row0 + row) * n_out + col) =
            make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      }
    }
  }
}

// ---------------------------------------------------------------------------
int ffn_fp4_choose_mb(int64_t, int) { return kRowBlocks; }

hipError_t launch_grouped_gemm_fp4(int mb, bool swiglu, const uint16_t* A, const int32_t* gather,
                                   int topk, const uint8_t* Q, const uint8_t* S, uint16_t* C,
                                   const int32_t* plan, int max_tiles, int K, int n_out,
                                   int up_row0, hipStream_t stream, const GemmBounds& bounds) {
  if (mb != kRowBlocks) return hipErrorInvalidValue;
  const int64_t items = (int64_t)max_tiles * (n_out / (swiglu ? 128 : 256));
  const int64_t grid = persistent_grid(1024, items);
  if (swiglu)
    hipLaunchKernelGGL(gemm_fp4_kernel<true>, dim3((unsigned)grid), dim3(256), 0, stream, A,
                       gather, topk, Q, S, C, plan, max_tiles, K, n_out, up_row0, bounds);
  else
    hipLaunchKernelGGL(gemm_fp4_kernel<false>, dim3((unsigned)grid), dim3(256), 0, stream, A,
                       gather, topk, Q, S, C, plan, max_tiles, K, n_out, up_row0, bounds);
  return hipGetLastError();
}

// A grid of at most 2^20 workgroups, whose threads walk on from there.
static unsigned walk_blocks(int64_t threads) {
  const int64_t blocks = (threads + 255) / 256;
  return (unsigned)(blocks < 1 << 20 ? blocks : 1 << 20);
}

hipError_t launch_quantize_fp4(const uint16_t* w, uint8_t* q, uint8_t* s, int E, int N, int K,
                               hipStream_t stream) {
  const int64_t groups = (int64_t)E * N * K / 32;
  hipLaunchKernelGGL(quantize_fp4_kernel, dim3(walk_blocks(groups)), dim3(256), 0,
                     stream, w, q, s, K, groups);
  return hipGetLastError();
}

hipError_t launch_pack_fp4(const uint8_t* codes, const uint8_t* scales, uint8_t* q, uint8_t* s,
                           int E, int N, int K, hipStream_t stream) {
  const int64_t lanes = (int64_t)E * N * K / 32;
  hipLaunchKernelGGL(pack_fp4_kernel, dim3(walk_blocks(lanes)), dim3(256), 0, stream,
                     codes, scales, q, s, K, lanes);
  return hipGetLastError();
}

BEAM_DEFINE_CHECK_READER(check_flags_ffn_fp4)

}  // namespace beam
