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
// is stored as [N/16][K/128] fragments.  A code fragment is [2][64 lanes][2][4
// bytes]: half h, lane l, word s holds the 8 codes of row 16b + l%16 at k = 128 t
// + 64 h + 32 s + 8 (l/16) .. +7 (lower k in lower bits), so that one 8-byte read
// per lane brings its operands of two MFMA steps.  A scale fragment is [16 rows]
// [4 bytes], one byte per 32 k.
#include <type_traits>

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
      *reinterpret_cast<uint32_t*>(q + frag * kCodeB + (step >> 1) * (kCodeB / 2) +
                                   (c * 16 + r) * 8 + (step & 1) * 4) = word;
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
    uint2 lo, hi;
    lo.x = *reinterpret_cast<const uint32_t*>(src);
    lo.y = *reinterpret_cast<const uint32_t*>(src + 16);
    hi.x = *reinterpret_cast<const uint32_t*>(src + 32);
    hi.y = *reinterpret_cast<const uint32_t*>(src + 48);
    uint8_t* dst = q + frag * kCodeB + l * 8;
    *reinterpret_cast<uint2*>(dst) = lo;
    *reinterpret_cast<uint2*>(dst + kCodeB / 2) = hi;
    if (c == 0)
      *reinterpret_cast<uint32_t*>(s + frag * kScaleB + r * 4) =
          *reinterpret_cast<const uint32_t*>(scales + row * (K / 32) + st * 4);
  }
}

// ---------------------------------------------------------------------------
// The grouped GEMM.  A work item is an m-tile (up to 16 MB rows of one expert)
// times 256 of its weight rows (gate/up: 128 gate rows and the matching up
// rows), walked by a persistent grid.
//
// Waves form RG row groups x 4 column groups: a wave computes 4 column blocks
// (gate/up: 2 gate blocks and their up blocks) for its share of the item's
// 16-row blocks.  Codes, scales and rows are staged in LDS by direct loads:
//   W stage q: 128 k of the 16 blocks' code fragments (16 KB) and scales (1 KB),
//              in slot q % SW
//   A stage p: 64 k of the item's rows, 2 KB per row block, in slot p % SA; each
//              row's 128 bytes with its 16-byte chunks swizzled by (row / 2) % 8,
//              so that the 16 rows of an operand read hit distinct banks
// A wave reads its codes of 64 k once (8 bytes per block and lane) and widens them
// to bf16 operands in registers, one MFMA step ahead and between the MFMAs of the
// step before: an MFMA holds the matrix cores for 16 cycles and the issue port for
// 4, so that the conversions fit beside it.
//
// Schedule.  Iteration p (64 k, two MFMA steps) waits for A(p + 1), and W((p + 1)
// / 2) where that is new, passes a barrier, and refills the slots that every
// wave has read by then: A(p + SA), then for odd p W((p - 1) / 2 + SW) (codes of
// stage p are read after the barrier of iteration p - 1).  The loads before the
// loop are those of iterations below 0 in the same order, so one rule gives every
// wait (wait_next).  A workgroup issues its next item's
// first loads before the current item's outputs are written.
constexpr int kBlocks = 16;      // weight-row blocks of an item
constexpr int kCols = 4;         // column blocks per wave
constexpr int kColGroups = kBlocks / kCols;
constexpr int kSlotW = kBlocks * (kCodeB + kScaleB);
constexpr int kBlockA = 2048;    // bytes of 64 k of a row block

// One direct global -> LDS load of 4 bytes per lane (see lds_dma16_sv).
__device__ __forceinline__ void lds_dma4_sv(const void* base, uint32_t off, uint32_t lds_addr) {
  lds_addr = __builtin_amdgcn_readfirstlane(lds_addr);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %3\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(off), "s"(lds_addr), "s"(base)
      : "memory");
}

__device__ __forceinline__ int a_chunk(int row) { return (row >> 1) & 7; }

struct Fp4Args {
  const uint16_t* A;
  const int32_t* gather;
  int topk;
  const uint8_t* Q;
  const uint8_t* S;
  uint16_t* C;
  const int32_t* plan;
  int max_tiles, K, n_out, up_row0;
  GemmBounds bounds;
};

template <int MB, int RG, int SA, int SW, bool SWIGLU>
struct Fp4Gemm {
  static constexpr int NW = kColGroups * RG;
  static constexpr int NBL = kCols / RG;              // code fragments a wave loads per W stage
  static constexpr int AMAX = (MB + NW - 1) / NW;     // row blocks a wave loads per A stage
  static constexpr int RB = (MB + RG - 1) / RG;       // row blocks a wave computes, at most
  static constexpr int HALF = SWIGLU ? kCols / 2 : kCols;
  static constexpr int WCOLS = kColGroups * HALF * 16;
  static constexpr int kLoadsW = NBL + 1;             // direct loads of a W stage per wave
  static constexpr int kSlotA = MB * kBlockA;
  static constexpr int kLds = SW * kSlotW + SA * kSlotA;
  static_assert(SA % 2 == 1 && 2 * SW > SA + 1, "a W stage is issued before the A stage it is waited with");
  static_assert(kLds <= 160 * 1024, "LDS");

  const Fp4Args& a;
  uint8_t* lds;
  int lane, wave, r, g, cg, rg;
  int nst, nw;                 // A and W stages of an item
  // the item whose loads are in flight
  int row0, nrows, ntile, na;
  const uint16_t* arow[AMAX][2];  // this lane's 16 bytes of stage 0 of the rows it loads
  const uint8_t* code;            // expert's codes and scales, at the next W stage
  const uint8_t* scale;
  uint32_t code_off[NBL], scale_off;
  uint32_t next_a, next_w;        // slots that the next stages go to (bytes into the ring)

  __device__ __forceinline__ Fp4Gemm(const Fp4Args& args, uint8_t* mem) : a(args), lds(mem) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    r = lane & 15;
    g = lane >> 4;
    cg = wave % kColGroups;
    rg = wave / kColGroups;
    nst = a.K / 64;
    nw = a.K / kStageK;
  }

  // first weight row of column block j of this wave
  __device__ __forceinline__ int weight_row(int j) const {
    return ntile * WCOLS + (cg * HALF + j % HALF) * 16 + (j >= HALF ? a.up_row0 : 0);
  }

  __device__ __forceinline__ uint32_t lds_base() const {
    return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)lds);
  }

  __device__ __forceinline__ void issue_a(int p) {
    const uint32_t slot = lds_base() + SW * kSlotW + next_a + (uint32_t)wave * kBlockA;
#pragma unroll
    for (int j = 0; j < AMAX; ++j)
      if (j < na) {
        lds_dma16(arow[j][0] + p * 64, slot + NW * j * kBlockA);
        lds_dma16(arow[j][1] + p * 64, slot + NW * j * kBlockA + 1024);
      }
    next_a = next_a + kSlotA == SA * kSlotA ? 0 : next_a + kSlotA;
  }
  __device__ __forceinline__ void issue_w(int q) {
    BEAM_CHECK(q >= 0 && q < nw, kCheckWeightOffset);
    const uint32_t slot = lds_base() + next_w;
#pragma unroll
    for (int t = 0; t < NBL; ++t)
      lds_dma16_sv<true>(code, code_off[t], slot + (uint32_t)(cg * kCols + rg + RG * t) * kCodeB);
    // every wave of a column group loads its four blocks' scales: the same
    // bytes to the same place, so that all waves count alike
    lds_dma4_sv(scale, scale_off, slot + kBlocks * kCodeB + (uint32_t)(cg * kCols) * kScaleB);
    code += kCodeB;
    scale += kScaleB;
    next_w = next_w + kSlotW == SW * kSlotW ? 0 : next_w + kSlotW;
  }
  // loads of iteration p
  __device__ __forceinline__ void issue(int p) {
    if (p + SA >= 0 && p + SA < nst) issue_a(p + SA);
    if (p & 1) {
      const int q = ((p - 1) >> 1) + SW;
      if (q >= 0 && q < nw) issue_w(q);
    }
  }
  // Waits for A(p + 1), and so for every older load: as many of this wave's
  // loads may stay in flight as were issued after it, namely A(p + 2) .. A(p +
  // SA - 1) and the W stages of the odd iterations p + 1 - SA .. p - 1.
  __device__ __forceinline__ void wait_next(int p) {
    constexpr int kA = SA - 2, kW = (SA - 1) / 2;
    const int last_w = (p >> 1) - 1 + SW;  // of the latest odd iteration below p
    if (p + SA - 1 < nst && last_w < nw) {
      if (na == AMAX) wait_vm<2 * AMAX * kA + kLoadsW * kW>();
      else wait_vm<2 * (AMAX - 1) * kA + kLoadsW * kW>();
    } else {
      const int as = min(max(nst - 2 - p, 0), kA);
      const int ws = min(max(nw - 1 - (last_w - kW), 0), kW);
      wait_vm_dyn<0, 2 * AMAX * kA + kLoadsW * kW>(2 * na * as + kLoadsW * ws);
    }
  }

  // Takes item `tile`, `nt` and issues its first loads.
  __device__ __forceinline__ void start(int tile, int nt) {
    const int* plan_expert = a.plan + 4;
    const int* plan_row0 = plan_expert + a.max_tiles;
    const int* plan_rows = plan_row0 + a.max_tiles;
    const int e = BEAM_CLAMP(plan_expert[tile], 0, a.bounds.n_experts - 1, kCheckPlanRows);
    row0 = plan_row0[tile];
    nrows = plan_rows[tile];
    ntile = nt;
    BEAM_CHECK(nrows >= 1 && nrows <= 16 * MB && row0 >= 0 &&
                   (int64_t)row0 + nrows <= a.bounds.n_rows, kCheckPlanRows);
    const int nrb = (nrows + 15) >> 4;
    na = (nrb - wave + NW - 1) / NW;
    // Rows past the tile repeat its last.  The gather's indices are scalar
    // loads of uniform addresses, which the vector memory counter that the
    // rings are waited on with does not count.
#pragma unroll
    for (int j = 0; j < AMAX; ++j) {
      const int blk = __builtin_amdgcn_readfirstlane((wave + NW * j) * 16);
      int v[16];
      if (a.gather) {
        const __attribute__((address_space(4))) int32_t* cgather =
            (const __attribute__((address_space(4))) int32_t*)a.gather;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          v[k] = cgather[BEAM_CLAMP(row0 + min(blk + k, nrows - 1), 0, a.bounds.n_rows - 1,
                                    kCheckGatherIndex)];
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        int x = row0 + min(blk + 8 * hf + (lane >> 3), nrows - 1);
        if (a.gather) {
          x = v[8 * hf];
#pragma unroll
          for (int k = 1; k < 8; ++k) x = (lane >> 3) == k ? v[8 * hf + k] : x;
          x /= a.topk;
        }
        x = BEAM_CLAMP(x, 0, a.bounds.n_src - 1, kCheckTokenIndex);
        arow[j][hf] = a.A + (size_t)x * a.K + 8 * ((lane & 7) ^ a_chunk(hf * 8 + (lane >> 3)));
      }
    }
    const int64_t blocks = (SWIGLU ? 2 * (int64_t)a.n_out : a.n_out) / 16;
    code = a.Q + e * blocks * nw * kCodeB;
    scale = a.S + e * blocks * nw * kScaleB;
#pragma unroll
    for (int t = 0; t < NBL; ++t)
      code_off[t] = (uint32_t)BEAM_CLAMP(weight_row(rg + RG * t) >> 4, 0, blocks - 1,
                                         kCheckWeightOffset) * (uint32_t)(nw * kCodeB) +
                    (uint32_t)lane * 16u;
    // lane l loads the scales of row l % 16 of column block l / 16
    int block = 0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) block = g == j ? weight_row(j) >> 4 : block;
    scale_off = (uint32_t)block * (uint32_t)(nw * kScaleB) + (uint32_t)r * 4u;
    next_a = next_w = 0;
    constexpr int kFirst = SA > 2 * SW ? SA : 2 * SW;
#pragma unroll
    for (int p = -kFirst; p < 0; ++p) issue(p);
  }

  // One item with this wave's N row blocks from block row_off; then `next` starts
  // the following one, and the outputs are written.
  template <int N, class Next>
  __device__ __forceinline__ void item(int row_off, Next next) {
    constexpr int NX = N > 0 ? N : 1;
    f32x4_t acc[NX][kCols];
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint4 af[NX];
    uint2 cw[kCols];
    uint32_t sw[kCols];
    bf16x8_t b0[kCols], b1[kCols];
    // this lane's operand (row r, chunk g) inside a row block's 2 KB; the second
    // 32 k (chunk 4 + g) flips bit 6
    const uint8_t* abase = lds + SW * kSlotW + row_off * kBlockA;
    const int aoff = (r >> 3) * 1024 + (r & 7) * 128 + ((g ^ a_chunk(r)) << 4);
    const uint8_t* wbase = lds + cg * kCols * kCodeB + 8 * lane;
    const uint8_t* sbase = lds + kBlocks * kCodeB + cg * kCols * kScaleB + 4 * r;
    auto read_a = [&](uint32_t slot, int half, int i) {
      return *reinterpret_cast<const uint4*>(abase + slot + i * kBlockA + (aoff ^ (half << 6)));
    };
    // codes of half a W stage, and with its first half its scales
    auto read_w = [&](uint32_t slot, int half) {
      if constexpr (N > 0) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          cw[j] = *reinterpret_cast<const uint2*>(wbase + slot + j * kCodeB + half * (kCodeB / 2));
          if (half == 0) sw[j] = *reinterpret_cast<const uint32_t*>(sbase + slot + j * kScaleB);
        }
      }
    };
    // operands of step s (of the 128 k that sw covers) of column block j
    auto widen = [&](int s, int j) {
      return widen_fp4(s & 1 ? cw[j].y : cw[j].x, e8m0_value((sw[j] >> (8 * s)) & 255u));
    };
    // One MFMA step on b and af.  Row block by row block af is read again from
    // `slot`, and step s (the next one) is widened into bn, LATE row blocks after
    // its codes were read.
    auto step = [&](const bf16x8_t (&b)[kCols], bf16x8_t (&bn)[kCols], int s, uint32_t slot,
                    int half, auto late) {
      if constexpr (N > 0) {
        constexpr int LATE = decltype(late)::value < N ? decltype(late)::value : N - 1;
        int done = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int upto = i < LATE ? 0 : (i - LATE + 1) * kCols / (N - LATE);
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            acc[i][j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], as_bf16x8(af[i]), acc[i][j], 0, 0, 0);
          af[i] = read_a(slot, half, i);
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            if (j >= done && j < upto) bn[j] = widen(s, j);
          // of this row block: an MFMA, its share of the conversions, and so on
          const int n = (6 * (upto - done) + kCols - 1) / kCols;
          done = upto;
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (n <= 0) continue;
            if (n <= 2) __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
            else if (n <= 3) __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
            else __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        // computed here, not sunk to their use behind the next barrier
#pragma unroll
        for (int j = 0; j < kCols; ++j) asm volatile("" : "+v"(bn[j]));
      }
    };
    using Late0 = std::integral_constant<int, 0>;
    using Late1 = std::integral_constant<int, 1>;
    auto pass = [&](int p) {  // makes A(p + 1) (and its W stage) visible
      wait_next(p);
      wait_lgkm0();
      stage_barrier();
    };

    uint32_t as = 0, ws = 0;  // slots of A(2q) and W(q)
    pass(-1);
    if constexpr (N > 0) {
      read_w(0, 0);
#pragma unroll
      for (int i = 0; i < N; ++i) af[i] = read_a(0, 0, i);
#pragma unroll
      for (int j = 0; j < kCols; ++j) b0[j] = widen(0, j);
    }
    int q = 0;
    for (; q + 1 < nw; ++q) {  // iterations 2q and 2q + 1
      const int p = 2 * q;
      const uint32_t as1 = as + kSlotA == SA * kSlotA ? 0 : as + kSlotA;
      const uint32_t as2 = as1 + kSlotA == SA * kSlotA ? 0 : as1 + kSlotA;
      const uint32_t ws1 = ws + kSlotW == SW * kSlotW ? 0 : ws + kSlotW;
      step(b0, b1, 1, as, 1, Late0{});
      pass(p);
      read_w(ws, 1);
      issue(p);
      step(b1, b0, 2, as1, 0, Late1{});
      step(b0, b1, 3, as1, 1, Late0{});
      pass(p + 1);
      read_w(ws1, 0);
      issue(p + 1);
      step(b1, b0, 0, as2, 0, Late1{});
      as = as2;
      ws = ws1;
    }
    {  // the last W stage
      const uint32_t as1 = as + kSlotA == SA * kSlotA ? 0 : as + kSlotA;
      step(b0, b1, 1, as, 1, Late0{});
      pass(2 * q);
      read_w(ws, 1);
      step(b1, b0, 2, as1, 0, Late1{});
      step(b0, b1, 3, as1, 1, Late0{});
      if constexpr (N > 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1[j], as_bf16x8(af[i]),
                                                                acc[i][j], 0, 0, 0);
      }
    }
    wait_lgkm0();
    stage_barrier();  // every wave is done with the rings

    const int out_row0 = row0, out_rows = nrows, col0 = ntile * WCOLS + cg * HALF * 16;
    next();

    // The weights are the first operand: lane (r, g) holds output columns 4g ..
    // 4g + 3 of row r of each 16 x 16 block.  Blocks j and j + 1 trade halves
    // between lane rows, so that a lane stores 8 columns at once; a lane whose
    // row lies past the tile gets an offset outside the store's range.
    if constexpr (N > 0) {
      const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
          a.C + (size_t)out_row0 * a.n_out, 0, out_rows * a.n_out * 2, kBufferRsrcWord3);
      int er = r, eg = g;  // opaque: the offsets are formed here, not kept through the loop
      asm volatile("" : "+v"(er), "+v"(eg));
      auto outputs = [&](int i, int j) {
        float o[4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
          o[v] = SWIGLU ? silu_mul(acc[i][j][v], acc[i][j + (SWIGLU ? HALF : 0)][v]) : acc[i][j][v];
        return u32x2_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      };
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = (row_off + i) * 16 + er;
#pragma unroll
        for (int j = 0; j < HALF; j += 2) {
          const u32x2_t d0 = outputs(i, j), d1 = outputs(i, j + 1);
          const auto sx = __builtin_amdgcn_permlane16_swap(d0[0], d1[0], false, false);
          const auto sy = __builtin_amdgcn_permlane16_swap(d0[1], d1[1], false, false);
          const int col = col0 + (j + (eg & 1)) * 16 + 4 * (eg & ~1);
          const uint32_t off = row < out_rows ? (uint32_t)(row * a.n_out + col) * 2u : 0x80000000u;
          const u32x4_t d = {sx[0], sy[0], sx[1], sy[1]};
          __builtin_amdgcn_raw_buffer_store_b128(d, out, off, 0, 0);
        }
      }
    }
  }

  template <int N, class Next>
  __device__ __forceinline__ void dispatch(int n, int row_off, Next next) {
    if constexpr (N <= RB) {
      if (n == N) item<N>(row_off, next);
      else dispatch<N + 1>(n, row_off, next);
    }
  }

  __device__ __forceinline__ void run() {
    const int nt_n = a.n_out / WCOLS;
    const int total = a.plan[0] * nt_n;
    const int grid = balanced_grid(total, gridDim.x), per_xcd = grid / 8;
    if ((int)blockIdx.x >= grid) return;  // whole workgroup
    int q = (blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    if (q >= total) return;
    start(q / nt_n, q % nt_n);
    while (q < total) {
      q += grid;
      // row group 0 takes the first half of the item's row blocks, rounded up
      const int nrb = (nrows + 15) >> 4, half = RG == 1 ? nrb : (nrb + 1) / 2;
      dispatch<0>(rg == 0 ? half : nrb - half, rg == 0 ? 0 : half, [&]() {
        if (q < total) start(q / nt_n, q % nt_n);
      });
    }
  }
};

template <int MB, int RG, int SA, int SW, bool SWIGLU>
__global__ __launch_bounds__(256 * RG, 1) void gemm_fp4_kernel(Fp4Args args) {
  using G = Fp4Gemm<MB, RG, SA, SW, SWIGLU>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[G::kLds];
  G(args, lds).run();
}

template <int MB, int RG, int SA, int SW, bool SWIGLU>
static hipError_t launch_fp4(const Fp4Args& args, hipStream_t stream) {
  using G = Fp4Gemm<MB, RG, SA, SW, SWIGLU>;
  auto kern = gemm_fp4_kernel<MB, RG, SA, SW, SWIGLU>;
  static int resident = 0;  // workgroups that the device holds, fixed per build
  if (resident == 0) {
    int dev = 0, n = 0, occ = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err == hipSuccess) err = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
    if (err == hipSuccess) err = hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, 64 * G::NW, 0);
    if (err != hipSuccess) return err;
    resident = n * (occ > 0 ? occ : 1);
  }
  const int64_t grid = persistent_grid(resident, (int64_t)args.max_tiles * (args.n_out / G::WCOLS));
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * G::NW), 0, stream, args);
  return hipGetLastError();
}

// m-tile height from the mean rows per expert.
int ffn_fp4_choose_mb(int64_t rows, int E) {
  const int64_t mean = rows / (E > 0 ? E : 1);
  if (mean <= 24) return 2;
  if (mean <= 80) return 8;
  return 12;
}

hipError_t launch_grouped_gemm_fp4(int mb, bool swiglu, const uint16_t* A, const int32_t* gather,
                                   int topk, const uint8_t* Q, const uint8_t* S, uint16_t* C,
                                   const int32_t* plan, int max_tiles, int K, int n_out,
                                   int up_row0, hipStream_t stream, const GemmBounds& bounds) {
  const Fp4Args args{A, gather, topk, Q, S, C, plan, max_tiles, K, n_out, up_row0, bounds};
#define BEAM_FP4_CASE(MBV, RGV, SAV, SWV)                                \
  case MBV:                                                              \
    return swiglu ? launch_fp4<MBV, RGV, SAV, SWV, true>(args, stream)   \
                  : launch_fp4<MBV, RGV, SAV, SWV, false>(args, stream);
  switch (mb) {
    BEAM_FP4_CASE(2, 1, 3, 4)
    BEAM_FP4_CASE(8, 2, 3, 5)
    BEAM_FP4_CASE(12, 2, 3, 4)
    default:
      return hipErrorInvalidValue;
  }
#undef BEAM_FP4_CASE
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
