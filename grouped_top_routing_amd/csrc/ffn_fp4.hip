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

// The float whose exponent field is the code, which is all that the conversion
// takes of its scale: 0 stands for 2^-127 (codes .5, 1 and 1.5 of it are subnormal
// in bf16, and the MFMA keeps them) and infinity for NaN.
__device__ __forceinline__ float e8m0_value(uint32_t code) { return __uint_as_float(code << 23); }

}  // namespace

// One thread per 32 consecutive weights of a row.  Load time only: gate/up of 256
// experts of 5120 x 2560 (13.4 GB read, 3.6 written) take 5.96 ms, 2.9 TB/s, since
// codes are stored four bytes at a time, in fragment order.
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
// fragments: one thread per lane of a fragment.  Gate/up of 256 experts of 5120 x
// 2560 (3.6 GB read, 3.6 written) take 1.78 ms, 4 TB/s.
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
// times 64 CG of its weight rows (gate/up: 32 CG gate rows and the matching up
// rows), walked by a persistent grid.
//
// Waves form RG row groups x CG column groups: a wave computes 4 column blocks
// (gate/up: 2 gate blocks and their up blocks) for its share of the item's
// 16-row blocks.  Up to 96 rows RG is 1 and a CU holds two workgroups of CG 4,
// which meet at no barrier: one's MFMAs run while the other waits, issues loads or
// writes its outputs.  Taller tiles have RG 2 and a CU to themselves: they load the
// weights of more rows once, and a row block is read from LDS by four waves, not
// eight.  A few tokens' items are single waves (CG 1), so that one token's eight
// experts still fill the CUs; of up to 1024 such items KS = 2 waves take half of the k
// each, in rings of their own, and the first adds the second's sums.
//
// Codes, scales and rows are staged in LDS by direct loads, 64 k at a time in a
// ring of S slots: per column block half a code fragment (512 bytes) and the scales
// of 128 k (64 bytes), per row block 2 KB: a row's 128 bytes with their 16-byte chunks
// swizzled by (row / 2) % 8, so that the 16 rows of an operand read hit distinct
// banks.  A wave reads its codes of a stage once (8 bytes per block and lane) and
// widens them to bf16 operands in registers, one MFMA step ahead and between the
// MFMAs of the step before: an MFMA holds the matrix cores for 16 cycles and the
// issue port for 4, so that the conversions fit beside it.
//
// Schedule.  Stage p is two MFMA steps.  After the first one the wave waits for
// stage p + 1 and for its own LDS reads, passes the barrier, refills the slot of
// stage p (which every wave has read by then) with stage p + S, reads the codes of
// stage p + 1, and takes the second step while it reads that stage's rows.  A
// workgroup issues its next item's first S stages before the current item's outputs
// are written.
//
// Measured at 256 experts of 5120 x 2560, gate/up and down in us, medians: 1 token 23
// and 13 (4.8 and 4.3 TB/s of codes and scales: launch and first latencies), 32 tokens
// 349 and 181 (6.6 and 6.3 TB/s: bound by HBM; a copy of the loop that only loads takes
// 0.96 of it), 512 tokens 604 and 348 (6.0 and 5.1 TB/s, HBM), 4096 tokens 1604 and 826
// (1.07 and 1.04 PFLOP/s; MFMAs take 52 % of the cycles, load issue and LDS reads do
// not hide behind them: of 1549 in the fastest runs 1244 without the loads, 960 without
// the MFMAs, no change without the widening).
constexpr int kCols = 4;         // column blocks per wave
constexpr int kHalfB = kCodeB / 2;  // codes of a block's 64 k
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
  const int32_t* offsets;
  GemmBounds bounds;
};

// Where the items' rows are.  A plan that was built before (tile_plan_kernel) ...
struct PlanTiles {
  const int* at;
  int max_tiles;
  __device__ __forceinline__ PlanTiles(const Fp4Args& a, int) : at(a.plan), max_tiles(a.max_tiles) {}
  __device__ __forceinline__ int count() const { return at[0]; }
  __device__ __forceinline__ void get(int tile, int& e, int& row0, int& nrows) const {
    e = at[4 + tile];
    row0 = at[4 + max_tiles + tile];
    nrows = at[4 + 2 * max_tiles + tile];
  }
};
// ... or, for 16-row tiles, worked out by each single-wave workgroup: lane l holds
// experts 4l .. 4l + 3 of 256, their first rows and the number of their first tile.
// One token's call is a launch shorter by it (plan 2.3 us and its gap).
struct OwnTiles {
  int lane, first[4], row[5], total;
  __device__ __forceinline__ OwnTiles(const Fp4Args& a, int lane_) : lane(lane_) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) row[i] = a.offsets[4 * lane + i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      first[i] = n;
      n += (row[i + 1] - row[i] + 15) >> 4;
    }
    int upto = n;  // tiles of the lanes up to this one
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(upto, off);
      upto += lane >= off ? v : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) first[i] += upto - n;
    total = __builtin_amdgcn_readlane(upto, 63);
  }
  __device__ __forceinline__ int count() const { return total; }
  __device__ __forceinline__ void get(int tile, int& e, int& row0, int& nrows) const {
    e = row0 = 0;
    nrows = 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row[i] + 16 * (tile - first[i]);  // the tile's first row, if it is this expert's
      const uint64_t has = __ballot(tile >= first[i] && r < row[i + 1]);
      if (has) {
        const int l = __builtin_ctzll(has);
        e = 4 * l + i;
        row0 = __builtin_amdgcn_readlane(r, l);
        nrows = min(16, __builtin_amdgcn_readlane(row[i + 1], l) - row0);
      }
    }
  }
};

template <int MB, int RG, int CG, int S, int KS, bool SWIGLU>
struct Fp4Gemm {
  static constexpr int NW = CG * RG;
  static constexpr int kBlocks = CG * kCols;          // weight-row blocks of an item
  static constexpr int kSlotW = kBlocks * (kHalfB + kScaleB);
  static constexpr int AMAX = (MB + NW - 1) / NW;     // row blocks a wave loads
  static constexpr int RB = (MB + RG - 1) / RG;       // row blocks a wave computes, at most
  static constexpr int kLoadsW = kCols / 2 / RG + 1;  // a wave's code and scale loads of a stage
  static constexpr int HALF = SWIGLU ? kCols / 2 : kCols;
  static constexpr int WCOLS = CG * HALF * 16;
  static constexpr int kSlot = kSlotW + MB * kBlockA;
  static constexpr int kLds = S * kSlot;
  static_assert(S >= 3 && (S - 1) * (2 * AMAX + kLoadsW) < 64, "vmcnt holds 6 bits");
  static_assert(KS == 1 || (NW == 1 && MB == 1 && kCols * 1024 <= kLds), "a wave's sums fit its ring");
  static_assert((RG == 1 || RG == 2) && kLds <= NW * 20 * 1024, "eight waves per CU");

  using Tiles = std::conditional_t<NW == 1 && MB == 1, OwnTiles, PlanTiles>;

  const Fp4Args& a;
  uint8_t* lds;
  Tiles tiles;
  int lane, wave, r, g, cg, rg;
  int kw;                         // of KS waves that share an item's k
  int k0, nst;                    // first stage and stages of an item (even)
  // the item whose loads are in flight
  int row0, nrows, ntile, na;
  const uint16_t* arow[AMAX][2];  // this lane's 16 bytes of stage 0 of the rows it loads
  const uint8_t* code;            // the expert's codes, at the next stage to load
  const uint8_t* scale;           // its scales
  uint32_t code_off[kCols / 2 / RG], scale_off;
  uint32_t next;                  // its slot (bytes into the ring)

  __device__ __forceinline__ Fp4Gemm(const Fp4Args& args, uint8_t* mem)
      : a(args), lds(mem), tiles(args, threadIdx.x & 63) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    k0 = kw = 0;
    nst = a.K / 64;
    if constexpr (KS > 1) {  // whole fragments of 128 k; a wave may have none
      kw = wave;
      wave = 0;
      lds += kw * kLds;
      const int frags = a.K / kStageK;
      k0 = kw * frags / KS * 2;
      nst = (kw + 1) * frags / KS * 2 - k0;
    }
    r = lane & 15;
    g = lane >> 4;
    cg = wave % CG;
    rg = wave / CG;
  }

  // first weight row of column block j of this wave
  __device__ __forceinline__ int weight_row(int j) const {
    return ntile * WCOLS + (cg * HALF + j % HALF) * 16 + (j >= HALF ? a.up_row0 : 0);
  }

  // Loads of stage p, the next one.
  __device__ __forceinline__ void issue(int p) {
    BEAM_CHECK(p >= 0 && p < nst, kCheckWeightOffset);
    const uint32_t slot =
        (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)lds) + next;
#pragma unroll
    for (int t = 0; t < kCols / 2 / RG; ++t)  // a pair of column blocks, 32 lanes each
      lds_dma16_sv<true>(code, code_off[t],
                         slot + (uint32_t)(cg * kCols + 2 * (rg + RG * t)) * kHalfB);
    // (RG 2: both waves of a column group load its four blocks' scales, the same
    // bytes to the same place, so that all waves count alike)
    lds_dma4_sv(scale, scale_off, slot + kBlocks * kHalfB + (uint32_t)(cg * kCols) * kScaleB);
#pragma unroll
    for (int j = 0; j < AMAX; ++j)
      if (j < na) {
        const uint32_t to = slot + kSlotW + (uint32_t)(wave + NW * j) * kBlockA;
        lds_dma16(arow[j][0] + p * 64, to);
        lds_dma16(arow[j][1] + p * 64, to + 1024);
      }
    code += kHalfB;
    scale += p & 1 ? kScaleB : 0;
    next = next + kSlot == kLds ? 0 : next + kSlot;
  }

  // Waits until at most `stages` stages of this wave's loads are in flight.
  template <int STAGES, int NA = AMAX>
  __device__ __forceinline__ void wait_stages() {
    if constexpr (NA == 0) {
      wait_vm<STAGES * kLoadsW>();
    } else {
      if (na == NA) wait_vm<STAGES*(2 * NA + kLoadsW)>();
      else wait_stages<STAGES, NA - 1>();
    }
  }
  template <int STAGES>
  __device__ __forceinline__ void wait_stages_dyn(int stages) {
    if constexpr (STAGES == 0) {
      wait_vm<0>();
    } else {
      if (stages >= STAGES) wait_stages<STAGES>();
      else wait_stages_dyn<STAGES - 1>(stages);
    }
  }

  // Takes item `tile`, `nt` and issues its first stages.
  __device__ __forceinline__ void start(int tile, int nt) {
    int e;
    tiles.get(tile, e, row0, nrows);
    e = BEAM_CLAMP(e, 0, a.bounds.n_experts - 1, kCheckPlanRows);
    ntile = nt;
    BEAM_CHECK(nrows >= 1 && nrows <= 16 * MB && row0 >= 0 &&
                   (int64_t)row0 + nrows <= a.bounds.n_rows, kCheckPlanRows);
    const int nrb = (nrows + 15) >> 4;
    na = (nrb - wave + NW - 1) / NW;
    // Rows past the tile repeat its last.  The gather's indices are scalar
    // loads of uniform addresses, which the vector memory counter that the
    // ring is waited on with does not count.
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
        arow[j][hf] = a.A + (size_t)x * a.K + k0 * 64 + 8 * ((lane & 7) ^ a_chunk(hf * 8 + (lane >> 3)));
      }
    }
    const int64_t blocks = (SWIGLU ? 2 * (int64_t)a.n_out : a.n_out) / 16;
    const int nfrag = a.K / kStageK;
    code = a.Q + e * blocks * nfrag * kCodeB + k0 * kHalfB;
    scale = a.S + e * blocks * nfrag * kScaleB + k0 / 2 * kScaleB;
#pragma unroll
    for (int t = 0; t < kCols / 2 / RG; ++t)
      code_off[t] = (uint32_t)BEAM_CLAMP(weight_row(2 * (rg + RG * t) + (lane >> 5)) >> 4, 0,
                                         blocks - 1, kCheckWeightOffset) *
                        (uint32_t)(nfrag * kCodeB) +
                    (uint32_t)(lane & 31) * 16u;
    // lane l loads the scales of row l % 16 of column block l / 16
    int block = 0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) block = g == j ? weight_row(j) >> 4 : block;
    scale_off = (uint32_t)block * (uint32_t)(nfrag * kScaleB) + (uint32_t)r * 4u;
    next = 0;
#pragma unroll
    for (int p = 0; p < S; ++p)
      if (p < nst) issue(p);
  }

  // One item with this wave's N row blocks from block row_off; then `then` starts
  // the following one, and the outputs are written.
  template <int N, class Then>
  __device__ __forceinline__ void item(int row_off, Then then) {
    constexpr int NX = N > 0 ? N : 1;
    f32x4_t acc[NX][kCols];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    uint4 af[NX];
    uint2 cw[kCols];
    uint32_t sw[kCols];
    bf16x8_t b0[kCols], b1[kCols];
    // this lane's operand (row r, chunk g) inside a row block's 2 KB; the second
    // 32 k (chunk 4 + g) flips bit 6
    const uint8_t* abase = lds + kSlotW + row_off * kBlockA;
    const int aoff = (r >> 3) * 1024 + (r & 7) * 128 + ((g ^ a_chunk(r)) << 4);
    const uint8_t* wbase = lds + cg * kCols * kHalfB + 8 * lane;
    const uint8_t* sbase = lds + kBlocks * kHalfB + cg * kCols * kScaleB + 4 * r;
    auto read_a = [&](uint32_t slot, int half, int i) {
      return *reinterpret_cast<const uint4*>(abase + slot + i * kBlockA + (aoff ^ (half << 6)));
    };
    // a stage's codes, and in even stages the scales of two
    auto read_w = [&](uint32_t slot, bool scales) {
      if constexpr (N == 0) return;
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        cw[j] = *reinterpret_cast<const uint2*>(wbase + slot + j * kHalfB);
        if (scales) sw[j] = *reinterpret_cast<const uint32_t*>(sbase + slot + j * kScaleB);
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
      if constexpr (N == 0) return;
      constexpr int LATE = decltype(late)::value < NX ? decltype(late)::value : NX - 1;
      int done = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int upto = i < LATE ? 0 : (i - LATE + 1) * kCols / (NX - LATE);
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
    };
    using Late0 = std::integral_constant<int, 0>;
    using Late1 = std::integral_constant<int, 1>;
    auto pass = [&]() {  // this wave's reads have landed; every wave's loads are visible
      wait_lgkm0();
      if constexpr (KS == 1) stage_barrier();
      else compiler_fence();  // a ring of the wave's own
    };
    auto after = [](uint32_t slot) { return slot + kSlot == kLds ? 0u : slot + kSlot; };

    if (KS == 1 || nst > 0) {
      uint32_t at = 0;  // slot of the current stage
      wait_stages_dyn<S - 1>(nst - 1);
      pass();
      read_w(0, true);
#pragma unroll
      for (int i = 0; i < N; ++i) af[i] = read_a(0, 0, i);
      if constexpr (N > 0) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) b0[j] = widen(0, j);
      }
      // stages p and p + 1 (p even); ALL: with stages p + S and p + 1 + S to come
      int p = 0;
      auto turn = [&](auto all) {
        constexpr bool ALL = decltype(all)::value;
        const uint32_t at1 = after(at), at2 = after(at1);
        step(b0, b1, 1, at, 1, Late0{});
        if constexpr (ALL) wait_stages<S - 2>();
        else wait_stages_dyn<S - 2>(nst - 2 - p);
        pass();
        read_w(at1, false);
        if (ALL || p + S < nst) issue(p + S);
        step(b1, b0, 2, at1, 0, Late1{});
        step(b0, b1, 3, at1, 1, Late0{});
        if constexpr (ALL) wait_stages<S - 2>();
        else wait_stages_dyn<S - 2>(nst - 3 - p);
        pass();
        read_w(at2, true);
        if (ALL || p + 1 + S < nst) issue(p + 1 + S);
        step(b1, b0, 0, at2, 0, Late1{});
        at = at2;
        p += 2;
      };
      for (; p + 1 + S < nst; ) turn(std::true_type{});
      for (; p + 2 < nst; ) turn(std::false_type{});
      {  // the last two stages
        const uint32_t at1 = after(at);
        step(b0, b1, 1, at, 1, Late0{});
        wait_vm<0>();
        pass();
        read_w(at1, false);
        step(b1, b0, 2, at1, 0, Late1{});
        step(b0, b1, 3, at1, 1, Late0{});
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            acc[i][j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1[j], as_bf16x8(af[i]), acc[i][j], 0, 0, 0);
      }
    }
    pass();  // every wave is done with the ring
    if constexpr (KS > 1 && N > 0) {  // the waves' sums, added in their order
      f32x4_t* sums = reinterpret_cast<f32x4_t*>(lds);
      if (kw > 0)
#pragma unroll
        for (int j = 0; j < kCols; ++j) sums[j * 64 + lane] = acc[0][j];
      __syncthreads();
      if (kw == 0)
#pragma unroll
        for (int w = 1; w < KS; ++w)
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            acc[0][j] += reinterpret_cast<const f32x4_t*>(lds + w * kLds)[j * 64 + lane];
      __syncthreads();  // read before the next item's loads
    }

    const int out_row0 = row0, out_rows = nrows, col0 = ntile * WCOLS + cg * HALF * 16;
    then();

    // The weights are the first operand: lane (r, g) holds output columns 4g ..
    // 4g + 3 of row r of each 16 x 16 block.  Blocks j and j + 1 trade halves
    // between lane rows, so that a lane stores 8 columns at once; a lane whose
    // row lies past the tile gets an offset outside the store's range.
    if constexpr (N == 0) return;
    if (kw > 0) return;
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

  template <int N, class Then>
  __device__ __forceinline__ void dispatch(int n, int row_off, Then then) {
    if constexpr (N <= RB) {
      if (n == N) item<N>(row_off, then);
      else dispatch<N + 1>(n, row_off, then);
    }
  }

  __device__ __forceinline__ void run() {
    const int nt_n = a.n_out / WCOLS;
    const int total = tiles.count() * nt_n;
    const int grid = balanced_grid(total, gridDim.x), per_xcd = grid / 8;
    if ((int)blockIdx.x >= grid) return;  // whole workgroup
    int q = (blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    if (q >= total) return;
    start(q / nt_n, q % nt_n);
    while (q < total) {
      q += grid;
      // row group 0 takes the first half of the item's row blocks, rounded up
      const int nrb = (nrows + 15) >> 4, half = RG == 1 ? nrb : (nrb + 1) / 2;
      dispatch<RG == 1 ? 1 : 0>(rg == 0 ? half : nrb - half, rg == 0 ? 0 : half, [&]() {
        if (q < total) start(q / nt_n, q % nt_n);
      });
    }
  }
};

template <int MB, int RG, int CG, int S, int KS, bool SWIGLU>
__global__ __launch_bounds__(64 * CG * RG * KS, 2) void gemm_fp4_kernel(Fp4Args args) {
  using G = Fp4Gemm<MB, RG, CG, S, KS, SWIGLU>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KS * G::kLds];
  G(args, lds).run();
}

template <int MB, int RG, int CG, int S, int KS, bool SWIGLU>
static hipError_t launch_fp4(const Fp4Args& args, hipStream_t stream) {
  using G = Fp4Gemm<MB, RG, CG, S, KS, SWIGLU>;
  auto kern = gemm_fp4_kernel<MB, RG, CG, S, KS, SWIGLU>;
  static int resident = 0;  // workgroups that the device holds, fixed per build
  if (resident == 0) {
    int dev = 0, n = 0, occ = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err == hipSuccess) err = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
    if (err == hipSuccess) err = hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, 64 * G::NW * KS, 0);
    if (err != hipSuccess) return err;
    resident = n * (occ > 0 ? occ : 1);
  }
  const int64_t grid = persistent_grid(resident, (int64_t)args.max_tiles * (args.n_out / G::WCOLS));
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * G::NW * KS), 0, stream, args);
  return hipGetLastError();
}

// m-tile height from the mean rows per expert.  Times of an MLP call at the Beam
// shape (hidden 5120, intermediate 2560) in us, tiles of 16 / 64 / 96 / 192 rows:
// 1 token 39 / 56, 5 tokens 137 / 154, 10 tokens 250 / 240, 32 tokens 584 / 581 /
// 640 / 737, 512 tokens 1333 / 1004 / 1053 / 1201, 1400 tokens - / 1237 / 1284 /
// 1521, 2000 tokens - / 1774 / 1471 / 1711, 3200 tokens - / 2449 / 2387 / 2069.
// Where the experts in use are small (`weights`: hidden * intermediate of each), the
// launch that 16-row tiles save counts with more rows too, tiles of 16 / 64: 1024 x
// 512 at 160 rows 25.0 / 27.8, 800 rows 42.9 / 47.5, 2048 rows 52.0 / 49.5; 768 x
// 384 at 1015 rows 30.1 / 36.2; 2048 x 1024 at 80 rows 52 / 65, 480 rows 139.5 /
// 139.5, 1600 rows 164 / 154.
int ffn_fp4_choose_mb(int64_t rows, int E, int64_t weights) {
  const int64_t mean = rows / (E > 0 ? E : 1);
  if (rows <= E / 4) return 1;
  if (rows <= 4 * E && (rows < E ? rows : E) * weights <= (int64_t)1 << 28) return 1;
  if (mean <= 50) return 4;
  if (mean <= 80) return 6;
  return 12;
}

bool ffn_fp4_planned(int mb) { return mb != 1; }

hipError_t launch_grouped_gemm_fp4(int mb, bool swiglu, const uint16_t* A, const int32_t* gather,
                                   int topk, const uint8_t* Q, const uint8_t* S, uint16_t* C,
                                   const int32_t* offsets, const int32_t* plan, int max_tiles,
                                   int K, int n_out, int up_row0, hipStream_t stream,
                                   const GemmBounds& bounds) {
  const Fp4Args args{A, gather, topk, Q, S, C, plan, max_tiles, K, n_out, up_row0, offsets, bounds};
#define BEAM_FP4_CASE(MBV, RGV, CGV, SV, KSV)                                 \
  case MBV:                                                                   \
    return swiglu ? launch_fp4<MBV, RGV, CGV, SV, KSV, true>(args, stream)    \
                  : launch_fp4<MBV, RGV, CGV, SV, KSV, false>(args, stream);
  // A token's few items: two waves share each one's k.  In us, one wave / two: 1 token
  // of 5120 x 2560 (720 items) 42.5 / 38.7, 4 of 1024 x 512 15.8 / 15.2, but 2 of 5120
  // x 2560 (1360 items, the CUs hold 1024 pairs) 66.8 / 70.9, 100 of 1024 x 512 42.8 /
  // 49.0; four waves 38.6, 13.7, 73.7, 55.5.  The order of a row's sums, and so its last
  // bits, go by this choice, that is by the pairs of the whole call.
  if (mb == 1 && (int64_t)max_tiles * (n_out / (swiglu ? 32 : 64)) <= 1024)
    return swiglu ? launch_fp4<1, 1, 1, 4, 2, true>(args, stream)
                  : launch_fp4<1, 1, 1, 4, 2, false>(args, stream);
  switch (mb) {
    BEAM_FP4_CASE(1, 1, 1, 4, 1)
    BEAM_FP4_CASE(4, 1, 4, 4, 1)
    BEAM_FP4_CASE(6, 1, 4, 3, 1)
    BEAM_FP4_CASE(12, 2, 4, 4, 1)
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
