/*
 * beam_moe.h -- C ABI of the Beam-1.0 mixture-of-experts block on one
 * AMD Instinct MI355X (gfx950).
 *
 * The block ("Welcome Beam: a 501B open model you can own, customize, and
 * scale", section "Mixture of Experts"; "Beam 1.0" miles recipes, section 1
 * "Model Introduction"):
 *   1. router GEMM in FP32 (router weights are kept in FP32; the same page's
 *      section "Residual Stream" lists the router among the FP32 computations),
 *   2. sigmoid score for every expert,
 *   3. experts split into num_groups contiguous groups; each group scored by the
 *      sum of its two best scores; the topk_groups best groups are kept,
 *   4. the topk best experts inside the kept groups are chosen,
 *   5. each chosen expert is a SwiGLU MLP (gate/up projection, SiLU(gate)*up
 *      in FP32, down projection), with no shared expert,
 *   6. the token's output is the sum of its experts' outputs, each weighted by
 *      its score over the sum of the chosen scores, times routed_scaling (2.5).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates or frees device memory; scratch space comes from the
 *     caller's workspace (size from moe_workspace_bytes).
 *   - bf16 tensors are passed as uint16_t bit patterns.  All tensors are dense
 *     row-major with the layouts stated per argument.  Tensor pointers and the
 *     workspace must be 16-byte aligned.
 *   - Every call validates its arguments on the host first.  On any error it
 *     enqueues nothing and returns a negative status; MOE_OK (0) otherwise.
 *     num_tokens == 0 is a valid no-op.  A failed kernel launch returns
 *     MOE_ERR_HIP.  Faults inside kernels surface at the caller's next
 *     synchronisation of `stream`.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = default stream) and
 *     the call never synchronises it.  Calls that share a workspace must be
 *     ordered on one stream.
 *   - Results are bitwise deterministic: no floating-point atomics.  They do
 *     not depend on the number of workgroups of the persistent expert GEMMs
 *     either; the environment variable BEAM_MOE_MAX_GRID=<n>, read at each
 *     launch, caps that number (for testing this).
 *   - Supported shapes: num_experts == 256; num_groups a power of two in
 *     [1, 64]; 1 <= topk_groups <= num_groups; 1 <= topk <= 8 and topk not
 *     above the experts in the kept groups; hidden a multiple of 256;
 *     intermediate a multiple of 128; num_tokens * topk < 2^31.  Other shapes return
 *     MOE_ERR_UNSUPPORTED.
 */
#ifndef BEAM_MOE_H
#define BEAM_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,  /* null pointer, negative size, misalignment     */
  MOE_ERR_UNSUPPORTED = -2,  /* valid but outside the shapes listed above     */
  MOE_ERR_WORKSPACE = -3,    /* workspace missing or smaller than required    */
  MOE_ERR_HIP = -4,          /* HIP runtime error (no device, launch failure) */
  MOE_ERR_TOO_LARGE = -5     /* moe_layer_forward_noalloc: the call needs more
                                scratch than the library's static array holds */
};

/* Which entry point a workspace size is asked for. */
enum moe_entry {
  MOE_ENTRY_ROUTE = 0,
  MOE_ENTRY_PERMUTE = 1,
  MOE_ENTRY_EXPERT_FFN = 2,
  MOE_ENTRY_LAYER = 3,
  MOE_ENTRY_EXPERT_STAGE = 4,  /* moe_expert_gate_up or moe_expert_down */
  MOE_ENTRY_EXPERT_FFN_LORA = 5,
  MOE_ENTRY_LAYER_LORA = 6,
  MOE_ENTRY_ROUTE_BACKWARD = 8  /* 7 names no entry */
};

typedef struct moe_config {
  int64_t num_tokens;     /* T >= 0 tokens in this call                           */
  int32_t hidden;         /* H: 5120 for Beam-1.0                                 */
  int32_t intermediate;   /* I: SwiGLU intermediate size, 2560 for Beam-1.0       */
  int32_t num_experts;    /* E = 256                                              */
  int32_t num_groups;     /* G = 8 groups of E/G contiguous experts               */
  int32_t topk_groups;    /* groups kept per token, 4                             */
  int32_t topk;           /* experts per token, 8                                 */
  int32_t renormalize;    /* 1: combine weight = score / sum of the topk chosen
                             scores (weights that sum to one); 0: raw score       */
  float routed_scaling;   /* factor applied to the combined output, 2.5          */
  int32_t weight_layout;  /* expert weight storage: MOE_LAYOUT_ROW_MAJOR or
                             MOE_LAYOUT_PACKED (written by moe_pack_weights) for
                             the bf16 expert calls, MOE_LAYOUT_FP8_PACKED for the
                             *_fp8 calls, MOE_LAYOUT_FP4_PACKED for the *_fp4
                             calls; calls that read no expert weights accept any */
} moe_config_t;

/* Expert weight layouts. */
enum moe_weight_layout {
  MOE_LAYOUT_ROW_MAJOR = 0,  /* w_gate_up [E, 2I, H], w_down [E, H, I], row-major    */
  MOE_LAYOUT_PACKED = 1,     /* same sizes, each expert's [N, K] matrix stored as
                                [N/16][K/32][64][8]: the 16 x 32 bf16 operand tiles of
                                the gfx950 matrix cores, lane-ordered, consecutive
                                along K (see moe_pack_weights)                        */
  MOE_LAYOUT_FP8_PACKED = 2, /* E4M3FN codes plus fp32 per-row scales (see
                                moe_quantize_fp8)                                     */
  MOE_LAYOUT_FP4_PACKED = 4  /* E2M1 codes plus E8M0 scales per 32 weights (see
                                moe_quantize_fp4); 3 names no layout                  */
};

/* Bytes of workspace `entry` needs for `cfg` (written to *bytes). */
int moe_workspace_bytes(const moe_config_t* cfg, int entry, size_t* bytes);

/*
 * Router: logits = x . W_r^T in FP32 (bf16 inputs widened exactly), scores =
 * sigmoid(logits), group-limited top-k selection, combine weights.
 *   x         [T, H] bf16
 *   w_router  [E, H] fp32, one row per expert
 *   sel_bias  [E] fp32 or NULL: added to the scores for choosing only (the
 *             checkpoint's FP32 "expert biases" read as a selection bias); the
 *             combine weights always use the unbiased scores
 *   topk_ids  [T, topk] int32 out, ordered by (selection value desc, id asc)
 *   topk_w    [T, topk] fp32 out, combine weights WITHOUT routed_scaling
 * Ties between equal values go to the lower group / expert index.
 */
int moe_route(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
              const float* sel_bias, int32_t* topk_ids, float* topk_w,
              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Routing replay: recompute scores and combine weights for caller-supplied
 * expert ids (e.g. recorded at rollout time), skipping selection.
 *   topk_ids  [T, topk] int32 in; an id outside [0, E) names no expert and is
 *             dropped, as moe_permute drops it: its weight is 0 and it is left
 *             out of the normalising sum (a token with no valid id gets all
 *             weights 0)
 *   topk_w    [T, topk] fp32 out
 * Replayed ids then go through moe_permute, the expert calls and moe_combine,
 * where a dropped slot contributes nothing.
 */
int moe_route_replay(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                     const int32_t* topk_ids, float* topk_w,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Token permutation and per-expert histogram (stable counting sort of the
 * T*topk (token, slot) pairs by expert).
 *   topk_ids  [T, topk] int32 in; ids outside [0, E) are dropped (their
 *             perm_dst entry is -1 and they are not counted)
 *   counts    [E] int32 out: pairs routed to each expert
 *   offsets   [E + 1] int32 out: exclusive prefix sum of counts
 *   perm_src  [T*topk] int32 out: row r of the expert-major order holds pair
 *             perm_src[r] = t*topk + j; rows of one expert ascend in t
 *   perm_dst  [T*topk] int32 out: inverse, perm_dst[t*topk + j] = r
 */
int moe_permute(const moe_config_t* cfg, const int32_t* topk_ids, int32_t* counts,
                int32_t* offsets, int32_t* perm_src, int32_t* perm_dst,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Expert SwiGLU MLPs over the permuted rows (bf16 grouped GEMMs with FP32
 * accumulation; SiLU(gate)*up in FP32, rounded to bf16 before the down GEMM).
 *   x          [T, H] bf16; row r reads token perm_src[r] / topk
 *   perm_src   [T*topk] int32, offsets [E + 1] int32 (from moe_permute)
 *   w_gate_up  [E, 2*I, H] bf16: rows [0, I) gate, rows [I, 2I) up
 *   w_down     [E, H, I] bf16
 *   (both in cfg->weight_layout)
 *   y_perm     [T*topk, H] bf16 out, expert-major row order
 * Experts with no rows read no weights.
 */
int moe_expert_ffn(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                   const int32_t* offsets, const uint16_t* w_gate_up, const uint16_t* w_down,
                   uint16_t* y_perm, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The two halves of moe_expert_ffn, for callers that time or schedule them
 * separately (same kernels, same results).
 *   moe_expert_gate_up: h [T*topk, I] bf16 out = bf16(SiLU(x_r . Wg^T) * (x_r . Wu^T))
 *   moe_expert_down:    y_perm [T*topk, H] bf16 out = bf16(h_r . Wd^T)
 * Each builds its own m-tile plan from `offsets` in its workspace
 * (moe_workspace_bytes with MOE_ENTRY_EXPERT_STAGE).
 */
int moe_expert_gate_up(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                       const int32_t* offsets, const uint16_t* w_gate_up, uint16_t* h,
                       void* workspace, size_t workspace_bytes, void* stream);
int moe_expert_down(const moe_config_t* cfg, const uint16_t* h, const int32_t* offsets,
                    const uint16_t* w_down, uint16_t* y_perm,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Weighted un-permute: out[t] = bf16(routed_scaling * sum_j topk_w[t, j] *
 * y_perm[perm_dst[t*topk + j]]), summed in FP32 in slot order.  Slots with
 * perm_dst < 0 contribute nothing.
 *   out  [T, H] bf16 out
 */
int moe_combine(const moe_config_t* cfg, const uint16_t* y_perm, const int32_t* perm_dst,
                const float* topk_w, uint16_t* out, void* stream);

/*
 * The whole block: route, permute, expert MLPs, combine.
 *   out           [T, H] bf16 out
 *   topk_ids_out  [T, topk] int32 out or NULL
 *   topk_w_out    [T, topk] fp32 out or NULL
 */
int moe_layer_forward(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                      const float* sel_bias, const uint16_t* w_gate_up, const uint16_t* w_down,
                      uint16_t* out, int32_t* topk_ids_out, float* topk_w_out,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_layer_forward for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same kernels and results, with no workspace argument.  The
 * scratch comes from a static device array of 128 MiB inside the library, one
 * per GPU it runs on, held until the process ends; the call allocates nothing.
 *   - It serves configurations whose moe_workspace_bytes(MOE_ENTRY_LAYER) is at
 *     most 128 MiB (at the Beam shape, hidden 5120 and intermediate 2560:
 *     batches of up to 1,090 tokens); larger ones return MOE_ERR_TOO_LARGE
 *     and enqueue nothing.
 *   - It uses the array of the current device; `stream` must belong to it.
 *   - Every call on one GPU shares that GPU's array and leaves its contents
 *     behind: calls that overlap on one GPU (on different streams, or from
 *     several threads without ordering) race.  Order them on one stream.
 * Other arguments are those of moe_layer_forward.
 */
int moe_layer_forward_noalloc(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                              const float* sel_bias, const uint16_t* w_gate_up,
                              const uint16_t* w_down, uint16_t* out, int32_t* topk_ids_out,
                              float* topk_w_out, void* stream);

/*
 * Rewrites expert weights from MOE_LAYOUT_ROW_MAJOR into MOE_LAYOUT_PACKED
 * (a pure permutation of each expert's elements; run once at load time).
 *   w_gate_up, w_down            row-major inputs (shapes as above)
 *   packed_gate_up, packed_down  outputs of the same sizes; must not overlap
 *                                the inputs
 * Either pair may be NULL to skip it.  num_tokens and weight_layout are
 * ignored.
 */
int moe_pack_weights(const moe_config_t* cfg, const uint16_t* w_gate_up, const uint16_t* w_down,
                     uint16_t* packed_gate_up, uint16_t* packed_down, void* stream);

/*
 * FP8 per-channel expert weights (vLLM recipe JSON "Beam-1.0-501B-A23B",
 * precision variant fp8: FP8 per-channel weights, router unquantized).
 *
 * Each expert matrix row n (output channel) has one fp32 scale s[n] and
 * E4M3FN codes q[n, k] (OCP FP8: 1 sign, 4 exponent bits with bias 7, 3
 * mantissa bits, largest finite value 448); the matrix the GEMMs use is
 * w[n, k] = s[n] * q[n, k].  Activations stay bf16, accumulation fp32, and
 * the scale multiplies the fp32 accumulator of its output column.  The
 * router, selection, permutation and combine are the bf16 path's.
 *
 * Code layout (MOE_LAYOUT_FP8_PACKED): each expert's [N, K] code matrix is
 * stored as [N/16][K/64][2][64][8] bytes; entry (b, s, h, l) holds the codes
 * of row 16b + l%16 at k = 64s + 32h + 8(l/16) .. +7.  Scales are plain
 * fp32 [E, N].
 *   q_gate_up [E, 2*I, H] codes, s_gate_up [E, 2*I]
 *   q_down    [E, H, I]   codes, s_down    [E, H]
 * The *_fp8 calls require cfg->weight_layout == MOE_LAYOUT_FP8_PACKED (else
 * MOE_ERR_INVALID_ARG).  Their workspace sizes are the ones moe_workspace_bytes
 * gives for MOE_ENTRY_EXPERT_FFN, MOE_ENTRY_EXPERT_STAGE and MOE_ENTRY_LAYER.
 */
/*
 * Quantise row-major bf16 expert weights: s[n] = fp32(max_k |w[n, k]|) / 448
 * in fp32 (1 for an all-zero row); q[n, k] = E4M3FN(clamp(w[n, k] / s[n],
 * -448, 448)) with fp32 division and round-to-nearest-even (ties to the even
 * code); codes are written in MOE_LAYOUT_FP8_PACKED.
 *   w_gate_up, w_down  row-major bf16 inputs [E, 2I, H], [E, H, I]
 *   q_*, s_*           outputs as above; must not overlap the inputs
 * Either set (w, q, s) may be all NULL to skip it.  num_tokens and
 * weight_layout are ignored.
 */
int moe_quantize_fp8(const moe_config_t* cfg, const uint16_t* w_gate_up, const uint16_t* w_down,
                     uint8_t* q_gate_up, float* s_gate_up, uint8_t* q_down, float* s_down,
                     void* stream);

/* moe_expert_ffn, moe_expert_gate_up, moe_expert_down and moe_layer_forward
 * with FP8 expert weights (arguments as in those calls). */
int moe_expert_ffn_fp8(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                       const int32_t* offsets, const uint8_t* q_gate_up, const float* s_gate_up,
                       const uint8_t* q_down, const float* s_down, uint16_t* y_perm,
                       void* workspace, size_t workspace_bytes, void* stream);
int moe_expert_gate_up_fp8(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                           const int32_t* offsets, const uint8_t* q_gate_up,
                           const float* s_gate_up, uint16_t* h,
                           void* workspace, size_t workspace_bytes, void* stream);
int moe_expert_down_fp8(const moe_config_t* cfg, const uint16_t* h, const int32_t* offsets,
                        const uint8_t* q_down, const float* s_down, uint16_t* y_perm,
                        void* workspace, size_t workspace_bytes, void* stream);
int moe_layer_forward_fp8(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                          const float* sel_bias, const uint8_t* q_gate_up, const float* s_gate_up,
                          const uint8_t* q_down, const float* s_down, uint16_t* out,
                          int32_t* topk_ids_out, float* topk_w_out,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * 4-bit expert weights with group scales (E2M1 codes with one E8M0 scale per 32
 * weights, the microscaling format MXFP4): 4.25 bits per weight.
 *
 * Each expert matrix row n (output channel) has E2M1 codes q[n, k] (1 sign, 2
 * exponent, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one E8M0 scale s[n,
 * k / 32]; the matrix the GEMMs use is w[n, k] = 2^(s - 127) * q[n, k], exact
 * in bf16 for every s but 255, subnormal values (s of 0 and 1) included; s = 255
 * is NaN with every code, and a value past the largest bf16 (s of 253 and 254) is
 * infinite.
 * Activations stay bf16, accumulation fp32.  The router, selection, permutation
 * and combine are the bf16 path's.
 *
 * Row-major form (moe_pack_fp4's input): codes [E, N, K / 2], two per byte, the
 * lower k in the low half; scales [E, N, K / 32].
 * Packed form (MOE_LAYOUT_FP4_PACKED), the same sizes: each expert's codes as
 * [N/16][K/128][2][64][2][4 bytes], entry (b, t, h, l, s) holding the codes of
 * row 16b + l%16 at k = 128t + 64h + 32s + 8(l/16) .. +7, lower k in lower bits; its
 * scales as [N/16][K/128][16][4 bytes], entry (b, t, r, s) that of row 16b + r
 * at k = 128t + 32s.
 *   q_gate_up [E, 2*I, H / 2] bytes, s_gate_up [E, 2*I, H / 32]
 *   q_down    [E, H, I / 2]   bytes, s_down    [E, H, I / 32]
 * Codes and scales are 16-byte aligned.  The *_fp4 calls require
 * cfg->weight_layout == MOE_LAYOUT_FP4_PACKED (else MOE_ERR_INVALID_ARG); their
 * workspace sizes are the ones moe_workspace_bytes gives for that layout and
 * MOE_ENTRY_EXPERT_FFN, MOE_ENTRY_EXPERT_STAGE and MOE_ENTRY_LAYER.  hidden *
 * intermediate is below 2^32, each of them at most 2^22 (else
 * MOE_ERR_UNSUPPORTED).
 */
/*
 * Quantise row-major bf16 expert weights into the packed form.  The scale of a
 * group is the least power of two, at least 2^-126, by which its largest
 * magnitude is at most 7 (so that no weight is off by more than half a step);
 * codes are to the nearest, ties to the even code, magnitudes above 6 to 6.  A
 * group with an infinity or a NaN gets the scale NaN; a weight past 7 * 2^125
 * (2.98e38) rounds to 4 * 2^126, which bf16 holds as infinity.
 *   w_gate_up, w_down  row-major bf16 inputs [E, 2I, H], [E, H, I]
 *   q_*, s_*           outputs as above; must not overlap the inputs or each other
 * Either set (w, q, s) may be all NULL to skip it.  num_tokens and
 * weight_layout are ignored.
 */
int moe_quantize_fp4(const moe_config_t* cfg, const uint16_t* w_gate_up, const uint16_t* w_down,
                     uint8_t* q_gate_up, uint8_t* s_gate_up, uint8_t* q_down, uint8_t* s_down,
                     void* stream);
/* The packed form of row-major codes c_* and scales r_* (arguments otherwise as
 * in moe_quantize_fp4). */
int moe_pack_fp4(const moe_config_t* cfg, const uint8_t* c_gate_up, const uint8_t* r_gate_up,
                 const uint8_t* c_down, const uint8_t* r_down, uint8_t* q_gate_up,
                 uint8_t* s_gate_up, uint8_t* q_down, uint8_t* s_down, void* stream);

/* moe_expert_ffn, moe_expert_gate_up, moe_expert_down and moe_layer_forward
 * with 4-bit expert weights (arguments as in those calls; the expert calls
 * refuse outputs or a workspace that overlap another argument).  A call repeated
 * gives the same bits.  Calls of different sizes may not for the same row: where a
 * call has few pairs a row is summed over the two halves of k, in others over all of
 * it in order. */
int moe_expert_ffn_fp4(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                       const int32_t* offsets, const uint8_t* q_gate_up, const uint8_t* s_gate_up,
                       const uint8_t* q_down, const uint8_t* s_down, uint16_t* y_perm,
                       void* workspace, size_t workspace_bytes, void* stream);
int moe_expert_gate_up_fp4(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                           const int32_t* offsets, const uint8_t* q_gate_up,
                           const uint8_t* s_gate_up, uint16_t* h,
                           void* workspace, size_t workspace_bytes, void* stream);
int moe_expert_down_fp4(const moe_config_t* cfg, const uint16_t* h, const int32_t* offsets,
                        const uint8_t* q_down, const uint8_t* s_down, uint16_t* y_perm,
                        void* workspace, size_t workspace_bytes, void* stream);
int moe_layer_forward_fp4(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                          const float* sel_bias, const uint8_t* q_gate_up,
                          const uint8_t* s_gate_up, const uint8_t* q_down, const uint8_t* s_down,
                          uint16_t* out, int32_t* topk_ids_out, float* topk_w_out,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Expert LoRA ("Beam 1.0" miles recipes, section 5.5 "LoRA": an adapter of
 * rank 16 and alpha 32 on every routed expert, router frozen).  Each expert's
 * fused gate/up weight and its down weight carry one adapter; an adapted
 * weight W [out, in] computes W a + scale * B (A a).  The rank-wide first
 * factor is rounded once to bf16 after scaling: t = bf16(scale * fp32(a . A^T));
 * the second factor t . B^T accumulates in fp32 with the base GEMM before the
 * SwiGLU (gate/up) or the output rounding (down).  The down adapter reads the
 * bf16 h the base down GEMM reads.
 */
typedef struct moe_lora {
  const uint16_t* a_gate_up;  /* [E, r, H] bf16 row-major  */
  const uint16_t* b_gate_up;  /* [E, 2I, r] bf16 (rows as in w_gate_up: gate, then up) */
  const uint16_t* a_down;     /* [E, r, I] bf16            */
  const uint16_t* b_down;     /* [E, H, r] bf16            */
  int32_t rank;               /* r in {16, 32, 48, 64}; Beam's recipe uses 16 */
  float scale;                /* alpha / r; Beam's recipe: 32 / 16 = 2 */
} moe_lora_t;

/*
 * moe_expert_ffn and moe_layer_forward with expert LoRA on bf16 base weights
 * (base weights in cfg->weight_layout; adapters row-major, 16-byte aligned).
 * Workspace: MOE_ENTRY_EXPERT_FFN_LORA / MOE_ENTRY_LAYER_LORA.  A missing or
 * malformed `lora` returns MOE_ERR_INVALID_ARG.
 */
int moe_expert_ffn_lora(const moe_config_t* cfg, const uint16_t* x, const int32_t* perm_src,
                        const int32_t* offsets, const uint16_t* w_gate_up, const uint16_t* w_down,
                        const moe_lora_t* lora, uint16_t* y_perm,
                        void* workspace, size_t workspace_bytes, void* stream);
int moe_layer_forward_lora(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                           const float* sel_bias, const uint16_t* w_gate_up,
                           const uint16_t* w_down, const moe_lora_t* lora, uint16_t* out,
                           int32_t* topk_ids_out, float* topk_w_out,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Training: the gradients of the block around its experts, and the optimizer.
 *
 * The chain of one router training step on frozen experts is
 *   moe_route_logits, moe_permute, moe_expert_ffn (or _fp8, _lora), moe_combine,
 *   <loss>, moe_combine_backward, moe_route_backward, moe_adamw_step;
 * experts of the caller's own go between moe_dispatch and moe_combine, and
 * their gradients between moe_combine_backward and moe_dispatch_backward.
 *
 * moe_dispatch, moe_dispatch_backward, moe_combine_rows and
 * moe_combine_backward move rows of `dtype` (moe_dtype) and read num_tokens, hidden, topk (and routed_scaling)
 * of cfg only: 1 <= hidden <= 2^28, 1 <= topk <= 8, num_tokens * topk < 2^31.
 * Rows are dense; row pointers must be 16-byte aligned, though rows of odd
 * length within a tensor need not be.  perm_dst is moe_permute's (or any
 * injective map of pairs to rows); an entry outside [0, num_tokens * topk)
 * drops its pair.  Sorted rows that no pair names are neither read nor written.
 * Outputs that overlap an input or each other are refused
 * (MOE_ERR_INVALID_ARG).
 */
enum moe_dtype { MOE_DTYPE_BF16 = 0, MOE_DTYPE_FP32 = 1 };

/*
 * moe_route (replay == 0) or moe_route_replay (replay == 1, topk_ids an input,
 * sel_bias unused) with one more output:
 *   topk_logits  [T, topk] fp32 out: the router logit of each chosen expert
 *                (0 for a replayed id that names no expert)
 * The other outputs are those calls' bit for bit; workspace MOE_ENTRY_ROUTE.
 */
int moe_route_logits(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                     const float* sel_bias, int replay, int32_t* topk_ids, float* topk_w,
                     float* topk_logits, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Tokens sorted by expert: x_perm[perm_dst[p]] = topk_w[p] * x[t] for every
 * pair p = t*topk + j, in fp32 rounded once (topk_w NULL: a copy).
 *   x       [T, H] rows;  x_perm  [T*topk, H] rows out
 *   topk_w  [T, topk] fp32 or NULL
 */
int moe_dispatch(const moe_config_t* cfg, int dtype, const void* x, const int32_t* perm_dst,
                 const float* topk_w, void* x_perm, void* stream);

/*
 * Gradient of moe_dispatch, sums in fp32 in slot order:
 *   grad_x[t]       = sum_j topk_w[p] * grad_x_perm[perm_dst[p]]   [T, H] rows out
 *   grad_topk_w[p]  = <x[t], grad_x_perm[perm_dst[p]]>             [T, topk] fp32 out
 * (0 for a dropped pair).  topk_w NULL: weights of one.  x and grad_topk_w are
 * both given or both NULL, and only with topk_w.
 */
int moe_dispatch_backward(const moe_config_t* cfg, int dtype, const void* grad_x_perm,
                          const int32_t* perm_dst, const float* topk_w, const void* x,
                          void* grad_x, float* grad_topk_w, void* stream);

/*
 * moe_combine for rows of either type and any width (moe_combine takes bf16
 * rows of a multiple of 256 elements).
 *   y_perm [T*topk, H] rows, topk_w [T, topk] fp32, out [T, H] rows out
 */
int moe_combine_rows(const moe_config_t* cfg, int dtype, const void* y_perm,
                     const int32_t* perm_dst, const float* topk_w, void* out, void* stream);

/*
 * Gradient of moe_combine and moe_combine_rows (out[t] = routed_scaling * sum_j topk_w[p] *
 * y_perm[perm_dst[p]]):
 *   grad_y_perm[perm_dst[p]] = routed_scaling * topk_w[p] * grad_out[t]
 *                                                     [T*topk, H] rows out, or NULL
 *   grad_topk_w[p] = routed_scaling * <grad_out[t], y_perm[perm_dst[p]]>
 *                                                     [T, topk] fp32 out, or NULL
 * (0 for a dropped pair).  At least one output is wanted; y_perm is read for
 * grad_topk_w, topk_w for grad_y_perm, and either may be NULL without it.
 */
int moe_combine_backward(const moe_config_t* cfg, int dtype, const void* grad_out,
                         const void* y_perm, const int32_t* perm_dst, const float* topk_w,
                         void* grad_y_perm, float* grad_topk_w, void* stream);

/*
 * Gradient of moe_route / moe_route_replay from that of the combine weights
 * (cfg as in the forward call: shapes and renormalize).  With s = sigmoid of
 * the chosen logits and g = grad_topk_w,
 *   renormalize:  w_j = s_j / sum_i s_i,  dz_j = w_j (1 - s_j) (g_j - sum_i g_i w_i)
 *   otherwise:    dz_j = s_j (1 - s_j) g_j
 *   grad_w_router[e] = sum over the pairs of e of dz[p] * x[t]     [E, H] fp32 out
 *   grad_x[t] = grad_x_add[t] + sum_j dz[p] * w_router[e_j]        [T, H] bf16 out
 * Ids outside [0, E) have no part in it.  The selection (and sel_bias) has no
 * gradient.
 *   topk_ids, topk_logits    [T, topk], of moe_route_logits
 *   grad_topk_w              [T, topk] fp32
 *   perm_src, offsets        of moe_permute on the same topk_ids
 *   accumulate               1: grad_w_router is added to, 0: overwritten
 *   grad_x_add               [T, H] bf16 or NULL: the hidden state's gradient from
 *                            elsewhere (the experts); may be grad_x itself
 *   grad_x                   NULL: not wanted (then grad_x_add is NULL too)
 * Sums are fp32 in a fixed order.  Other than grad_x_add == grad_x, outputs (and
 * the workspace) that overlap an input or each other are refused.  With no
 * tokens nothing is written, grad_w_router included.  Workspace
 * MOE_ENTRY_ROUTE_BACKWARD.  Batches whose grids reach 2^32 threads return
 * MOE_ERR_UNSUPPORTED: num_tokens * topk * hidden around 2^40 (2^37 for 8
 * slots), num_tokens from 2^29, hidden from 2^24, and up to 4095 tokens with
 * grad_x num_tokens * hidden around 2^34.
 */
int moe_route_backward(const moe_config_t* cfg, const uint16_t* x, const float* w_router,
                       const int32_t* topk_ids, const float* topk_logits,
                       const float* grad_topk_w, const int32_t* perm_src, const int32_t* offsets,
                       const uint16_t* grad_x_add, int accumulate, float* grad_w_router,
                       uint16_t* grad_x, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One AdamW step (decoupled weight decay) over a list of tensors.  With
 * g = grad_scale * grad and t the step of the tensor (its own where it has one,
 * the list's otherwise; the moments are corrected for the steps they hold):
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p - lr weight_decay p - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32, p being the parameter, or the fp32 master of a bf16 one (which is
 * then rounded to nearest into the parameter).
 *
 * 32-bit states: m and v [n] fp32.  8-bit states: m and sqrt(v) as E4M3FN codes
 * [n], with one E8M0 scale (2^(code - 127)) per block of 32 consecutive
 * elements [ceil(n / 32)]; the scale is the least power of two, at least
 * 2^-126, by which the block's largest finite magnitude is at most 448.  Codes
 * are rounded stochastically, by a hash of (seed, step, place in the list,
 * element): 16 random bits against the remainder, so that the state's mean
 * follows changes far below a code step.  A sqrt(v) above zero keeps at least
 * the smallest code.  The update itself uses m and v before rounding.
 *
 * A gradient that is not finite reaches its own element alone (in 8 bits as
 * NaN).  All tensor pointers are 16-byte aligned except the scales; n may be
 * any number, 0 included.  State memory of zeros is a valid start (scale code 0
 * stands for 0).
 */
typedef struct moe_adamw_tensor {
  void* param;         /* [n] fp32, or bf16 with `master`                      */
  float* master;       /* [n] fp32 for a bf16 param, NULL for an fp32 one      */
  const void* grad;    /* [n] of grad_dtype                                    */
  void* m;             /* [n] fp32 or E4M3FN codes                             */
  void* v;             /* [n] fp32, or E4M3FN codes of sqrt(v)                 */
  uint8_t* m_scale;    /* [ceil(n/32)] E8M0, NULL with 32-bit states           */
  uint8_t* v_scale;
  int64_t n;           /* below 2^34                                           */
  int32_t param_dtype; /* moe_dtype                                            */
  int32_t grad_dtype;  /* moe_dtype                                            */
  int32_t state_bits;  /* 32 or 8                                              */
  /* The tensor's own t, where it has made fewer steps than the list (one whose
   * gradient came late, or comes now and then): step_dev (>= 1, read when the
   * step runs), or else step; NULL and 0 stand for the list's. */
  int64_t step;
  const int64_t* step_dev;
} moe_adamw_tensor_t;

typedef struct moe_adamw {
  double lr, beta1, beta2, eps, weight_decay; /* betas in [0, 1), the others >= 0 */
  double grad_scale;           /* factor on every gradient (clipping, loss scaling) */
  int64_t step;                /* t >= 1 of this step, for tensors without their own */
  /* Device scalars for steps replayed from a captured graph, each NULL or read
   * when the step runs: the step number in place of `step` (>= 1), the rate in
   * place of `lr`, and a further factor on the gradients. */
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale_dev;
  uint32_t seed;               /* of the 8-bit states' rounding                */
} moe_adamw_t;

/* `tensors`: host array, read during the call.  Tensors must not overlap. */
int moe_adamw_step(const moe_adamw_t* opt, const moe_adamw_tensor_t* tensors, int num_tensors,
                   void* stream);

/*
 * ---------------------------------------------------------------------------
 * Routing from logits: softmax or sigmoid scores over any number of experts,
 * its gradient, and the loss that balances the experts' load.
 *
 * With z the logits of a token and b an optional selection bias:
 *   s_e = 1 / (1 + exp(-z_e))              MOE_SCORE_SIGMOID
 *   s_e = exp(z_e) / sum_i exp(z_i)        MOE_SCORE_SOFTMAX
 *   v_e = s_e + b_e
 * A group's score is the sum of its group_best (1 or 2) largest v; the
 * topk_groups best groups are kept and the topk largest v in them chosen, in
 * descending order.  Values are compared in 64 bits; without a bias experts
 * are ordered by their logits.  Ties go to the lower index.
 *   A logit of -inf masks its expert, and so does a bias of -inf or NaN: it is
 * never chosen.  Where fewer than topk experts are left, the last slots get id
 * -1 and weight 0, as moe_permute and moe_combine drop them.  A logit of +inf
 * counts as the largest finite number.  A NaN logit is not chosen and makes
 * its row's weights, and its row's part of the gradient and of the loss, NaN.
 *
 * Limits: num_experts <= 1024, num_groups <= 64 (a divisor of num_experts),
 * topk <= 32, num_tokens < 2^26; others return MOE_ERR_UNSUPPORTED.  (The calls
 * that take the ids on, moe_permute and the expert calls, have 256 experts and topk
 * <= 8; other counts are for experts of the caller's own.)  Logits and
 * their gradient are dense [T, E] of logits_dtype and need only the alignment
 * of their elements.  Outputs that overlap an input or each other are refused.
 */
enum moe_score { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SOFTMAX = 1 };

typedef struct moe_select_config {
  int64_t num_tokens;   /* T >= 0                                                */
  int32_t num_experts;  /* E                                                     */
  int32_t num_groups;   /* groups of E / num_groups contiguous experts           */
  int32_t topk_groups;  /* groups kept                                           */
  int32_t group_best;   /* 1 or 2: values that a group's score adds              */
  int32_t topk;         /* at most the experts of the kept groups                */
  int32_t score;        /* moe_score                                             */
  int32_t renormalize;  /* 1: weight = s over the sum of the chosen s; 0: s      */
  int32_t logits_dtype; /* moe_dtype                                             */
} moe_select_config_t;

/*
 *   logits    [T, E]
 *   sel_bias  [E] fp32 or NULL: for choosing only
 *   topk_ids  [T, topk] int32 out, topk_w [T, topk] fp32 out
 */
int moe_select(const moe_select_config_t* cfg, const void* logits, const float* sel_bias,
               int32_t* topk_ids, float* topk_w, void* stream);

/*
 * moe_select on the logits of the block's router, x . W_r^T in FP32 as
 * moe_route computes them.  cfg gives num_tokens and hidden (shapes as in
 * moe_route), sel the selection, with cfg's num_tokens, 256 experts and fp32
 * logits.
 *   logits  [T, E] fp32 out or NULL: what moe_select_backward starts from
 * Workspace MOE_ENTRY_ROUTE of cfg.
 * By the block's rule (sigmoids, groups by two best) the choice is moe_route's but
 * where values are as near as fp32 roundings: moe_route and moe_layer_forward compare
 * fp32 scores, also without a bias, and take the lower index where all are 1.  A
 * router that those are to serve is trained on the ids of moe_route.
 */
int moe_route_select(const moe_config_t* cfg, const moe_select_config_t* sel, const uint16_t* x,
                     const float* w_router, const float* sel_bias, int32_t* topk_ids,
                     float* topk_w, float* logits, void* workspace, size_t workspace_bytes,
                     void* stream);

/*
 * Balance loss over the rows with an expert (an id in [0, E); T' of them).
 * With n_e the pairs of expert e, n their sum, and q the scores over their sum
 * over all experts (the softmax itself, or the sigmoids normalised):
 *   f_e = E n_e / n,   P_e = sum_t q_te / T',   loss = coef * sum_e f_e P_e
 *   load_e = coef f_e / T'
 * load is the loss's derivative by every q_te (f is a count: no gradient).
 *   topk_ids  [T, topk] int32 in
 *   loss      [1] fp32 out, load [E] fp32 out (zeros without such rows)
 * Sums by expert are 64 bits within a wave's tokens, fp32 over the 16 waves of a
 * workgroup and 64 bits across them, in a fixed order.  With no tokens nothing is written.  Workspace:
 * moe_balance_workspace_bytes.  Reads num_tokens, num_experts, topk, score and
 * logits_dtype of cfg.
 */
int moe_balance_workspace_bytes(const moe_select_config_t* cfg, size_t* bytes);
int moe_balance_loss(const moe_select_config_t* cfg, const void* logits, const int32_t* topk_ids,
                     float coef, float* loss, float* load, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Gradient of the weights of moe_select, and of moe_balance_loss, with respect
 * to all logits.  With g = grad_topk_w and C a row's slots that name an expert:
 *   sigmoid:                dz_e = s_e (1 - s_e) sum_{j of e} g_j
 *   sigmoid, renormalized:  dz_e = (1 - s_e) sum_{j of e} w_j (g_j - sum_C g_i w_i)
 *   softmax:                dz_e = s_e (sum_{j of e} g_j - sum_C g_i s_i)
 *   softmax, renormalized:  dz_e = sum_{j of e} w_j (g_j - sum_C g_i w_i)
 *   balance loss:           + grad_loss q_e (load_e - sum_i load_i q_i), times
 *                           (1 - s_e) for the sigmoid
 * Rows without such a slot get zeros.  The selection has no gradient.
 *   topk_ids     [T, topk] int32, in any order, repeated ones added up
 *   grad_topk_w  [T, topk] fp32, or NULL with load: no gradient of the weights
 *   load         [E] fp32 of moe_balance_loss, or NULL: no balance loss
 *   grad_loss    [1] fp32 on the device, or NULL: 1 (only with load)
 *   grad_logits  [T, E] out
 * Reads num_tokens, num_experts, topk, score, renormalize and logits_dtype of cfg.
 */
int moe_select_backward(const moe_select_config_t* cfg, const void* logits,
                        const int32_t* topk_ids, const float* grad_topk_w, const float* load,
                        const float* grad_loss, void* grad_logits, void* stream);

/* Static description of a status code; never NULL. */
const char* moe_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_MOE_H */
