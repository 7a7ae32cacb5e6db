/*
 * moe_decode.h -- C ABI of the MI355X (gfx950) small-row MoE decode library.
 *
 * One call runs the decode / verify step of a top-8 routed mixture-of-experts
 * layer for 1..8 token rows, entirely in hand-written HIP kernels on the
 * caller's stream:
 *   RMSNorm folded into the router logits -> top-8 (ties to the lower expert
 *   ID) -> softmax gates -> expert dedup table -> FP8 activation blocks ->
 *   up/gate GEMV over low-bit weights -> SiLU * gate, mid re-quantised to FP8
 *   per 1x128 block -> down GEMV -> gate-weighted combine with a shared expert.
 * A second entry point, lowbit_gemv, is a dense decode GEMV over 1-bit
 * group-128 weights or, for the LM head after the last layer, FP8 weights.
 * Beside them stand the operators on rows grouped by an index: tokens sorted
 * by expert and back, with gradients (moe_sort, moe_gather, moe_combine), the
 * experts' step for any number of tokens (moe_wide_step), low-rank adapters of
 * many requests (lora_apply, lowbit_gemv_lora), and matrix products of the
 * sorted rows in bf16, with gradients (moe_product).  At the model's ends stand
 * the embedding lookup (embed) and the LM head's loss (lm_head_loss), with
 * gradients.
 *
 * Sources.  The operations follow the body of sgl-amd-mono PR #85 ("...MoE
 * expert dedup and weight loads, kernarg reload, LM-head loads"), quoted on the
 * GitHub page of sglang PR #47324 (cited below as "#85", with "Mod. row N" for
 * row N of its Modifications table), the README page "SGLang 1-Bit Turbo"
 * (section "PrismML 1-Bit GGUF Model Support (Q1_0_G128)"), and the page of
 * sglang PR #31683 "[ROCm][MI35X] Enable GLM-5.2-MXFP4 MTP speculative
 * decoding" for MXFP4 experts.
 *
 * Conventions for every function below:
 *  - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *    never allocates, frees or copies device memory on its own; all scratch
 *    lives in the caller's workspace.  Host objects (the context) are the only
 *    allocations it makes.
 *  - Layouts are row-major; "[N, K]" is N rows of K contiguous elements.
 *    Every pointer must be 16-byte aligned.
 *  - bf16 values are passed as uint16_t bit patterns.
 *  - Validation is synchronous and happens before anything is enqueued; on an
 *    error nothing is launched.  Device faults surface at the caller's next
 *    synchronisation of the stream.  No C++ exception crosses the ABI.
 *  - Work is enqueued on `stream` in stream order; the functions do not
 *    synchronise.  One context per stream: two steps that overlap on one
 *    workspace race.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* null / misaligned pointer, rows out of range, aliasing */
  MOE_ERR_UNSUPPORTED = 2, /* shape or format outside what the kernels implement */
  MOE_ERR_WORKSPACE = 3,   /* workspace missing or smaller than moe_decode_workspace_size */
  MOE_ERR_DEVICE = 4       /* a HIP launch error (hipGetLastError) */
} moe_status;

/* Weight formats. */
typedef enum {
  /* FP8 E4M3 (OCP E4M3FN, largest finite 448) codes uint8 [N, K] with one fp32
   * scale per 128x128 block, scales float [N/128, K/128] (#85 Mod. rows 18, 21:
   * FP8 expert weights; also lowbit_gemv's FP8 form). */
  MOE_FMT_FP8_E4M3_B128 = 1,
  /* MXFP4: E2M1 codes packed two per byte, element 2i in the low nibble,
   * uint8 [N, K/2], with one E8M0 exponent per 32 elements along K, uint8
   * [N, K/32] (MXFP4 page; #85 Mod. row 1: MXFP4 experts).  Routed experts
   * only; their mid is kept in fp32 (not re-quantised).  Needs hidden % 256
   * == 0 and inter <= 4096. */
  MOE_FMT_MXFP4 = 2,
  /* 1-bit group-128: [N, K/128] blocks of 18 bytes, an fp16 scale d
   * (little-endian) then 16 bytes of sign bits; bit i of byte b is element
   * 8b+i; bit 1 means -d, bit 0 means +d (1-Bit Turbo, Q1_0_G128).
   * lowbit_gemv, and routed experts of the decode step: their scales
   * pointers are unused (may be NULL), their mid is re-quantised to FP8 per
   * 1x128 block as for FP8 experts; needs hidden % 512 == 0, inter % 256 ==
   * 0, inter <= 4096 and FP8 activations. */
  MOE_FMT_Q1_G128 = 3,
  /* bf16 weights [N, K], no scales.  lowbit_gemv only (the tail's LM head
   * kept in bf16). */
  MOE_FMT_BF16 = 4
} moe_wfmt;

/* The experts' input (the up/gate activation). */
typedef enum {
  /* FP8 E4M3 per 1x128 block of u = bf16(x * gamma), scale amax/448 in fp32,
   * rstd applied after the dot (#85 Mod. row 10: FP8 activation blocks).  The
   * default (0, so a zero-initialised config gets it). */
  MOE_ACT_FP8_B128 = 0,
  /* u itself (bf16), rstd applied after the dot: no activation rounding, for
   * measuring what the FP8 blocks cost.  FP8 routed experts only (with
   * MXFP4 routed experts the config is MOE_ERR_UNSUPPORTED). */
  MOE_ACT_BF16 = 1
} moe_afmt;

/* flags */
enum {
  /* Skip the dedup: every (row, pick) streams its expert separately.  For the
   * bitwise A/B check that dedup changes no output bit (#85 Mod. row 16: a
   * row adds its units up in the order it would alone). */
  MOE_F_NO_DEDUP = 1u << 1
};

typedef struct {
  int32_t hidden;       /* H: multiple of 128, at most 16384 */
  int32_t inter;        /* I of a routed expert: multiple of 128, at most 16384 */
  int32_t n_experts;    /* E: multiple of 16, 16..1024 */
  int32_t top_k;        /* must be 8 */
  int32_t shared_inter; /* I of the shared expert: 0 for none, else equal to inter */
  int32_t max_rows;     /* 1..8: the widest step this context will run */
  float rms_eps;        /* RMSNorm epsilon */
  int32_t routed_fmt;   /* MOE_FMT_FP8_E4M3_B128, MOE_FMT_MXFP4 or MOE_FMT_Q1_G128 */
  int32_t shared_fmt;   /* MOE_FMT_FP8_E4M3_B128 */
  uint32_t flags;       /* MOE_F_* */
  int32_t act_fmt;      /* moe_afmt: MOE_ACT_FP8_B128 (0) or MOE_ACT_BF16 */
} moe_decode_config;

/* One stored matrix: codes and scales in the layout its format fixes. */
typedef struct {
  const void* codes;
  const void* scales;
} moe_tensor;

typedef struct {
  const uint16_t* rms_gamma; /* bf16 [H] */
  const uint16_t* router_w;  /* bf16 [E, H] */
  moe_tensor gate, up;       /* routed, expert-major stacks of [I, H] */
  moe_tensor down;           /* routed, expert-major stack of [H, I] */
  moe_tensor sh_gate, sh_up; /* shared expert [Is, H] (unused when Is == 0) */
  moe_tensor sh_down;        /* shared expert [H, Is] */
} moe_decode_weights;

typedef struct moe_decode_ctx moe_decode_ctx;

/* Bytes of device workspace a context with this config needs, or 0 when the
 * config is not supported. */
size_t moe_decode_workspace_size(const moe_decode_config* cfg);

/* Validate cfg, bind the caller's workspace (device, >= the size above) and
 * create a context.  Enqueues one small kernel on `stream` that clears the
 * workspace (so debug views read before the first step are defined); later
 * steps on the same stream are ordered after it.  The workspace must be
 * 256-byte aligned.
 * Returns MOE_ERR_UNSUPPORTED for configs the kernels do not implement,
 * MOE_ERR_WORKSPACE for a missing or short workspace. */
moe_status moe_decode_init(const moe_decode_config* cfg, void* workspace, size_t ws_bytes,
                           hipStream_t stream, moe_decode_ctx** out);

/* One decode step (#85: the MoE part of a decoder-layer launch).
 *  x    bf16 [rows, H] token rows (device)
 *  rows 0..max_rows; 0 enqueues nothing and returns MOE_OK (zero-work
 *       launches are skipped)
 *  w    weights; every pointer it holds is a device pointer
 *  out  bf16 [rows, H] (device); must not overlap x
 * The output is the MoE branch only: sum_j g_j * expert_{e_j}(x) + shared(x),
 * with no residual.  Selection, gates, dedup table, activation blocks and mid
 * of the last step stay readable through moe_decode_debug_view until the next
 * step on this context. */
moe_status moe_decode_step(moe_decode_ctx* ctx, const uint16_t* x, int32_t rows,
                           const moe_decode_weights* w, uint16_t* out, hipStream_t stream);

/* The decode step without a context or workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): the same validation, kernels and result
 * as moe_decode_step with a context created from `cfg`, but the step's
 * intermediates live in a static device array of the library
 * (MOE_DECODE_NOALLOC_MAX_WORKSPACE bytes, one per GPU, held until the
 * process ends).  It calls no hipMalloc, hipFree or other allocating routine;
 * the first call on a device looks up that array's device address.
 *  cfg  as for moe_decode_init; its workspace (moe_decode_workspace_size) must
 *       be at most MOE_DECODE_NOALLOC_MAX_WORKSPACE bytes, else
 *       MOE_ERR_WORKSPACE (a GLM-scale layer at 8 rows needs about 2.6 MB)
 *  x, rows, w, out, stream  as for moe_decode_step
 * Every call on one GPU shares that GPU's array, and the array keeps the
 * last call's intermediates: two calls that overlap on one GPU (other
 * streams, other threads) race and may corrupt each other's output.  No
 * debug view, timing or relaunch is available for these steps. */
#define MOE_DECODE_NOALLOC_MAX_WORKSPACE ((size_t)8 << 20)
moe_status moe_decode_step_noalloc(const moe_decode_config* cfg, const uint16_t* x,
                                   int32_t rows, const moe_decode_weights* w, uint16_t* out,
                                   hipStream_t stream);

/* Device pointers into the workspace holding the last step's intermediates. */
typedef struct {
  const float* logits;       /* [max_rows, E]: the fp32 values the top-8 compared */
  const float* rstd;         /* [max_rows] */
  const int32_t* ids;        /* [max_rows, 8] picks in top-8 order */
  const float* gates;        /* [max_rows, 8] softmax of the 8 picked logits */
  const int32_t* n_groups;   /* [1] D, the number of distinct routed experts */
  const int32_t* grp_expert; /* [max_groups] expert of group g (slot-major first use) */
  const uint8_t* grp_owner;  /* [max_groups, 2] (slot, row) of the group's first use */
  const uint8_t* grp_mask;   /* [max_groups] bit r set when row r uses the group */
  const uint8_t* grp_slot;   /* [max_groups, 8] slot where row r picked it, 0xFF if none */
  const uint8_t* act_q;      /* [max_rows, H] FP8 activation codes (zero with MOE_ACT_BF16) */
  const float* act_s;        /* [max_rows, H/128] their block scales (zero with MOE_ACT_BF16) */
  /* mid, per (row r, pick j) with j = 8 for the shared expert, at index
   * r * 9 + j, with stride mid_stride elements (a deduplicated expert's mid
   * appears under every (row, pick) that uses it): */
  const float* mid;          /* [max_rows, 9, mid_stride] fp32, before quantisation */
  const uint8_t* midq;       /* [max_rows, 9, mid_stride] FP8 codes */
  const float* midqs;        /* [max_rows, 9, mid_stride/128] block scales */
  const float* y;            /* [max_rows, 9, H] fp32 down output per (row, pick), before
                                the gate-weighted combine; same indexing as mid */
  int32_t max_groups;        /* min(8 * max_rows, E), or 8 * max_rows with MOE_F_NO_DEDUP */
  int32_t mid_stride;        /* max(I, Is) */
} moe_decode_debug;

moe_status moe_decode_debug_view(const moe_decode_ctx* ctx, moe_decode_debug* view);

/* Optional per-kernel timing: when `events` is non-null, every later step
 * records events[0] before its first kernel and events[i+1] after kernel i
 * (MOE_DECODE_N_KERNELS kernels), on the step's stream.  The caller owns the
 * events (hipEventCreate) and must keep them alive; pass NULL to stop. */
#define MOE_DECODE_N_KERNELS 5 /* router, routing (with the up/gate of the shared and the
                                  routed experts + mid), up/gate + mid (an empty span when
                                  the routing launch ran it), down, combine */
moe_status moe_decode_set_timing(moe_decode_ctx* ctx, hipEvent_t* events);

/* Kernel timing without per-kernel events: enqueues `reps` more launches of
 * one kernel of the last step enqueued on this context (the up/gate or the
 * down GEMV), with that step's row count, router logits, routing table and
 * activations in the workspace, and the weights `w` -- which must hold the
 * same experts at
 * possibly other addresses, e.g. another copy of the layer, so that repeated
 * launches stream from HBM rather than from a cache.  The relaunched kernel
 * rewrites the same workspace values (mid, or the down outputs); the step's
 * output is not touched.  For measurement only (the caller brackets the
 * launches with its own events).
 * Returns MOE_ERR_INVALID_ARG without a previous step, for another kernel, for
 * reps < 0 or for weights that step validation rejects. */
/* MOE_DECODE_K_UPGATE relaunches the launch that ran the step's up/gate: the
 * routing launch, routing included, when the up/gate runs in it. */
#define MOE_DECODE_K_UPGATE 2
#define MOE_DECODE_K_DOWN 3
moe_status moe_decode_relaunch(moe_decode_ctx* ctx, int32_t kernel,
                               const moe_decode_weights* w, int32_t reps, hipStream_t stream);

/* The routing launch's waits (#85 Mod. row 3 and its `poll` section: the
 * routed experts' weights stream as soon as the routing has chosen them).
 * In steps of up to 4 rows the up/gate runs in the routing launch, whose
 * routed up/gate blocks each wait for a record that the routing block
 * publishes (wider steps run the routing alone and do not wait); a wait gives up after `cap_ticks` of the GPU's
 * 100 MHz real-time counter (0 restores the default, 10 ms), and a block that
 * gives up counts itself and skips its work, so that the step's output is then
 * wrong but every kernel ends.  withhold = 1 makes the routing block publish no
 * record, so that every routed block gives up: for tests of that path only.
 * Applies to later steps and relaunches of this context.
 * Returns MOE_ERR_INVALID_ARG for a null context or withhold not 0 or 1. */
moe_status moe_decode_set_wait(moe_decode_ctx* ctx, uint32_t cap_ticks, int32_t withhold);

/* The number of routed blocks that gave up waiting, summed over every step and
 * relaunch of this context's workspace since moe_decode_init (0 when every
 * routed block got its record).  Reads it on `stream`, after the work enqueued
 * there, and synchronizes that stream. */
moe_status moe_decode_wait_timeouts(moe_decode_ctx* ctx, uint32_t* count, hipStream_t stream);

void moe_decode_destroy(moe_decode_ctx* ctx);

const char* moe_status_string(moe_status s);

/* Dense decode GEMV, in one of three weight formats.
 *
 * MOE_FMT_Q1_G128 -- 1-bit group-128 weights (1-Bit Turbo, Q1_0_G128):
 *   y[n] = bf16( sum_g d[n,g] * sum_{k in g} sign[n,k] * x[k] ),
 * x used as bf16 directly, fp32 accumulation.  w->k a multiple of 128 (at
 * most 16384); w->codes points to the [N, K/128, 18] blocks (device);
 * w->scales is unused (the scales are in the blocks).  rows 1..8 (the
 * page's path was batch 1; several rows need K a multiple of 256 and are
 * computed together, each row as its batch-1 definition).  x bf16 [rows, K],
 * y bf16 [rows, N], both 16-byte aligned.
 *
 * MOE_FMT_FP8_E4M3_B128 -- FP8 weights with one fp32 scale per 128x128 block,
 * for the tail's LM-head GEMV after the last layer (#85 Mod. row 24: the tail
 * keeps its LM-head weight loads in flight across its tiles):
 *   y[r][n] = bf16( sum_k dec(W[n,k]) * s[n/128,k/128] * x[r][k] ),
 * x bf16 used directly (no activation quantisation), fp32 accumulation.
 * w->n and w->k multiples of 128; w->codes uint8 [N, K] (16-byte aligned),
 * w->scales float [N/128, K/128]; rows 1..8; x bf16 [rows, K] (16-byte
 * aligned), y bf16 [rows, N].
 *
 * MOE_FMT_BF16 -- bf16 weights, the same tail GEMV with the LM head kept in
 * bf16 (#85 Mod. row 24; the page names no weight format for the tail):
 *   y[r][n] = bf16( sum_k W[n,k] * x[r][k] ),
 * fp32 accumulation.  w->n a multiple of 128, w->k of 64; w->codes bf16
 * [N, K] (16-byte aligned); w->scales is unused; rows 1..8; x bf16 [rows, K]
 * (16-byte aligned), y bf16 [rows, N].
 *
 * All forms: all pointers are device memory owned by the caller; x and y must not
 * overlap; rows == 0 or N == 0 is a no-op.  Validation runs before anything
 * is enqueued: a null or misaligned pointer, negative sizes or overlap ->
 * MOE_ERR_INVALID_ARG; an unknown format, sizes off the form's grid or too
 * many rows -> MOE_ERR_UNSUPPORTED; a launch error -> MOE_ERR_DEVICE. */
typedef struct {
  int32_t fmt, n, k;
  const void* codes;
  const void* scales;
} lowbit_matrix;

moe_status lowbit_gemv(const lowbit_matrix* w, const uint16_t* x, int32_t rows, uint16_t* y,
                       hipStream_t stream);

/* ---- Tokens sorted by expert and back, for batches of any width.
 *
 * ids [T, k] are the picks of T tokens (flat pick i = t k + j); an id outside
 * [0, n_experts) puts its pick in no group (a padded token, an expert of
 * another rank).  Work is enqueued on `stream` of the current device, where
 * every pointer has to live; pointers are 16-byte aligned (int32 and gate
 * pointers 4-byte). */
#define MOE_MAX_TOP_K 16
#define MOE_MAX_ROW (1 << 20) /* elements of a row */

/* Bytes of workspace moe_sort needs (0 for small batches), or 0 when the
 * shape is not supported. */
size_t moe_sort_workspace_size(int32_t tokens, int32_t top_k, int32_t n_experts);

/* The stable sort of the picks by expert:
 *  offsets  int32 [n_experts + 1]: expert e's rows are offsets[e] ..
 *           offsets[e+1] - 1 of the sorted order
 *  order    int32 [T k]: the flat pick of each sorted row, ascending within
 *           an expert; entries from offsets[n_experts] on are left as they were
 *  pos      int32 [T, k]: the sorted row of each pick, -1 for one in no group
 * top_k 1..16, n_experts 1..1024, tokens * top_k at most 2^24 (more:
 * MOE_ERR_UNSUPPORTED).  tokens == 0 writes offsets only.  The buffers must
 * not overlap.  `workspace` may be NULL where the size above is 0; it is
 * scratch, and two sorts that overlap in time need one each. */
moe_status moe_sort(const int32_t* ids, int32_t tokens, int32_t top_k, int32_t n_experts,
                    int32_t* offsets, int32_t* order, int32_t* pos, void* workspace,
                    size_t ws_bytes, hipStream_t stream);

typedef enum { MOE_BF16 = 0, MOE_F32 = 1 } moe_dtype;

/* Shapes of the row movements below.  `rows` is the number of rows of the
 * sorted buffers (tokens * top_k holds every pick; fewer do where only that
 * many picks are in a group); a pos outside [0, rows) is a pick without a
 * row.  pos is as moe_sort writes it: no row occurs twice. */
typedef struct {
  int32_t dtype; /* moe_dtype of every row buffer */
  int32_t tokens, top_k, hidden, rows;
} moe_row_shape;

/* xs[pos[t,j]] = x[t] for every pick with a row; x [tokens, hidden], xs
 * [rows, hidden].  Rows that no pick has are left as they were. */
moe_status moe_gather(const moe_row_shape* shape, const void* x, const int32_t* pos, void* xs,
                      hipStream_t stream);

/* Its gradient: dx[t] = sum_j dxs[pos[t,j]] over the picks with a row (0
 * without any), in pick order in fp32, rounded once. */
moe_status moe_gather_backward(const moe_row_shape* shape, const void* dxs, const int32_t* pos,
                               void* dx, hipStream_t stream);

/* out[t] = sum_j gates[t,j] y[pos[t,j]] (+ add[t] where add is not NULL), in
 * pick order in fp32, rounded once; gates fp32 [tokens, top_k].  The gates of
 * picks without a row are not used.  out may be add itself. */
moe_status moe_combine(const moe_row_shape* shape, const void* y, const int32_t* pos,
                       const float* gates, const void* add, void* out, hipStream_t stream);

/* Its gradients: dy[pos[t,j]] = gates[t,j] dout[t] (rows that no pick has are
 * left as they were) and dgates[t,j] = sum_h dout[t,h] y[pos[t,j],h] (fp32; 0
 * for a pick without a row).  The gradient of add is dout itself. */
moe_status moe_combine_backward(const moe_row_shape* shape, const void* dout, const void* y,
                                const int32_t* pos, const float* gates, void* dy, float* dgates,
                                hipStream_t stream);

/* The experts' step for any number of token rows whose routing is given: what
 * moe_decode_step computes after its top-8 (activation blocks, up/gate, mid,
 * down, gate-weighted sum with the shared expert), for batches wider than 8
 * rows.
 *  cfg     as for moe_decode_init, with FP8 routed experts and FP8
 *          activations (else MOE_ERR_UNSUPPORTED); max_rows and flags have no
 *          effect
 *  x       bf16 [tokens, H], 0..65536 tokens (0: nothing is enqueued)
 *  ids     int32 [tokens, 8] picks, as moe_decode_debug's; an id outside
 *          [0, n_experts) adds nothing to its token.  An expert may occur
 *          twice in a token's picks.
 *  gates   fp32 [tokens, 8]
 *  w       as for moe_decode_step; router_w is not used and may be NULL
 *  out     bf16 [tokens, H], overlapping no input
 *  workspace  device memory of at least moe_wide_workspace_size bytes,
 *          256-byte aligned; scratch of this call: steps that overlap in time
 *          need one each
 * Up to 16 picks an expert (tokens * 8 / n_experts) every sum is fp32's; in
 * wider batches the 128 products of a block of the routed experts' matrices and
 * of the shared expert's down matrix are added by the FP8 MFMA, as in the decode
 * step, which keeps 13 bits below the largest of each 8.  Among batches of either
 * kind a token's results are the same bits whatever else the batch holds.
 * Between the two, and against the decode step, whose sums run in other
 * groupings, they agree within rounding. */
#define MOE_WIDE_MAX_TOKENS 65536
size_t moe_wide_workspace_size(const moe_decode_config* cfg, int32_t tokens);
moe_status moe_wide_step(const moe_decode_config* cfg, const uint16_t* x, int32_t tokens,
                         const int32_t* ids, const float* gates, const moe_decode_weights* w,
                         uint16_t* out, void* workspace, size_t ws_bytes, hipStream_t stream);

/* ---- Matrix products of rows grouped by expert, between moe_gather and
 * moe_combine: with expert e's rows offsets[e] .. offsets[e+1] - 1 of the sorted
 * buffers (moe_sort's offsets),
 *   y[r] = W_e x[r].
 * bf16 operands, every sum in fp32, rounded once. */
#define MOE_MAX_PRODUCT_SIDE 32768
typedef struct {
  int32_t dtype;      /* moe_dtype of y (moe_product), of dw (moe_product_backward) */
  int32_t n_experts;  /* 1..1024 */
  int32_t rows;       /* rows of the sorted buffers, 0..2^24 */
  int32_t n, k;       /* an expert's matrix: multiples of 8, 8..MOE_MAX_PRODUCT_SIDE */
} moe_product_shape;

/* Bytes of workspace the two calls below need, or 0 when the shape is not
 * supported; 0 for most shapes, not where a few small tiles have long sums, whose
 * parts it holds.  The second is dw's: without dw none is needed. */
size_t moe_product_workspace_size(const moe_product_shape* shape);
size_t moe_product_backward_workspace_size(const moe_product_shape* shape);

/* y[r] = W_e x[r] for the rows r of every expert e:
 *  x        bf16 [rows, k], w bf16 [n_experts, n, k]
 *  offsets  int32 [n_experts + 1], ascending, at most rows (no access leaves
 *           the buffers where they are not; what the rows hold is then not
 *           defined)
 *  y        [rows, n]; rows of no expert are left as they were
 * The buffers must not overlap.  `workspace` may be NULL where the size above is
 * 0; it is scratch, 16-byte aligned, and calls that overlap in time need one
 * each. */
moe_status moe_product(const moe_product_shape* shape, const uint16_t* x, const uint16_t* w,
                       const int32_t* offsets, void* y, void* workspace, size_t ws_bytes,
                       hipStream_t stream);

/* Its gradients, of dy bf16 [rows, n] (each may be NULL, and is then not
 * computed):
 *  dx   bf16 [rows, k]: dx[r] = W_e^T dy[r]; rows of no expert are left as they
 *       were.  (x may be NULL without dw.)
 *  dw   [n_experts, n, k]: dw[e] = sum_r dy[r] x[r]^T over e's rows, 0 without
 *       any; with add != 0 it is added to dw, in fp32 before the rounding.
 *       (w may be NULL without dx.) */
moe_status moe_product_backward(const moe_product_shape* shape, const uint16_t* dy,
                                const uint16_t* x, const uint16_t* w, const int32_t* offsets,
                                uint16_t* dx, void* dw, int32_t add, void* workspace,
                                size_t ws_bytes, hipStream_t stream);

/* ---- Softmax cross entropy of the LM head: with the logits z[r, v] = w[v] . h[r]
 * of bf16 rows and weights (lowbit_gemv's bf16 head, for any number of rows),
 * which no call keeps.  Logits, exponentials and sums are fp32's. */
#define MOE_LOSS_MAX_ROWS (1 << 20)
#define MOE_LOSS_MAX_VOCAB (1 << 20)
typedef struct {
  int32_t dtype;   /* moe_dtype of dw (lm_head_loss_backward) */
  int32_t rows;    /* 0..MOE_LOSS_MAX_ROWS */
  int32_t vocab;   /* 1..MOE_LOSS_MAX_VOCAB */
  int32_t hidden;  /* a multiple of 8, 8..32768 */
} lm_head_shape;

/* Bytes of workspace the two calls below need, or 0 when the shape is not
 * supported (or has no rows). */
size_t lm_head_loss_workspace_size(const lm_head_shape* shape);
size_t lm_head_loss_backward_workspace_size(const lm_head_shape* shape);

/* lse[r] = log sum_v exp z[r, v] and loss[r] = lse[r] - z[r, targets[r]], the
 * loss 0 where the target is outside [0, vocab) (a padded row):
 *  h        bf16 [rows, hidden], w bf16 [vocab, hidden]
 *  targets  int32 [rows]
 *  loss, lse  fp32 [rows]
 * The buffers must not overlap.  The workspace is scratch of this call, 16-byte
 * aligned; calls that overlap in time need one each. */
moe_status lm_head_loss(const lm_head_shape* shape, const uint16_t* h, const uint16_t* w,
                        const int32_t* targets, float* loss, float* lse, void* workspace,
                        size_t ws_bytes, hipStream_t stream);

/* Its gradients: with d[r, v] = (exp(z[r, v] - lse[r]) - [v = targets[r]])
 * dloss[r], which enters dh and a bf16 dw as bf16 (at the target as the sum of
 * two), an fp32 dw as the sum of two bf16 everywhere (within 2^-16 of each term),
 *  dh  bf16 [rows, hidden]: dh[r] = sum_v d[r, v] w[v]
 *  dw  [vocab, hidden]: dw[v] = sum_r d[r, v] h[r]; with add != 0 it is added to
 *      dw, in fp32 before the rounding
 * of which either may be NULL, and is then not computed.  lse is lm_head_loss's
 * of the same h and w, dloss fp32 [rows].  A row whose target is outside [0,
 * vocab) has a dh of 0 and adds nothing to dw, whatever its h, lse and dloss
 * hold. */
moe_status lm_head_loss_backward(const lm_head_shape* shape, const uint16_t* h, const uint16_t* w,
                                 const int32_t* targets, const float* lse, const float* dloss,
                                 uint16_t* dh, void* dw, int32_t add, void* workspace,
                                 size_t ws_bytes, hipStream_t stream);

/* ---- Embedding lookup, rows of a table by token.  An id outside [0, vocab) is a
 * row without a token (padding).  Where the table is also the LM head, dtable is
 * lm_head_loss_backward's dw, which embed_backward adds to. */
#define MOE_EMBED_MAX_ROWS (1 << 24)
#define MOE_EMBED_MAX_VOCAB (1 << 20)
typedef struct {
  int32_t dtype;   /* moe_dtype of table and out, of dout */
  int32_t rows;    /* 0..MOE_EMBED_MAX_ROWS */
  int32_t vocab;   /* 1..MOE_EMBED_MAX_VOCAB */
  int32_t hidden;  /* 1..MOE_MAX_ROW */
} embed_shape;

/* out[r] = scale table[ids[r]], in fp32, rounded once; 0 for a row without a
 * token: ids int32 [rows], table [vocab, hidden], out [rows, hidden]. */
moe_status embed(const embed_shape* shape, const int32_t* ids, const void* table, float scale,
                 void* out, hipStream_t stream);

/* Bytes of workspace embed_backward needs (0 for few rows), or 0 when the shape
 * is not supported. */
size_t embed_backward_workspace_size(const embed_shape* shape);

/* Its gradient: dtable[v] = scale sum_r dout[r] over the rows r with ids[r] = v,
 * in fp32, rounded once; 0 for a token without rows.  With add != 0 the sum is
 * added to dtable, in fp32 before the rounding, and the tokens without rows are
 * left as they were.
 *  dout          [rows, hidden] of the shape's dtype
 *  dtable        [vocab, hidden] of table_dtype (moe_dtype)
 * The order of a sum depends on the ids alone.  `workspace` may be NULL where
 * the size above is 0; it is scratch, 16-byte aligned, and calls that overlap in
 * time need one each.  The buffers must not overlap. */
moe_status embed_backward(const embed_shape* shape, const int32_t* ids, const void* dout,
                          float scale, int32_t table_dtype, void* dtable, int32_t add,
                          void* workspace, size_t ws_bytes, hipStream_t stream);

/* ---- Low-rank adapters of many requests beside a projection they share.
 *
 * Row r with adapter i = ids[r] gets scale[i] * B_i (A_i x[r]) added to the
 * projection's output; an id outside [0, n_adapters) is a row without one.
 * A x is summed and kept in fp32; where rows * max_rank passes 2048 it enters the
 * second product as the sum of two bf16 parts, within 2^-16 of its value. */
typedef struct {
  int32_t n_adapters;   /* 0..1023 */
  int32_t max_rank;     /* a multiple of 8, 8..128 */
  int32_t n, k;         /* the projection's [n, k]; n a multiple of 8, at most MOE_MAX_ROW,
                           k a multiple of 64, at most 32768 */
  const uint16_t* a;    /* bf16 [n_adapters, max_rank, k] (device) */
  const uint16_t* b;    /* bf16 [n_adapters, n, max_rank] (device) */
  const int32_t* rank;  /* [n_adapters] (device) ranks used of each adapter, 0..max_rank, the
                           entries of a and b past them not used; NULL: all of max_rank */
  const float* scale;   /* [n_adapters] (device) */
} lora_set;

#define MOE_LORA_MAX_ROWS (1 << 20)

/* Bytes of workspace the two calls below need for `rows` rows, or 0 when the
 * set or the row count is not supported. */
size_t lora_workspace_size(const lora_set* l, int32_t rows);

/* y[r] = bf16( base[r] + scale_i B_i (A_i x[r]) ): x bf16 [rows, k], ids int32
 * [rows], base and y bf16 [rows, n]; y may be base itself.  rows == 0 or n ==
 * 0 is a no-op.  The workspace is scratch of this call, 16-byte aligned. */
moe_status lora_apply(const lora_set* l, const uint16_t* x, const int32_t* ids, int32_t rows,
                      const uint16_t* base, uint16_t* y, void* workspace, size_t ws_bytes,
                      hipStream_t stream);

/* lowbit_gemv with the adapters' terms added in its epilogue, before the one
 * rounding: y[r] = bf16( W x[r] + scale_i B_i (A_i x[r]) ), rows 0..8, every
 * weight format of lowbit_gemv.  l->n and l->k must be w's. */
moe_status lowbit_gemv_lora(const lowbit_matrix* w, const lora_set* l, const uint16_t* x,
                            const int32_t* ids, int32_t rows, uint16_t* y, void* workspace,
                            size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_DECODE_H */
