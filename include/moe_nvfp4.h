/*
 * moe_nvfp4.h -- C ABI of the routed mixture-of-experts FFN over NVFP4
 * weights, for one NVIDIA GB300 (sm_103a).
 *
 * What it computes, for every token t of a batch x[T][H]:
 *
 *   out[t] = sum_{j<k} w[t][j] * FFN_{id[t][j]}(x_t)   (+ FFN_shared(x_t))
 *   FFN_e(v) = Wd_e ( silu(Wg_e v) * (Wu_e v) ),   silu(z) = z / (1 + e^-z)
 *
 * with the router choosing id[t][*] and w[t][*] (softmax or sigmoid, top-k,
 * renormalised) and every weight W = E2M1(code) * E4M3(block scale) *
 * tensor_scale.  Sources (page title, section):
 *   "NVIDIA FP4-Local checkpoints on DGX Spark (TP=1, TP=2) ... #565",
 *   section 4 Round 1: NVFP4 weights as U8 codes and F8_E4M3 scales held as
 *   stored (#489); routed experts with a gate, up and down product and one
 *   tensor scale an expert (#517, #545); a whole batch routed in one run so
 *   each expert is read once (#740); gate, up and SwiGLU in one launch (#766);
 *   W4A16 / W4A4 activation formats (#687, list of formats at the end of the
 *   section); the SwiGLU output quantised for the down product (#760); down
 *   rows in BF16 rounded to nearest even (#914); the combine folded into the
 *   card sum (#701); the shared expert beside the routed ones (#686);
 *   router logits in fp32 (#763).  "bloomery 0.3.9", From our contributors:
 *   the router's normalisation policy is a named value (#772).
 *
 * Formats (the pages name them; the bit layouts are the OCP Microscaling ones):
 *   - NVFP4 tensor W[N][K]: codes uint8[N][K/2], element 2i in bits 0..3 and
 *     element 2i+1 in bits 4..7; scales uint8[N][K/16], one E4M3 byte per 16
 *     consecutive K values, row-major; one fp32 tensor scale.
 *   - E2M1: sign bit 3, magnitudes {0, .5, 1, 1.5, 2, 3, 4, 6}.
 *   - E4M3 ("FN"): bias 7, max 448, 0x7F/0xFF NaN, no infinities.
 *   - NVFP4 quantiser (weights and W4A4 activations), fp32 arithmetic:
 *       ts = amax / 2688;  s = E4M3_rne_sat((block_amax / 6) / ts);
 *       code = E2M1_rne_sat(x / (E4M3(s) * ts)).
 *
 * Conventions for every entry point:
 *   - Every pointer argument is DEVICE memory unless its comment says host;
 *     the caller owns it.  Pointers must be 16-byte aligned
 *     (MOE_ERR_MISALIGNED otherwise).
 *   - Calls are asynchronous and ordered on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream).  No call below allocates or synchronises
 *     except moe_plan_create / moe_plan_destroy / moe_plan_sync_status.
 *   - Host-side checks return an error at once and launch nothing.  Errors
 *     found on the device (a non-finite activation, a wait that ran out) set
 *     the plan's error word, which moe_plan_sync_status returns; outputs are
 *     unspecified after a device error.
 *   - A plan is used by one stream at a time.
 */
#ifndef MOE_NVFP4_H
#define MOE_NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,       /* null pointer, bad enum, T > max_tokens ... */
    MOE_ERR_UNSUPPORTED_SHAPE = 2, /* H or I not a multiple of 256/128, k > E ... */
    MOE_ERR_MISALIGNED = 3,        /* a pointer not 16-byte aligned */
    MOE_ERR_NONFINITE = 4,         /* device: an activation is NaN or infinite */
    MOE_ERR_TIMEOUT = 5,           /* device: a bounded wait ran out */
    MOE_ERR_CUDA = 6,              /* a CUDA runtime call failed */
    MOE_ERR_OOM = 7,               /* moe_plan_create could not allocate */
    MOE_ERR_DEVICE = 8             /* device: an internal check failed */
} moe_status;

typedef enum { MOE_ROUTER_SOFTMAX = 0, MOE_ROUTER_SIGMOID = 1 } moe_router_kind;

/* Word type of the router weight: fp32, or the checkpoint's bf16 words read
 * as they are stored ("NVIDIA FP4-Local checkpoints on DGX Spark ... #565",
 * section 4 Round 1: the router kept in its BF16 words, #732).  A bf16 word
 * widens to fp32 exactly, so the logits keep the fixed fp32 order below; the
 * router reads half the bytes. */
typedef enum { MOE_ROUTER_F32 = 0, MOE_ROUTER_BF16 = 1 } moe_router_dtype;

/* Block format of the expert weights.
 *   NVFP4: E2M1 codes, one E4M3 scale a 16-value block, one fp32 tensor scale a
 *          weight (the format described above).
 *   MXFP4: E2M1 codes, one E8M0 scale (2^(byte - 127)) a 32-value block, no
 *          tensor scale; the OCP Microscaling conversion: byte =
 *          clamp(floor(log2(block amax)) - 2 + 127, 0, 254), code =
 *          E2M1_rne_sat(x / 2^(byte - 127)).  The pages name MXFP4 routed
 *          experts and an MXFP4 routed prompt GEMM on block-scaled tensor cores
 *          ("NVIDIA FP4-Local checkpoints on DGX Spark ... #565", section 6
 *          Round 3; "bloomery 0.3.13", Also, #1154) and MX blocks of 32 with an
 *          E8M0 scale (#521).  In W4A4 the activations and the SwiGLU output
 *          are then MXFP4 as well (every block on its own scale, no batch
 *          amax).  MXFP4 plans need H, I (and the shared I) multiples of 512;
 *          they run on the CUDA cores, W4A4 also on the tcgen05 block-scaled
 *          MMAs (kind::mxf4, E8M0 scales), and W4A16 also on the warp MMAs
 *          (whose f16 operands hold code x scale exactly only for block scales
 *          from 2^-23 to 2^13: a weight block outside that range is a device
 *          error there). */
typedef enum { MOE_WEIGHTS_NVFP4 = 0, MOE_WEIGHTS_MXFP4 = 1 } moe_weight_format;

/* W4A16: activations stay bf16; the SwiGLU output is rounded to bf16 (RNE)
 *        before the down product.
 * W4A4:  activations are NVFP4-quantised (tensor scale from the batch amax);
 *        the SwiGLU output of all routed rows is rounded to fp32 and
 *        NVFP4-quantised with the tensor scale from its own batch amax (the
 *        shared expert's with its own). */
typedef enum { MOE_W4A16 = 0, MOE_W4A4 = 1 } moe_mode;

typedef struct {
    int32_t hidden;       /* H: multiple of 256, at most 8192 */
    int32_t inter;        /* I: per-expert intermediate, multiple of 128, at most 8192 */
    int32_t num_experts;  /* E: 1..1024 */
    int32_t top_k;        /* k: 1..min(E, 32) */
    int32_t max_tokens;   /* largest T a call may pass (sizes the workspace) */
    int32_t router;       /* moe_router_kind */
    int32_t renormalize;  /* 1: weights renormalised over the top-k; 0: not */
    int32_t mode;         /* moe_mode */
    int32_t has_shared;   /* 1: a shared expert is added to every token */
    int32_t shared_inter; /* shared expert's intermediate (multiple of 128, at most 8192) */
    int32_t router_dtype; /* moe_router_dtype of router_w in moe_route / moe_forward */
    int32_t weight_format; /* moe_weight_format of the expert weights */
} moe_config;

/* One weight stacked over `count` experts: codes [count][N][K/2] and
 *   NVFP4: scales [count][N][K/16] (E4M3), tensor_scale [count] fp32;
 *   MXFP4: scales [count][N][K/32] (E8M0), tensor_scale ignored (may be NULL).
 * All device memory. */
typedef struct {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *tensor_scale;
} moe_nvfp4;

/* gate and up are [I][H]; down is [H][I].  For the routed set count = E; for
 * the shared expert count = 1 and I = shared_inter. */
typedef struct {
    moe_nvfp4 gate, up, down;
} moe_expert_set;

typedef struct moe_plan_s *moe_plan;

/* Validate `cfg` (host memory), then allocate the plan and its device
 * workspace on the current device for cfg->max_tokens tokens.  *out receives
 * the plan (NULL on error).  This and moe_plan_set_profiling are the only
 * calls that allocate. */
moe_status moe_plan_create(const moe_config *cfg, moe_plan *out);

/* Free the plan and its workspace (synchronises the device first). */
moe_status moe_plan_destroy(moe_plan plan);

/* Router + grouping only (the steps "route" and "group by expert").
 *   x_bf16      [T][H] bf16 activations
 *   router_w    [E][H] fp32, or bf16 words when cfg.router_dtype is
 *               MOE_ROUTER_BF16 (16-byte aligned either way)
 *   router_bias [E] fp32 or NULL; added to the logits, so it moves both the
 *               selection and the weights
 * Outputs (device, caller-owned):
 *   topk_ids       [T][k] int32, experts by decreasing logit, ties -> lower id
 *   topk_w         [T][k] fp32 routing weights
 *   expert_offsets [E+1] int32, exclusive prefix of per-expert pair counts
 *   sorted_rows    [T*k] int32, pair indices t*k+j grouped by expert, each
 *                  expert's pairs in increasing t*k+j
 * Logits are fp32 with a fixed order: position h of the H dimension belongs to
 * lane h mod 32, each lane sums fmaf in increasing h from +0, the 32 lane
 * sums are combined by an xor butterfly over offsets 16, 8, 4, 2, 1, and the
 * bias is added last.  Indices and offsets are therefore reproducible bit for
 * bit. */
moe_status moe_route(moe_plan plan, const void *x_bf16, int32_t T, const void *router_w,
                     const float *router_bias, int32_t *topk_ids, float *topk_w,
                     int32_t *expert_offsets, int32_t *sorted_rows, void *stream);

/* The whole MoE FFN: route, group, [W4A4: quantise x], permute, gate/up +
 * SwiGLU, down with the routing weight, combine, [+ shared expert], bf16 out.
 *   routed: E experts' NVFP4 gate/up/down (host struct of device pointers)
 *   shared: NULL, or the shared expert (count 1) when cfg.has_shared
 *   out_bf16 [T][H] bf16, written with one round-to-nearest-even of the fp32
 *            sum.  T = 0 is a no-op. */
moe_status moe_forward(moe_plan plan, const void *x_bf16, int32_t T, const void *router_w,
                       const float *router_bias, const moe_expert_set *routed,
                       const moe_expert_set *shared, void *out_bf16, void *stream);

/* moe_forward with HOST activations and output: copies x (host, ideally
 * pinned) to the plan's device staging buffer, runs moe_forward, and copies
 * the result back to out_bf16_host.  The weights stay device pointers.
 * The copies are ordered on `stream`; the call returns before they finish
 * (synchronise the stream before reading out_bf16_host). */
moe_status moe_forward_host(moe_plan plan, const void *x_bf16_host, int32_t T, const void *router_w,
                            const float *router_bias, const moe_expert_set *routed,
                            const moe_expert_set *shared, void *out_bf16_host, void *stream);

/* W4A4 activation quantisation on its own (the step moe_forward runs first in
 * W4A4): tensor scale from the amax of all of x[T][H], then per 16-block
 * E4M3 scales and E2M1 codes.
 *   codes [T][H/2], scales [T][H/16], tensor_scale [1] fp32 (device).
 * An MXFP4 plan writes MXFP4 instead: scales [T][H/32] E8M0, tensor_scale 1. */
moe_status moe_quantize_act(moe_plan plan, const void *x_bf16, int32_t T, uint8_t *codes,
                            uint8_t *scales, float *tensor_scale, void *stream);

/* NVFP4 quantisation of fp32 weights w[batch][rows][cols] (device), one
 * tensor scale per batch item (amax of that item / 2688).  Writes codes
 * [batch][rows][cols/2], scales [batch][rows][cols/16], tensor_scale [batch].
 * cols must be a multiple of 16.  Needs no plan and no workspace:
 * tensor_scale doubles as the amax accumulator while the call runs. */
moe_status moe_quantize_nvfp4(const float *w, int32_t batch, int32_t rows, int32_t cols,
                              uint8_t *codes, uint8_t *scales, float *tensor_scale, void *stream);

/* Test hook: the device's fp32 -> E4M3 and fp32 -> E2M1 conversions, exactly
 * as the quantisers above apply them (round to nearest even, saturating to the
 * largest finite value; the sign is kept).  For every i < n, dst[i] =
 *   format MOE_FMT_E4M3: the E4M3 byte of src[i];
 *   format MOE_FMT_E2M1: the 4-bit E2M1 code of src[i] in bits 0..3.
 * src [n] fp32 and dst [n] uint8 are device memory (src 16-byte aligned).
 * Needs no plan.  MOE_ERR_INVALID_ARG for an unknown format or n < 0. */
typedef enum { MOE_FMT_E4M3 = 0, MOE_FMT_E2M1 = 1 } moe_format;
moe_status moe_convert_f32(const float *src, int64_t n, int32_t format, uint8_t *dst, void *stream);

/* MXFP4 quantisation (OCP MX, see moe_weight_format) of fp32 weights
 * w[rows][cols] (device; stack experts as rows): codes [rows][cols/2], E8M0
 * scales [rows][cols/32].  cols must be a multiple of 32.  Needs no plan. */
moe_status moe_quantize_mxfp4(const float *w, int64_t rows, int32_t cols, uint8_t *codes, uint8_t *scales,
                              void *stream);

/* Synchronise `stream`, then return and clear the plan's device error word
 * (MOE_OK, MOE_ERR_NONFINITE, MOE_ERR_TIMEOUT or MOE_ERR_DEVICE). */
moe_status moe_plan_sync_status(moe_plan plan, void *stream);

/* Device address and size of a plan workspace buffer, for tests that check a
 * step in isolation.  name: "h_codes", "h_scales", "h_scale_atoms" (W4A4 on
 * the tensor cores: the SwiGLU scales in 512-byte atoms of 128 rows x 4
 * blocks, byte (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of atom
 * (r / 128, b / 4)), "h_ts", "x_ts", "acc", "counts" (pairs an expert, where
 * the grouping runs as a launch of its own), "padded_offsets", "offsets",
 * "sorted", "pad_pair", "tiles", "h".
 * Returns MOE_ERR_INVALID_ARG for an unknown name. */
moe_status moe_plan_debug_buffer(moe_plan plan, const char *name, void **ptr, size_t *bytes);

/* W4A4 with MXFP4 weights on the tensor cores quantises the SwiGLU output in
 * the gate/up launch (every 32-value block on its own scale, one pass) and by
 * default writes only its codes and scales.  keep = 1: also store the fp32 h
 * (debug buffer "h"), for stage-by-stage checks.  Every other path stores h
 * anyway.  MOE_ERR_INVALID_ARG for a NULL plan. */
moe_status moe_plan_keep_h(moe_plan plan, int32_t keep);

/* Expert-FFN implementation moe_forward uses.  CUDA_CORE: weight-streaming
 * kernels on the CUDA cores (any shape).  TENSOR_CORE: grouped GEMMs on the
 * 5th-generation tensor cores (tcgen05; W4A4 block-scaled FP4, W4A16 with the
 * weights widened to f16 in tensor memory).  WARP_MMA (W4A16 only): the
 * weights widened in registers straight into warp-level f16 MMAs, for tiles
 * of up to 32 token rows.  AUTO picks WARP_MMA for W4A16 batches with fewer
 * than 2 (token, expert) pairs an expert on average (decode), the tcgen05
 * GEMMs for larger W4A16 batches and for W4A4 batches of 64 or more pairs,
 * and CUDA_CORE otherwise; the tensor paths need H and I multiples of 256.
 * MXFP4 W4A16 plans take no TENSOR_CORE (AUTO: WARP_MMA).  All compute the
 * same function (the tolerance of the parity tests covers their different
 * summation orders). */
typedef enum { MOE_PATH_AUTO = 0, MOE_PATH_CUDA_CORE = 1, MOE_PATH_TENSOR_CORE = 2, MOE_PATH_WARP_MMA = 3 } moe_path;

/* Select the expert-FFN implementation for later calls on this plan.
 * MOE_ERR_UNSUPPORTED_SHAPE if MOE_PATH_TENSOR_CORE or MOE_PATH_WARP_MMA is
 * asked for a plan whose mode or shapes it does not cover. */
moe_status moe_plan_set_path(moe_plan plan, int32_t path);

/* Stages of moe_forward, for moe_plan_read_profile. */
typedef enum {
    MOE_STAGE_ROUTE = 0,      /* logits + top-k (one kernel for T <= 16, else two) */
    MOE_STAGE_GROUP = 1,      /* histogram scan, stable placement, work lists */
    MOE_STAGE_QUANT_X = 2,    /* W4A4 activation quantisation */
    MOE_STAGE_PERMUTE = 3,    /* gather of activations into per-expert tiles */
    MOE_STAGE_GATE_UP = 4,    /* gate + up + SwiGLU */
    MOE_STAGE_QUANT_H = 5,    /* W4A4 quantisation of the SwiGLU output */
    MOE_STAGE_DOWN = 6,       /* down + routing weight + scatter-add */
    MOE_STAGE_FINALIZE = 7,   /* bf16 write of the combine */
    MOE_NUM_STAGES = 8
} moe_stage;

/* Turn per-stage timing on (1) or off (0).  While on, moe_forward records a
 * CUDA event pair on its stream around every stage (events come from a pool
 * the plan allocates here) and counts the kernels it launches. */
moe_status moe_plan_set_profiling(moe_plan plan, int32_t enable);

/* Synchronise the device, then add into ms[MOE_NUM_STAGES] the summed event
 * time of every stage recorded since the last read, and into
 * launches[MOE_NUM_STAGES] / calls[MOE_NUM_STAGES] the kernels launched and
 * the stage executions; clears the record.  Host arrays; any may be NULL. */
moe_status moe_plan_read_profile(moe_plan plan, float *ms, int64_t *launches, int64_t *calls);

/* Failure-detection check: launch one block whose waits use the same bounded
 * mbarrier wait as the expert kernels, on a barrier nothing will arrive on,
 * with the bound set to `wait_ns` nanoseconds (at most one second).  The wait
 * runs out, the kernel records MOE_ERR_TIMEOUT in the plan's error word and
 * returns normally; moe_plan_sync_status then reports it and the context stays
 * usable.  Faults nothing and hangs nothing. */
moe_status moe_plan_check_timeout(moe_plan plan, int64_t wait_ns, void *stream);

/* Routing and grouping, as moe_route, for callers that cannot allocate device
 * memory: code running inside another allocator's arena or under a
 * memory-capped runtime, or a host that forbids device allocations after
 * start-up.  The pages have no counterpart of this entry point; it exists for
 * those callers only.
 *
 * It needs no plan and calls no cudaMalloc, cudaFree or other allocating
 * routine.  Its scratch (logits, counts, offsets, placement) is one
 * file-scope device array of about 5.6 MB, held on every GPU that loads the
 * library until the process exits.  Limits: T * num_experts <= 2^20,
 * T * top_k <= 2^16, num_experts <= 1024, hidden a multiple of 256 up to
 * 8192; beyond them it returns MOE_ERR_UNSUPPORTED_SHAPE and launches nothing.
 * The first call on a device looks up the array's device address and sets the
 * grouping kernel's shared-memory size; make that first call before any stream
 * capture.  Every call shares the one array: calls that overlap on the GPU
 * (other streams, other threads) race and must be serialised by the caller.
 * The counts are cleared at the start of each call.  Outputs and argument
 * layout are moe_route's, with an fp32 router weight; router:
 * moe_router_kind; renormalize: 0 or 1.
 * Device-side findings (a non-finite activation) are not reported here. */
moe_status moe_route_static(const void *x_bf16, int32_t T, int32_t hidden, const float *router_w,
                            const float *router_bias, int32_t num_experts, int32_t top_k, int32_t router,
                            int32_t renormalize, int32_t *topk_ids, float *topk_w, int32_t *expert_offsets,
                            int32_t *sorted_rows, void *stream);

/* ======================================================================
 * The token path around the experts' products, for callers whose products are
 * their own (8-bit or bf16 products, training): the layer's norm, the sort of
 * the (token, slot) pairs by expert, rows to expert order and back, and the
 * gradients.  These entry points need no plan, allocate nothing, keep nothing
 * between calls and replay from CUDA graphs.  They launch on the current device,
 * which has to be the stream's and the arrays'.  Rows (x, residual, sum, y, q,
 * their gradients, weight) are 16-byte aligned, every other array is aligned to
 * its element.  Row counts, row offsets and strides may pass 32 bits in bytes.
 * ====================================================================== */

/* Element type of activations and of a norm's weight. */
typedef enum { MOE_DTYPE_F32 = 0, MOE_DTYPE_BF16 = 1, MOE_DTYPE_F16 = 2 } moe_dtype;

/* 8-bit output of moe_rms_norm.  Codes are E4M3 bytes q[T][H]; a group's scale
 * is what its codes are multiplied by.
 *   NONE:     no 8-bit output.
 *   E4M3_128: groups of 128 consecutive values, fp32 scales [T][ceil(H/128)].
 *   E4M3_ROW: one group a row, fp32 scales [T].
 *             For both: a = max(amax of |n| in the group, 2^-100), scale =
 *             a / 448, code = E4M3_rne_sat(n * 448 / a), where n * 448 / a is
 *             (s * weight) * (448 / amax |s * weight|), but n * (448 / a) in
 *             groups with amax |n| or amax |s * weight| of 2^-100 or less.  A
 *             NaN makes its group NaN.
 *   MXFP8:    groups of 32, E8M0 scales uint8[T][ceil(H/32)]: byte =
 *             clamp(floor(log2(amax)) - 8 + 127, 0, 254) (0 for an all-zero
 *             group), code = E4M3_rne_sat(n * 2^(127 - byte)); a group whose
 *             amax is not finite gets byte 255 and NaN codes.
 * The last group of a row is shorter where H is not a multiple of the group. */
typedef enum {
    MOE_QUANT_NONE = 0, MOE_QUANT_E4M3_128 = 1, MOE_QUANT_E4M3_ROW = 2, MOE_QUANT_MXFP8 = 3
} moe_quant8;

/* Residual addition and root-mean-square norm of T rows of H values:
 *   s = round(x + residual)  (s = x without a residual),
 *   rstd = 1 / sqrt(mean(s^2) + eps),  n = (s * weight) * rstd  in fp32,
 *   y = round(n), and/or n in 8 bits (moe_quant8).
 * The statistic is that of the stored (rounded) sum, summed in fp32: a row
 * whose sum of squares leaves fp32's range has rstd 0.  s * weight is held in
 * fp32 as well: what of it leaves that range, or its normal numbers, is lost.
 *   x        [T] rows of H, x_stride elements apart
 *   residual NULL, or [T] rows of H, residual_stride elements apart
 *   weight   [H], in `dtype` as x, residual, sum and y are
 *   sum      NULL, or [T][H] (only with a residual).  May be x's or residual's
 *            own memory where that one's stride is H.
 *   y        [T][H]; may be NULL when quant is not MOE_QUANT_NONE
 *   q, scales  as moe_quant8 says; NULL for MOE_QUANT_NONE
 *   rstd     NULL, or [T] fp32 (for the backward pass)
 * H: a multiple of 8 up to 16384; strides: multiples of 8, at least H;
 * eps > 0 and finite.  T = 0 is a no-op. */
moe_status moe_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                        const void *weight, int32_t T, int32_t H, int32_t dtype, float eps, int32_t quant,
                        void *sum, void *y, uint8_t *q, void *scales, float *rstd, void *stream);

/* Gradients of moe_rms_norm's y (and of its sum) for one shared input: with
 * n = sum * rstd and g = grad_y * weight,
 *   grad_in = rstd * (g - n * mean(g * n)) + grad_sum   (x's and residual's)
 *   grad_w  = sum over rows of grad_y * n               (fp32)
 * grad_y, sum, grad_sum (NULL: none), grad_in: [T][H] of `dtype`; grad_in may
 * be grad_y's or grad_sum's memory.  weight [H] of `dtype`, rstd [T], grad_w
 * [H] fp32 (written, not added to).  workspace: device memory of at least
 * moe_rms_norm_backward_workspace_for(T, H, dtype) bytes (0 for a few rows:
 * NULL then; moe_rms_norm_backward_workspace(T, H) is enough for any type),
 * 16-byte aligned, used during the call only.  Rows are added in a fixed
 * order: the same inputs on the same device give the same bits.  T = 0 writes
 * grad_w = 0. */
size_t moe_rms_norm_backward_workspace(int32_t T, int32_t H);
size_t moe_rms_norm_backward_workspace_for(int32_t T, int32_t H, int32_t dtype);
moe_status moe_rms_norm_backward(const void *grad_y, const void *sum, const void *weight, const float *rstd,
                                 const void *grad_sum, int32_t T, int32_t H, int32_t dtype, void *grad_in,
                                 float *grad_w, void *workspace, size_t workspace_bytes, void *stream);

/* Rows of the sorted layout of `pairs` pairs: enough for any routing when
 * every expert's segment is padded to a multiple of `align` rows, that is
 * floor((pairs + min(E, pairs) * (align - 1)) / align) * align.  -1 for
 * arguments moe_sort_pairs refuses. */
int64_t moe_sorted_rows(int64_t pairs, int32_t num_experts, int32_t align);

/* Stable sort of the pairs p = t*k + j by expert, from any router's ids.
 *   topk_ids       [T][k] int32; a pair whose id is outside [0, E) is dropped
 *   expert_offsets [E+1] int32: the first row of every expert's segment; each
 *                  segment holds its pairs in increasing p, then padding up to
 *                  a multiple of `align` rows (none for align = 1)
 *   sorted_rows    [rows] int32: the pair at a row, -1 where there is none
 *   pair_rows      [T][k] int32: the row of a pair, -1 where it is dropped
 * rows = moe_sorted_rows(T*k, E, align), at most 2^31 - 1; align a power of
 * two up to 256; k up to 32; E up to 1024.  With align = 1 and no pair dropped,
 * expert_offsets and sorted_rows are moe_route's.  T = 0 writes zero offsets.
 * More than 4096 pairs take a cluster of 16 blocks: MOE_ERR_CUDA on a partition
 * of a device that cannot hold one. */
moe_status moe_sort_pairs(const int32_t *topk_ids, int32_t T, int32_t k, int32_t num_experts, int32_t align,
                          int64_t rows, int32_t *expert_offsets, int32_t *sorted_rows, int32_t *pair_rows,
                          void *stream);

/* Token rows into expert order: row r of out is token sorted_rows[r] / k's row
 * of x, and zeros where sorted_rows[r] is -1.  Rows are copied as bytes, so x
 * is of any type; scales (NULL: none) are rows that go with them, such as
 * moe_rms_norm's.  Its gradient is moe_combine without weights.
 *   x      [T] rows of row_bytes, x_stride_bytes apart (multiples of 16)
 *   scales [T][scale_bytes], out_scales [rows][scale_bytes]
 *   out    [rows][row_bytes]
 * sorted_rows and pair_rows are moe_sort_pairs' of the same T, k and rows; an
 * entry out of range counts as -1 (a row about which the two disagree is
 * unspecified). */
moe_status moe_dispatch(const void *x, int64_t x_stride_bytes, int64_t row_bytes, const void *scales,
                        int32_t scale_bytes, int32_t T, int32_t k, const int32_t *sorted_rows,
                        const int32_t *pair_rows, int64_t rows, void *out, void *out_scales, void *stream);

/* Expert rows back into token order:
 *   out[t] = round(sum over j of weights[t][j] * y[pair_rows[t][j]] + base[t])
 * in fp32, in increasing j, base last.  Dropped pairs add nothing and rows of
 * padding are not read; a token without pairs gets base (0 without one).
 *   y [rows][H], base (NULL: none) and out [T][H] of `dtype`; weights [T][k]
 *   fp32 or NULL for 1 (the gradient of moe_dispatch).  out may be base's
 *   memory.  H: a multiple of 8 up to 65536. */
moe_status moe_combine(const void *y, int32_t dtype, int32_t T, int32_t k, int32_t H, const int32_t *pair_rows,
                       int64_t rows, const float *weights, const void *base, void *out, void *stream);

/* Gradients of moe_combine (base's is grad_out itself):
 *   grad_y[r] = round(weights[p] * grad_out[p / k]) for p = sorted_rows[r],
 *               zeros where that is -1
 *   grad_weights[t][j] = dot(grad_out[t], y[pair_rows[t][j]]) fp32, 0 where
 *               the pair is dropped
 * grad_out [T][H], y and grad_y [rows][H] of `dtype`; grad_y may be y's
 * memory.  weights, grad_weights [T][k] fp32. */
moe_status moe_combine_backward(const void *grad_out, const void *y, int32_t dtype, int32_t T, int32_t k, int32_t H,
                                const int32_t *sorted_rows, const int32_t *pair_rows, int64_t rows,
                                const float *weights, void *grad_y, float *grad_weights, void *stream);

/* ======================================================================
 * Around attention and in a decode step: the norm of query and key heads with
 * the position rotation, its gradients, products of a few tokens with a 4-bit
 * weight, and the whole layer of a few tokens with experts that are not
 * quantised.  As the entry points above: no plan, no allocation, nothing kept
 * between calls, graph replay, the current device.
 * ====================================================================== */

/* Root-mean-square norm of every query and key head, then the rotation by the
 * token's position.  Of a head row x of D values:
 *   n = (x * weight) / sqrt(mean(x^2) + eps)   in fp32,
 *   the first R values of n turn in R/2 planes: (a, b) -> (a cos - b sin,
 *   b cos + a sin), plane i being values i and i + R/2, or 2i and 2i + 1 where
 *   interleaved is 1; the other D - R values stay; rounded once.
 * The angle of plane i at position p is p * turns[i] / 2^64 of a whole turn, the
 * product taken modulo 2^64: turns[i] = floor(frequency_i / (2 pi) * 2^64)
 * modulo 2^64 for a frequency in radians a position.  Far and negative positions are exact.
 *   q [T][q_heads][D], k [T][k_heads][D]: the heads of a token lie behind one
 *     another, tokens q_stride and k_stride values apart (so both may be parts
 *     of the rows of one product)
 *   q_weight, k_weight [D], all of `dtype`; positions [T] int32; turns [R/2]
 *     (both unused and possibly NULL for R = 0)
 *   q_out, k_out: as q and k, with strides of their own; each may be its input
 *     in place (the same address and stride), and overlaps nothing else
 * D: a multiple of 16 up to 512; R: a multiple of 16 up to D; heads: up to 1024;
 * strides: multiples of 8, at least heads * D; eps > 0 and finite. */
moe_status moe_head_norm(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                         const void *k_weight, const int32_t *positions, const uint64_t *turns, int32_t T,
                         int32_t q_heads, int32_t k_heads, int32_t D, int32_t R, int32_t interleaved, int32_t dtype,
                         float eps, void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream);

/* Gradients of moe_head_norm.  With g = grad turned back and n = x * rstd:
 *   grad_in = rstd * (g * weight - n * mean(g * weight * n)),
 *   grad_weight = sum over tokens and heads of g * n   (fp32, written)
 * rstd is computed again from q and k.  grad_q, grad_k, q, k as above with
 * strides; grad_q_in [T][q_heads][D] and grad_k_in [T][k_heads][D] without;
 * each may be the memory of its grad or of its input where that one has no
 * stride either.  workspace: moe_head_norm_backward_workspace bytes (0 for a few
 * rows: NULL then), 16-byte aligned, used during the call only.  Sums are taken
 * in a fixed order.  T = 0 writes zeros to grad_qw and grad_kw. */
size_t moe_head_norm_backward_workspace(int32_t T, int32_t q_heads, int32_t k_heads, int32_t D, int32_t R);
moe_status moe_head_norm_backward(const void *grad_q, int64_t grad_q_stride, const void *grad_k, int64_t grad_k_stride,
                                  const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                  const void *q_weight, const void *k_weight, const int32_t *positions,
                                  const uint64_t *turns, int32_t T, int32_t q_heads, int32_t k_heads, int32_t D,
                                  int32_t R, int32_t interleaved, int32_t dtype, float eps, void *grad_q_in,
                                  void *grad_k_in, float *grad_qw, float *grad_kw, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Products of a few tokens with one 4-bit weight W[N][K], as moe_quantize_nvfp4
 * and moe_quantize_mxfp4 write it (moe_weight_format):
 *   out[t][n] = round(sum over k of x[t][k] * W[n][k]),  summed in fp32
 *   x      [T] rows of K, x_stride values apart, of `dtype` (bf16 or f16)
 *   weight host struct: codes [N][K/2], scales [N][K/16] (E4M3, none negative) or
 *          [N][K/32], tensor_scale one fp32 (NVFP4; ignored for MXFP4)
 *   out    [T][N] of out_dtype: `dtype` or MOE_DTYPE_F32; overlaps nothing else
 *   workspace: moe_linear_fp4_workspace_for(weight_format, dtype, T, N, K) bytes (0
 *          for most products: NULL then), 256-byte aligned, used during the call only;
 *          moe_linear_fp4_workspace(weight_format, T, N, K) is enough for either dtype
 * W is not rounded (a value has at most six significant bits and the tensor
 * scale is applied to the sum).  Small products take f16 rows as they are and bf16
 * ones to within 2^-32 of the largest finite magnitude of each of their blocks of
 * 256 (128 for more than 16 tokens) values.  Large ones, those that want a workspace,
 * take rows as integers of 23 bits: to within 2^-22 of the largest finite magnitude
 * of the 16 (MXFP4: 32) values that share a weight's scale or, where that is more, for
 * NVFP4 2^-39 of the row's, for MXFP4 2^-108 of the row's and at most 2^-128.  A sum is
 * finite where it is in fp32 arithmetic, whatever the sizes of rows, scales and tensor
 * scale.  A row that holds an infinity or a NaN gives what fp32 arithmetic gives and
 * leaves the other rows alone.  Sums are taken in a fixed order: equal inputs give equal
 * bits.  Waits inside a launch end after a second; if one ever runs out, out is NaN.
 * N: up to 2^31 - 1025; K: a multiple of 128 up to 65536; x_stride: a multiple of
 * 8, at least K; T: up to 2^20, made for up to 64 (every 32 tokens, of large products
 * every 16, read the weight once, the later ones from cache).  T = 0 is a no-op. */
size_t moe_linear_fp4_workspace(int32_t weight_format, int32_t T, int32_t N, int32_t K);
size_t moe_linear_fp4_workspace_for(int32_t weight_format, int32_t dtype, int32_t T, int32_t N, int32_t K);
moe_status moe_linear_fp4(const void *x, int64_t x_stride, const moe_nvfp4 *weight, int32_t weight_format, int32_t T,
                          int32_t N, int32_t K, int32_t dtype, int32_t out_dtype, void *out, void *workspace,
                          size_t workspace_bytes, void *stream);

/* The whole mixture-of-experts layer of up to 16 tokens with experts that are not
 * quantised, in two launches:
 *   out[t] = round(base[t] + sum over j of topk_w[t][j] * FFN_{topk_ids[t][j]}(x_t) + FFN_shared(x_t))
 * with the FFN of moe_forward, everything between x and out in fp32 (the SwiGLU
 * output is not rounded).  Logits, top-k and weights are moe_route's, in the same
 * order of sums, so both choose the same experts; an expert whose logit is NaN is
 * chosen after all others.
 *   x        [T][hidden] of `dtype` (moe_dtype), as the experts, base and out are
 *   router_w [E][hidden] fp32 or bf16 words (moe_router_dtype); router_bias [E] fp32 or NULL
 *   gate, up [E][inter][hidden], down [E][hidden][inter]
 *   shared_* the shared expert's [shared_inter][hidden] and [hidden][shared_inter],
 *            or NULL with shared_inter = 0
 *   base     NULL, or [T][hidden] added to the sum (the residual stream)
 *   out      [T][hidden]; may be base's or x's memory
 *   topk_ids [T][k] int32, topk_w [T][k] fp32: written
 *   workspace: moe_decode_layer_workspace bytes, 16-byte aligned, used during the
 *            call only
 * Sums are taken in a fixed order: equal inputs on the same device give equal
 * bits.  The second launch waits inside for its own first half, for a second at
 * most; if that ever runs out, out is NaN.
 * T: 0 to 16 (0 is a no-op); hidden, inter, shared_inter: multiples of 8 up to
 * 16384; E: 1 to 1024; k: 1 to min(E, 32).  x, router_w and the experts are
 * 16-byte aligned, the other arrays to their element. */
size_t moe_decode_layer_workspace(int32_t T, int32_t num_experts, int32_t inter, int32_t top_k, int32_t shared_inter);
moe_status moe_decode_layer(const void *x, int32_t dtype, int32_t T, int32_t hidden, const void *router_w,
                            int32_t router_dtype, const float *router_bias, int32_t num_experts, int32_t top_k,
                            int32_t router, int32_t renormalize, const void *gate, const void *up, const void *down,
                            int32_t inter, const void *shared_gate, const void *shared_up, const void *shared_down,
                            int32_t shared_inter, const void *base, void *out, int32_t *topk_ids, float *topk_w,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Text of a status code (static storage). */
const char *moe_status_string(moe_status s);

/* Library version string (static storage). */
const char *moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NVFP4_H */
