/*
 * moe_experts.h -- C ABI of the MI355X (gfx950) routed top-k experts forward.
 *
 * What is computed (Hugging Face Transformers docs, "Experts backends" page,
 * introduction): for each token a router has chosen k experts; the token's hidden
 * state is projected through each chosen expert and the k results are summed with
 * the routing weights.  The expert is a gated MLP -- gate/up projection, SwiGLU,
 * down projection (same page, backend table "deepgemm_megamoe" row and the
 * "SonicMoE" section, where silu maps to SwiGLU):
 *
 *     out[t,:] = sum_{j<k} w[t,j] * W_down[e] ( silu(W_gate[e] x_t) * (W_up[e] x_t) ),
 *     e = idx[t,j],  silu(z) = z / (1 + exp(-z)).
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers, row-major, contiguous, 16-byte
 *     aligned, owned by the caller.  The library never frees or retains them.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *     on it and the call returns without waiting, except where stated.
 *   - Every argument is validated on the host before the first HIP call; on a
 *     validation error nothing is enqueued and no output is written.
 *   - The library allocates no device memory per call: scratch comes from the
 *     caller's workspace (size from moe_workspace_size).  Its only state is a
 *     lazily built per-device record (CU count), made on the first call on a
 *     device (the page's "DeepGEMM" section loads its kernel lazily as well).
 *   - Calls on one stream are ordered; two calls that share a workspace must not
 *     overlap in time.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 1

typedef enum {
  MOE_OK = 0,
  MOE_ERR_NULL_ARG = 1,            /* a required pointer is NULL                     */
  MOE_ERR_BAD_SHAPE = 2,           /* sizes out of range / not multiples / misaligned */
  MOE_ERR_UNSUPPORTED = 3,         /* dtype / scale-format combination not provided  */
  MOE_ERR_WORKSPACE_TOO_SMALL = 4, /* workspace_bytes < moe_workspace_size()         */
  MOE_ERR_BAD_INDEX = 5,           /* an expert id outside [0, E) (CHECK_INDICES)    */
  MOE_ERR_HIP = 6                  /* a HIP runtime call failed                      */
} moe_status;

typedef enum {
  MOE_F32 = 0,      /* IEEE binary32                                   */
  MOE_BF16 = 1,     /* bfloat16                                        */
  MOE_FP8_E4M3 = 2, /* OCP 8-bit E4M3 ("e4m3fn": max 448, no infinity) */
  MOE_FP4_E2M1 = 3  /* OCP 4-bit E2M1 (MX FP4: max 6), two codes per byte     */
} moe_dtype;

typedef enum {
  MOE_SCALE_NONE = 0,
  MOE_SCALE_F32 = 1,   /* fp8: one float32 scale per 128x128 weight block          */
  MOE_SCALE_UE8M0 = 2  /* one uint8 exponent b per block, scale = 2^(b-127); the
                          block is 128x128 for fp8 weights and 1x32 (one weight
                          row, 32 consecutive input channels) for fp4 weights      */
} moe_scale_fmt;

enum {
  /* Synchronise `stream` after the forward and return MOE_ERR_BAD_INDEX if any
   * topk_idx entry was outside [0, E).  Without it such a slot contributes
   * nothing and the call still returns MOE_OK. */
  MOE_FLAG_CHECK_INDICES = 1u,
  /* Bit-reproducible combine at every size: each slot's weighted expert output is
   * written to its own row and the k rows of a token are summed in slot order.
   * Without the flag this combine is used while the slot rows are small (float32
   * rows, 4*T*k*H bytes, at most 512 MiB; the bf16 rows of a bf16, fp8 or fp4 layer
   * on the grouped path, 2*T*k*H bytes, at most 1 GiB), and floating-point atomic adds
   * into a [T, H] accumulator above (or always with MOE_FLAG_ATOMIC_COMBINE). */
  MOE_FLAG_DETERMINISTIC = 2u,
  /* Path selection (both give the same result within tolerance): the grouped
   * path sorts slots by expert and runs grouped GEMMs; the decode path streams
   * each selected expert's weights once against its few tokens.  Default: decode
   * when T * k <= min(16 * E, 512) (at most one 16-row pass per expert on average)
   * and the decode path takes the problem, grouped otherwise.  The decode path takes bf16 weights with
   * I % 128 == 0 and T * k <= 2048 (its routing tables live in LDS); forcing it
   * on any other problem returns MOE_ERR_UNSUPPORTED. */
  MOE_FLAG_FORCE_GROUPED = 4u,
  MOE_FLAG_FORCE_DECODE = 8u,
  /* Combine with floating-point atomic adds into a float32 [T, H] accumulator at
   * every size (the smaller workspace); not with MOE_FLAG_DETERMINISTIC. */
  MOE_FLAG_ATOMIC_COMBINE = 16u,
  /* The gated activation a = gate(g) * u of the expert MLP (SonicMoE section: gated
   * activations silu, gelu or relu map to SwiGLU, GeGLU or ReGLU).  Default: SwiGLU,
   * gate = silu.  GELU: gate = GELU in its exact form z * Phi(z).  RELU: gate =
   * max(z, 0).  At most one of the two. */
  MOE_FLAG_ACT_GELU = 32u,
  MOE_FLAG_ACT_RELU = 64u
};

/* Problem description (plain values; no pointers). */
typedef struct {
  int64_t T;            /* tokens, >= 0                                              */
  int32_t H;            /* hidden size                                               */
  int32_t I;            /* expert intermediate size                                  */
  int32_t E;            /* number of experts, 1..1024                                */
  int32_t k;            /* experts per token, 1..E                                   */
  int32_t act_dtype;    /* moe_dtype of hidden and out: MOE_F32 or MOE_BF16          */
  int32_t weight_dtype; /* moe_dtype of the weights: MOE_F32 (with act MOE_F32),
                           MOE_BF16 (with act MOE_BF16), MOE_FP8_E4M3 or
                           MOE_FP4_E2M1 (act MOE_BF16)                               */
  int32_t scale_fmt;    /* moe_scale_fmt: != NONE exactly when weights are fp8 or
                           fp4; fp4 takes MOE_SCALE_UE8M0 only                       */
  uint32_t flags;       /* MOE_FLAG_*                                                */
} moe_problem;

/* Shape rules checked by every call taking a moe_problem:
 *   H % 128 == 0, I % 64 == 0 (f32, bf16 weights); H % 128 == 0, I % 128 == 0 (fp8, fp4);
 *   1 <= E <= 1024, 1 <= k <= E, T * k < 2^31, H, I <= 65536, and each of hidden,
 *   the intermediate [T*k, I] rows and one expert's W_gate_up below 4 GiB.            */

/* ABI version of the loaded library (MOE_ABI_VERSION). */
int moe_abi_version(void);

/* Human-readable name of a status code (static string). */
const char* moe_status_str(moe_status s);

/* Bytes of device workspace moe_experts_forward needs for problem *p (host only,
 * closed form, no HIP call).  The page's backend table sets the memory of the
 * "grouped_mm" row (tokens sorted by expert, activations of the selected experts
 * only) against the "batched_mm" row (the selected experts' parameters duplicated
 * per token); this sizes the grouped form's buffers, which hold the sorted slots
 * and their activations, never a copy of a weight.  Grows with T*k*(I + H) and T*H.
 * Errors: NULL_ARG (p or bytes NULL), BAD_SHAPE / UNSUPPORTED as for the forward.  When the k rows of a
 * token are combined as per-slot rows (always with MOE_FLAG_DETERMINISTIC; by default
 * while 4*T*k*H <= 512 MiB, or 2*T*k*H <= 1 GiB for a bf16, fp8 or fp4 layer, where that combine is
 * the faster one; never with MOE_FLAG_ATOMIC_COMBINE) it holds a [T*k, H] buffer instead
 * of the float32 [T, H]
 * accumulator: float32 rows with MOE_FLAG_DETERMINISTIC, and bf16 rows (each slot's
 * weighted row rounded once, the k rows summed in float32) on the default grouped path
 * of bf16, fp8 and fp4 layers. */
moe_status moe_workspace_size(const moe_problem* p, size_t* bytes);

/*
 * The routed top-k experts forward.
 *
 *   hidden          [T, H]        act_dtype
 *   topk_idx        [T, k] int32  chosen expert ids, 0 <= id < E (a repeated id in
 *                                 one row counts once per slot)
 *   topk_w          [T, k] float32 routing weights (used as given; no renormalising)
 *   w_gate_up       [E, 2I, H]    weight_dtype; rows [0, I) of expert e are the gate
 *                                 projection, rows [I, 2I) the up projection
 *   w_down          [E, H, I]     weight_dtype
 *   w_gate_up_scale [E, 2I/128, H/128]  fp8 only: float32, or uint8 for UE8M0; NULL otherwise
 *   w_down_scale    [E, H/128, I/128]   fp8 only; NULL otherwise
 *                   fp4 weights instead: w_gate_up [E, 2I, H/2] and w_down [E, H, I/2]
 *                   uint8, byte j of a row holding element 2j in its low nibble and
 *                   2j + 1 in its high nibble; UE8M0 scales w_gate_up_scale [E, 2I, H/32],
 *                   w_down_scale [E, H, I/32] (uint8, 4-byte aligned)
 *   out             [T, H]        act_dtype; overwritten (never accumulated into)
 *   workspace       device scratch of workspace_bytes >= moe_workspace_size(p)
 *
 * fp8 weights (page section "FP8 and FP4 quantized experts" and its note: float32
 * or UE8M0 block scales consumed directly; dynamic per-row activation scales):
 * the bf16 hidden states are quantised per token and per 128 channels to e4m3
 * with a float32 scale amax/448, and so is the SwiGLU output before the down
 * projection; weight block (r, c) dequantises to code * scale[r/128][c/128].
 * fp4 weights (same section: packed two per int8 with UE8M0 scales, DeepSeek-V4
 * style): the activations are quantised exactly as for fp8, and weight (r, c)
 * dequantises to e2m1(code) * 2^(scale[r][c/32] - 127).
 *
 * Returns MOE_OK once the work is enqueued (T == 0: nothing is enqueued).
 * Errors: NULL_ARG, BAD_SHAPE, UNSUPPORTED, WORKSPACE_TOO_SMALL before any HIP
 * call; BAD_INDEX only with MOE_FLAG_CHECK_INDICES (after a stream sync); HIP.
 *
 * Stream capture: without MOE_FLAG_CHECK_INDICES the call only launches kernels on
 * `stream` (no host wait, no memset, no allocation), with grids fixed by T, k, E, H
 * and I, so it can be captured into a HIP graph once (after one call outside the
 * capture on the device) and replayed for any ids and weights written into the same
 * buffers.
 */
moe_status moe_experts_forward(const moe_problem* p, const void* hidden, const int32_t* topk_idx,
                               const float* topk_w, const void* w_gate_up, const void* w_down,
                               const void* w_gate_up_scale, const void* w_down_scale, void* out,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward of e4m3 or fp4 experts on hidden rows that are quantised already, as
 * moe_rms_norm's 8-bit output or moe_quantize_rows_fp8 leave them: hidden_q [T, H] e4m3 codes
 * and hidden_scale [T, H/128] float32 (16-byte aligned) stand for hidden, and the forward's own
 * quantisation is left out.  Everything else, `out` (bf16) and the workspace among it, is as
 * in moe_experts_forward, and so is the result, bit for bit, for the same codes and
 * scales.  MOE_ERR_UNSUPPORTED for float32 and bf16 weights.
 */
moe_status moe_experts_forward_quantized(const moe_problem* p, const uint8_t* hidden_q, const float* hidden_scale,
                                         const int32_t* topk_idx, const float* topk_w, const void* w_gate_up,
                                         const void* w_down, const void* w_gate_up_scale, const void* w_down_scale,
                                         void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward without a workspace argument and without any allocation, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, results and errors as
 * moe_experts_forward, minus workspace and workspace_bytes: the workspace is a device
 * array inside the library of moe_noalloc_scratch_bytes() bytes (128 MiB), one copy per
 * GPU, held until the process ends (looked up once per device on its first call).
 * Problems whose moe_workspace_size exceeds it return MOE_ERR_WORKSPACE_TOO_SMALL before
 * any HIP call (the Qwen1.5-MoE-A2.7B-shaped prefill layer, T = 4096, needs 108 MiB; the
 * DeepSeek-V3-shaped layers need more: use moe_experts_forward for them).  The call makes
 * no hipMalloc, hipFree or other allocation.  Every call on one GPU uses that GPU's one
 * array: calls that overlap on one GPU (on different streams, or from different host
 * threads without ordering) race and may produce wrong results; calls ordered on one
 * stream are safe.  The array keeps the last call's contents; nothing the forward reads
 * from it needs to start at zero.
 */
moe_status moe_experts_forward_noalloc(const moe_problem* p, const void* hidden, const int32_t* topk_idx,
                                       const float* topk_w, const void* w_gate_up, const void* w_down,
                                       const void* w_gate_up_scale, const void* w_down_scale, void* out,
                                       void* stream);

/* Bytes of the allocation-free forward's device array (its largest workspace). */
size_t moe_noalloc_scratch_bytes(void);

/*
 * Routing bookkeeping alone: the stable sort of the T*k slots a = t*k + j by
 * chosen expert (page backend table, "grouped_mm" row: tokens are sorted by
 * their selected expert before one grouped GEMM).
 *
 *   counts  [E]   int32  slots choosing expert e
 *   offsets [E+1] int32  exclusive prefix sum of counts (offsets[E] = valid slots)
 *   perm    [T*k] int32  perm[p] = the slot at sorted position p; slots of one
 *                        expert stay in increasing slot order
 *   inv     [T*k] int32  inv[perm[p]] = p; -1 for a slot whose id is out of range
 *
 * Same workspace rules as moe_experts_forward (size from moe_workspace_size).
 * Out-of-range ids are left out of every output; with MOE_FLAG_CHECK_INDICES
 * the call synchronises and returns MOE_ERR_BAD_INDEX if there were any.
 */
moe_status moe_route(const moe_problem* p, const int32_t* topk_idx, int32_t* counts,
                     int32_t* offsets, int32_t* perm, int32_t* inv, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * The router step in front of the routing bookkeeping (Experts backends page,
 * introduction: tokens go to the top-k experts the router scores, and their
 * outputs are combined with the routing weights).  For each token t:
 *   p[e]        = softmax over the E logits of row t (float32: max-shifted expf,
 *                 divided by the sum);
 *   topk_idx[t] = the k experts of largest p in decreasing order, equal logits
 *                 going to the lower expert id (softmax is increasing, so the
 *                 choice is made on the logits themselves, exactly);
 *   topk_w[t]   = their p, divided by the sum of the k when renorm != 0;
 * then the bookkeeping of moe_route on the chosen ids, in the same pass.
 *
 *   logits   [T, E] float32, device; every row needs a finite entry and no NaN
 *   topk_idx [T, k] int32 out;  topk_w [T, k] float32 out
 *   counts, offsets, perm, inv: as moe_route
 *
 * k <= 64 (MOE_ERR_UNSUPPORTED above).  Same workspace rules as moe_route;
 * ids are always in range, so no index check is needed.
 */
moe_status moe_route_logits(const moe_problem* p, const float* logits, int renorm, int32_t* topk_idx,
                            float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm,
                            int32_t* inv, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dynamic per-row e4m3 quantisation (page section "FP8 and FP4 quantized
 * experts": per-row activation scales, static per-tensor scales rejected).
 * For each row and each group of 128 consecutive columns:
 *   amax = max |x| (float32), s = amax / 448 (float32, correctly rounded; 1 if
 *   amax == 0), q = e4m3(x / s) (float32 division, round to nearest even,
 *   saturating at +-448).
 *
 *   x_bf16 [rows, cols] bf16;  q [rows, cols] uint8 e4m3 codes;
 *   scales [rows, cols/128] float32.   cols % 128 == 0, rows >= 0.
 */
moe_status moe_quantize_rows_fp8(const void* x_bf16, int64_t rows, int32_t cols, uint8_t* q,
                                 float* scales, void* stream);

/* Describe the plan chosen for *p into buf (NUL terminated, truncated to len):
 * the path ("grouped" or "decode"), weight and scale formats, activation, combine,
 * tile shapes and workspace bytes.  Host only, no HIP call.  This is the library's
 * counterpart of the page's get_experts_implementation() ("Set an experts backend"
 * section), which reports the experts backend a model will run with; here the
 * choice between the sort-then-group path and the few-token decode path ("Decode
 * stage switch" section) is made per call from T, k, E and the flags, and this
 * reports it.  For fp8 and fp4 weights it also gives act_codes_offset and
 * act_scales_offset: byte offsets into the forward's workspace of the e4m3 SwiGLU
 * rows [T*k][I] (uint8) and their scales [T*k][I/128] (float32), in expert-sorted
 * slot order (the order of moe_route's perm); they hold the last forward's values
 * until the workspace is reused.  Errors: NULL_ARG (p or buf NULL, or len == 0),
 * BAD_SHAPE / UNSUPPORTED as for the forward. */
moe_status moe_plan_describe(const moe_problem* p, char* buf, size_t len);

/*
 * Instruction check (test export): nblocks independent block products on the block-scaled
 * 16x16x128 MFMA that the e4m3 and FP4 grouped kernels use for each 128-long block of
 * their dot products ("FP8 and FP4 quantized experts" section: the fp8 and fp4 expert
 * GEMMs), with the same operand layout and a zero accumulator.  It exists so that the
 * instruction's accumulation can be compared with exact sums; the parity window of the
 * requantised SwiGLU rows rests on that comparison.
 *
 *   fmt 0: a [nblocks][16][128] e4m3 codes, b [nblocks][16][128] e4m3 codes;
 *   fmt 1: a as above, b [nblocks][16][64] bytes of e2m1 codes (element k in the low
 *          nibble of byte k/2 for even k), b_scale [nblocks][16][4] UE8M0 exponents (one
 *          per column and 32-long k block);
 *   fmt 2: a and b as for fmt 0, b_scale [nblocks][16][4] UE8M0 bytes passed as the
 *          instruction's B scales by lane (column, k block) as for fmt 1; only one
 *          exponent per block (all 64 equal, as the e4m3 kernels pass UE8M0 weight
 *          scales) has a defined result;
 *   d [nblocks][16][16] float32 out: d[i][r][n] = sum_k a[i][r][k] * b[i][n][k] (fmt 1:
 *          times 2^(b_scale[i][n][k/32] - 127); fmt 2: times 2^(s - 127), s the block's
 *          exponent).
 * Device pointers; a and b 16-byte aligned.  Errors: UNSUPPORTED (fmt), BAD_SHAPE,
 * NULL_ARG, HIP.  Asynchronous on `stream`.
 */
moe_status moe_check_mfma_blocks(int fmt, const uint8_t* a, const uint8_t* b, const uint8_t* b_scale, float* d,
                                 int nblocks, void* stream);

/* Stages of one forward, in launch order (a stage a path does not use is skipped). */
enum {
  MOE_STAGE_ZERO = 0,      /* clear the float32 accumulator                      */
  MOE_STAGE_ROUTE = 1,     /* routing bookkeeping                                */
  MOE_STAGE_QUANT_X = 2,   /* fp8 and fp4: quantise the hidden states             */
  MOE_STAGE_GATE_UP = 3,   /* gate/up projection + SwiGLU                        */
  MOE_STAGE_QUANT_ACT = 4, /* not launched: fp8 / fp4 gate_up kernels quantise the
                              SwiGLU output in their epilogue                    */
  MOE_STAGE_DOWN = 5,      /* down projection + routing weight + combine         */
  MOE_STAGE_FINALIZE = 6,  /* round the accumulator to the output type           */
  MOE_STAGE_COUNT = 7
};

/*
 * Per-stage timing hook for profilers and benchmarks.  `events` points to
 * 2 * MOE_STAGE_COUNT hipEvent_t handles (entries may be NULL); while set, each
 * later moe_experts_forward (or _noalloc, _quantized) on the calling host thread
 * records events[2*s] on its stream just before stage s and events[2*s+1] just after
 * it.  The events of a stage that the call's path skips are not recorded:
 * moe_experts_forward_quantized skips MOE_STAGE_QUANT_X.  The handles are
 * copied; the caller keeps ownership of the events.  events == NULL (or n == 0)
 * clears the hook.  n must be 0 or 2 * MOE_STAGE_COUNT (else MOE_ERR_BAD_SHAPE).
 */
moe_status moe_set_stage_events(void* const* events, int n);

/* ---------------------------------------------------------------------------------------
 * Dense operators around the routed experts: the norm in front of the layer, the router's
 * projection, and the experts every token takes (gated projection, then a linear whose
 * residual is the routed experts' output).  Forward and backward.
 *
 * They keep the conventions above with one addition: activations have a row pitch.  A
 * pitch is in elements, 0 stands for packed rows, and otherwise it is at least the row's
 * length and at most 2^22.  Weights are packed.  No matrix has more than 2^34 elements.  Types are MOE_F32 or MOE_BF16; sums,
 * statistics and activations are computed in float32 and every output is rounded once to
 * its type (bf16: nearest even).  Results do not depend on timing: sums over workgroups
 * are added in a fixed order, without atomics.  Calls launch kernels only (no host wait, no
 * allocation, no memset), so they can be captured into a HIP graph; the current device
 * must be the one that `stream` and the buffers belong to.  Outputs do not overlap inputs,
 * except where stated.  T == 0: forward calls enqueue nothing, backward calls write zeros
 * to the parameters' gradients.
 * ------------------------------------------------------------------------------------- */

typedef enum { MOE_ACT_NONE = 0, MOE_ACT_SILU = 1, MOE_ACT_GELU = 2 /* z * Phi(z) */, MOE_ACT_RELU = 3 } moe_act;

typedef struct {
  int64_t T;          /* rows, 0 .. 2^22 - 1                                               */
  int32_t H;          /* row length, a multiple of 8, 8 .. 65536                           */
  int32_t dtype;      /* moe_dtype of every tensor that is not float32 by its name         */
  float eps;          /* >= 0 and finite                                                   */
  int64_t ldx;        /* pitch of x (backward: of dx)           a multiple of 8, or 0      */
  int64_t ldr;        /* pitch of residual (backward: of dh)    a multiple of 8, or 0      */
  int64_t ldh;        /* pitch of h                             a multiple of 8, or 0      */
  int64_t ldy;        /* pitch of y (backward: of dy)           a multiple of 8, or 0      */
} moe_norm_problem;

/*
 * Root-mean-square norm with the residual's addition.  Per row:
 *   h = x + residual, rounded to dtype (h = x without a residual);
 *   rstd = 1 / sqrt(mean_j h_j^2 + eps);   y_j = h_j * rstd * weight_j.
 * (The sum of squares is float32: where it passes 3.4e38 rstd is 0.)
 * The 8-bit output takes the same y in float32, before any rounding, by the rule of
 * moe_quantize_rows_fp8 (scale amax / 448 per 128 columns, 1 for a group where that is zero; codes
 * saturate at 448): the rows moe_experts_forward_quantized takes.
 *
 *   x [T, H], residual [T, H] or NULL, weight [H]
 *   y [T, H] out, or NULL when q is wanted alone;  rstd [T] float32 out
 *   h [T, H] out, required exactly when residual is given; may be x or residual itself
 *     (same pitch), which it then replaces
 *   q [T, H] uint8 e4m3 codes and q_scale [T, H/128] float32, packed, out; both or neither
 *     (MOE_BF16 only, H % 128 == 0)
 * Errors: NULL_ARG, BAD_SHAPE, UNSUPPORTED before any HIP call; HIP.
 */
moe_status moe_rms_norm(const moe_norm_problem* p, const void* x, const void* residual, const void* weight, void* y,
                        void* h, float* rstd, uint8_t* q, float* q_scale, void* stream);

/* Bytes of workspace moe_rms_norm_backward takes (partial sums of dweight). */
moe_status moe_rms_norm_workspace_size(const moe_norm_problem* p, size_t* bytes);

/*
 * Gradients of moe_rms_norm's y and h (n_j = h_j * rstd, g_j = dy_j * weight_j):
 *   dx_j = rstd * (g_j - n_j * mean_i(g_i n_i)) + dh_j;   dweight_j = sum_t dy_j n_j.
 * dx is the gradient of x and of the residual alike.
 *
 *   dy [T, H], h [T, H], weight [H], rstd [T] float32 (both as the forward left them)
 *   dh [T, H] or NULL: the gradient that reaches h along the residual stream
 *   dx [T, H] out; may be dy or dh itself (same pitch)
 *   dweight [H] out, or NULL
 */
moe_status moe_rms_norm_backward(const moe_norm_problem* p, const void* dy, const void* h, const void* weight,
                                 const float* rstd, const void* dh, void* dx, void* dweight, void* workspace,
                                 size_t workspace_bytes, void* stream);

typedef struct {
  int64_t T;          /* rows, 0 .. 2^22 - 1                                               */
  int32_t K;          /* inputs, a multiple of 8, 8 .. 65536                               */
  int32_t N;          /* outputs, 1 .. 2^20                                                */
  int32_t dtype;      /* moe_dtype of x, w, bias, pre, dx, dw and dbias                    */
  int32_t out_dtype;  /* moe_dtype of y, residual and dy: dtype or MOE_F32                 */
  int32_t act;        /* moe_act                                                           */
  int64_t ldx;        /* pitch of x                             a multiple of 8, or 0      */
  int64_t ldy;        /* pitch of y (backward: of dy)                                      */
  int64_t ldr;        /* pitch of residual                                                 */
  int64_t ldp;        /* pitch of pre                                                      */
  int64_t lddx;       /* pitch of dx                            a multiple of 8, or 0      */
} moe_linear_problem;

/* Which call a workspace is for: the forward, the backward call, or that without dbias (any other value: MOE_BACKWARD). */
enum { MOE_FORWARD = 0, MOE_BACKWARD = 1, MOE_BACKWARD_NO_BIAS = 2 };

/* Bytes of workspace of moe_linear (backward == MOE_FORWARD) or moe_linear_backward. */
moe_status moe_linear_workspace_size(const moe_linear_problem* p, int backward, size_t* bytes);

/*
 * Linear with bias, activation and residual:  z = x w^T + bias;  y = act(z) + residual.
 *
 *   x [T, K], w [N, K], bias [N] or NULL, residual [T, N] or NULL
 *   y [T, N] out; may be residual itself (same pitch), which it then replaces
 *   pre [T, N] out or NULL: z in dtype, what the backward pass of an activation reads
 * A router's logits are a linear with out_dtype MOE_F32.
 */
moe_status moe_linear(const moe_linear_problem* p, const void* x, const void* w, const void* bias, const void* residual,
                      void* y, void* pre, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of moe_linear:  dz = dy * act'(pre);  dx = dz w;  dw = dz^T x;  dbias = sum_t dz.
 * (The gradient of the residual is dy itself.)  relu'(0) = 0, and where pre <= 0 relu's dz is 0 whatever dy is;
 * relu of NaN is NaN, and so is its slope.  The two products take dz
 * rounded to dtype; with at most 32 rows, and unless it is a bf16 value already, in two such parts (16
 * bits of it; where the first part's sum is not finite it is the result, so infinities and NaN come out as with
 * more rows).  dbias sums it in float32 before that rounding.
 *
 *   dy [T, N], x [T, K], w [N, K]; pre [T, N] (not read, may be NULL, with MOE_ACT_NONE)
 *   dx [T, K], dw [N, K], dbias [N] out; each may be NULL, and then is not computed, and
 *   w (without dx) and x (without dw) may be NULL too
 */
moe_status moe_linear_backward(const moe_linear_problem* p, const void* dy, const void* x, const void* w,
                               const void* pre, void* dx, void* dw, void* dbias, void* workspace,
                               size_t workspace_bytes, void* stream);

typedef struct {
  int64_t T;          /* rows, 0 .. 2^22 - 1                                               */
  int32_t H;          /* inputs, a multiple of 8, 8 .. 65536                               */
  int32_t I;          /* outputs, a multiple of 8, 8 .. 65536                              */
  int32_t dtype;      /* moe_dtype of every tensor                                         */
  int32_t act;        /* moe_act of the gate: SILU, GELU or RELU                           */
  int64_t ldx;        /* pitch of x                             a multiple of 8, or 0      */
  int64_t lda;        /* pitch of a (backward: of da)           a multiple of 8, or 0      */
  int64_t ldp;        /* pitch of pre (rows of 2I)              a multiple of 8, or 0      */
  int64_t lddx;       /* pitch of dx                            a multiple of 8, or 0      */
} moe_gated_problem;

/* Bytes of workspace of moe_gated_linear (backward == MOE_FORWARD) or moe_gated_linear_backward. */
moe_status moe_gated_linear_workspace_size(const moe_gated_problem* p, int backward, size_t* bytes);

/*
 * Gated projection (SwiGLU, GeGLU, ReGLU) in one kernel:
 *   [gate | up] = x w_gate_up^T + bias;   a = act(gate) * up.
 * With moe_linear as its down projection it is the expert every token takes; w_gate_up
 * has the layout of one routed expert's weights.
 *
 *   x [T, H]; w_gate_up [2I, H], rows [0, I) gate, rows [I, 2I) up; bias [2I] or NULL
 *   a [T, I] out
 *   pre [T, 2I] out or NULL: [gate | up] in dtype, what the backward pass reads
 */
moe_status moe_gated_linear(const moe_gated_problem* p, const void* x, const void* w_gate_up, const void* bias, void* a,
                            void* pre, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of moe_gated_linear:  dz = [da * up * act'(gate) | da * act(gate)];
 * dx = dz w_gate_up;  dw = dz^T x;  dbias = sum_t dz.  Roundings as in moe_linear_backward.
 *
 *   da [T, I], x [T, H], w_gate_up [2I, H], pre [T, 2I]
 *   dx [T, H], dw [2I, H], dbias [2I] out; each may be NULL, with w_gate_up and x as there
 */
moe_status moe_gated_linear_backward(const moe_gated_problem* p, const void* da, const void* x, const void* w_gate_up,
                                     const void* pre, void* dx, void* dw, void* dbias, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------
 * Rows in expert order and back.  For layers whose experts run on sorted rows as calls of their
 * own (training, e4m3 experts one product at a time): moe_route's or moe_route_logits' inv gives
 * every slot's sorted position.  The conventions are those of the dense operators above.
 * ------------------------------------------------------------------------------------- */

typedef struct {
  int64_t T;          /* tokens, 0 .. 2^22 - 1                                             */
  int64_t rows;       /* rows of the sorted matrix, 0 .. 2^31 - 1                          */
  int32_t H;          /* row length, a multiple of 8 (e4m3: of 128), .. 65536              */
  int32_t k;          /* slots of a token, 1 .. 1024                                       */
  int32_t dtype;      /* moe_dtype of the rows: MOE_F32, MOE_BF16; moe_permute alone also MOE_FP8_E4M3 */
  int64_t ldt;        /* pitch of the tokens' rows (x, out, dout)  a multiple of 8 (e4m3: 16), or 0 */
  int64_t ldy;        /* pitch of the sorted rows (y, dy)          a multiple of 8 (e4m3: 16), or 0 */
} moe_permute_problem;

/*
 * y[inv[t*k + j]] = x[t] for every slot (t, j) with a position: 0 <= inv < rows (others, -1 among them, are left out).
 * Rows of y (and of y_scale) that no slot names are left as they were.  Positions are distinct, as moe_route leaves them.
 *
 *   x [T, H], inv [T*k] int32, y [rows, H] out
 *   x_scale [T, H/128] and y_scale [rows, H/128] float32, packed: the scales of e4m3 rows, moved along; both or neither
 * The gradient of x is moe_unpermute of y's gradient without weights.
 */
moe_status moe_permute(const moe_permute_problem* p, const void* x, const float* x_scale, const int32_t* inv, void* y,
                       float* y_scale, void* stream);

/*
 * out[t] = sum_j topk_w[t, j] y[inv[t*k + j]] over the slots with a position, in slot order, float32 sums rounded once; a
 * token without any gets zeros.
 *
 *   y [rows, H], inv [T*k] int32, topk_w [T, k] float32 or NULL (weights of 1), out [T, H]
 */
moe_status moe_unpermute(const moe_permute_problem* p, const void* y, const int32_t* inv, const float* topk_w, void* out,
                         void* stream);

/*
 * Gradients of moe_unpermute:  dy[inv[t*k + j]] = topk_w[t, j] dout[t];  dtopk_w[t, j] = <dout[t], y[inv[t*k + j]]>, 0 for a
 * slot without a position.  Rows of dy that no slot names are left as they were.
 *
 *   dout [T, H]; y [rows, H] (needed for dtopk_w alone); topk_w [T, k] or NULL
 *   dy [rows, H] out or NULL; may be y itself, which it then replaces;  dtopk_w [T, k] float32 out or NULL
 */
moe_status moe_unpermute_backward(const moe_permute_problem* p, const void* dout, const void* y, const int32_t* inv,
                                  const float* topk_w, void* dy, float* dtopk_w, void* stream);

/* ---------------------------------------------------------------------------------------
 * e4m3 matrix products with a scale for each block of 128: the dense operators on the weights of fp8
 * experts, for one matrix (a shared expert) or for all experts on sorted rows, with gradients.
 * The conventions are those of the dense operators above.
 *
 * x arrives as moe_rms_norm's 8-bit output, moe_quantize_rows_fp8 or moe_permute leave it: codes and one float32
 * scale per row and 128 columns.  Weights are codes with one scale per 128 x 128 block.  A slice
 * of 128 products is summed by the block-scaled MFMA, to within 2^-10 of its largest product; slices are added in
 * float32.  Results are rounded once to bf16.
 *
 * With E != 0 expert e multiplies rows offsets[e] .. offsets[e+1] - 1 of x by its own matrix: the offsets of
 * moe_route, int32, non-decreasing, at most T.  (Others are taken into [0, T] and made non-decreasing.)  Rows of y, a, pre
 * and dx that belong to no expert are left as they were.
 * ------------------------------------------------------------------------------------- */

typedef struct {
  int64_t T;          /* rows, 0 .. 2^22 - 1                                               */
  int32_t K;          /* inputs, a multiple of 128, 128 .. 65536                           */
  int32_t N;          /* outputs (gated: I), a multiple of 128, 128 .. 65536               */
  int32_t E;          /* experts, 1 .. 1024, or 0: one matrix for all rows                 */
  int32_t scale_fmt;  /* moe_scale_fmt of the weights: MOE_SCALE_F32 or MOE_SCALE_UE8M0    */
  int32_t act;        /* moe_act; linear with E != 0: MOE_ACT_NONE; gated: SILU, GELU or RELU */
  int64_t ldx;        /* pitch of x (codes, or bf16 in a backward call)  a multiple of 16, or 0 */
  int64_t ldy;        /* pitch of y or a (backward: of dy or da)  a multiple of 8, or 0    */
  int64_t ldr;        /* pitch of residual                        a multiple of 8, or 0    */
  int64_t ldp;        /* pitch of pre (gated: rows of 2N)         a multiple of 8, or 0    */
  int64_t lddx;       /* pitch of dx                              a multiple of 8, or 0    */
} moe_fp8_problem;

/*
 * Weights to e4m3 with one scale per 128 x 128 block, for `count` matrices [N, K] one after the other: up to 1024 of them and
 * 2^34 elements in all; N and K multiples of 128, 128 .. 65536, and N also twice such a number (gate and up rows).
 * The block's scale is amax / 448: float32, correctly rounded (MOE_SCALE_F32), or the smallest power of two that is not
 * below it, at least 2^-126 (MOE_SCALE_UE8M0); 1 for a block of zeros.  Codes as in moe_quantize_rows_fp8.
 *
 *   w [count, N, K] in dtype (MOE_F32 or MOE_BF16); q [count, N, K] uint8 out
 *   scales [count, N/128, K/128] float32, or uint8 exponents, out
 */
moe_status moe_quantize_blocks_fp8(const void* w, int32_t dtype, int32_t count, int32_t N, int32_t K, int32_t scale_fmt,
                                   uint8_t* q, void* scales, void* stream);

/* Bytes of workspace of moe_linear_fp8 (backward == MOE_FORWARD) or moe_linear_fp8_backward. */
moe_status moe_linear_fp8_workspace_size(const moe_fp8_problem* p, int backward, size_t* bytes);

/*
 * z = x w^T + bias;  y = act(z) + residual.
 *
 *   x_q [T, K] codes, x_scale [T, K/128] float32; w_q [N, K] codes, w_scale [N/128, K/128] (each with E first when E != 0)
 *   offsets [E+1] int32, or NULL with E == 0
 *   bias [N], residual [T, N], pre [T, N] out (z in bf16): each may be NULL, and is with E != 0 (MOE_ERR_UNSUPPORTED)
 *   y [T, N] bf16 out; may be residual itself (same pitch), which it then replaces
 */
moe_status moe_linear_fp8(const moe_fp8_problem* p, const uint8_t* x_q, const float* x_scale, const uint8_t* w_q,
                          const void* w_scale, const int32_t* offsets, const void* bias, const void* residual, void* y,
                          void* pre, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of moe_linear_fp8:  dz = dy * act'(pre);  dx = dz w;  dw = dz^T x;  dbias = sum_t dz.
 * w is the codes times their scales, x the bf16 rows that were quantised for the forward.  The products take e4m3: dz in
 * groups of 128 of its columns for dx; dz and x in groups of 128 of their rows (counted from the expert's
 * first) for dw.  These groups' scales are the smallest powers of two that are not below amax / 448, at least 2^-126 (1 for a
 * group of zeros); a value that is not finite has the NaN code.  dbias sums the float32 dz.
 *
 *   dy [T, N], x [T, K], pre [T, N] bf16 (pre is not read with MOE_ACT_NONE)
 *   dx [T, K], dw [E, N, K], dbias [N] bf16 out; each may be NULL, and then is not computed; w_q, w_scale
 *   (without dx) and x (without dw) may be NULL too; dbias is NULL with E != 0 (MOE_ERR_UNSUPPORTED)
 * An expert without rows gets zeros in dw.
 */
moe_status moe_linear_fp8_backward(const moe_fp8_problem* p, const void* dy, const void* x, const uint8_t* w_q,
                                   const void* w_scale, const int32_t* offsets, const void* pre, void* dx, void* dw,
                                   void* dbias, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of moe_gated_linear_fp8 (backward == MOE_FORWARD) or moe_gated_linear_fp8_backward. */
moe_status moe_gated_linear_fp8_workspace_size(const moe_fp8_problem* p, int backward, size_t* bytes);

/*
 * [gate | up] = x w_gate_up^T;  a = act(gate) * up.  w_gate_up_q [2N, K], rows [0, N) gate, as one routed expert's weights.
 *
 *   a [T, N] bf16 out;  pre [T, 2N] bf16 out or NULL: [gate | up], what the backward pass reads
 */
moe_status moe_gated_linear_fp8(const moe_fp8_problem* p, const uint8_t* x_q, const float* x_scale, const uint8_t* w_gate_up_q,
                                const void* w_scale, const int32_t* offsets, void* a, void* pre, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Gradients of moe_gated_linear_fp8:  dz = [da * up * act'(gate) | da * act(gate)];  dx = dz w_gate_up;  dw = dz^T x, in e4m3 as
 * in moe_linear_fp8_backward.   da [T, N], x [T, K], pre [T, 2N];  dx [T, K], dw [E, 2N, K] out or NULL
 */
moe_status moe_gated_linear_fp8_backward(const moe_fp8_problem* p, const void* da, const void* x, const uint8_t* w_gate_up_q,
                                         const void* w_scale, const int32_t* offsets, const void* pre, void* dx, void* dw,
                                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
