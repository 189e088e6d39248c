/*
 * mep.h -- C ABI of libmep: MoE token dispatch and combine on one gfx950 GPU.
 *
 * The operation is the MORI-EP intra-node dispatch/combine ("MORI-EP User
 * Guide", sections 2 Configuration and 3 Operator API; standard-MoE layout in
 * section 4), restated for one device: the receive buffers of R "virtual
 * ranks" are ordinary device buffers in local HBM, and this device's T tokens
 * are routed into them.  Ranks own contiguous expert blocks: expert e lives on
 * rank e / num_experts_per_rank.
 *
 * Conventions (every entry point):
 *   - Pointers named x, scales, recv_*, y, y8, out, em_*, indices, weights,
 *     recv_counts, src_token_pos and workspace, and all tensors of the router
 *     and expert calls, are DEVICE pointers, caller-owned, borrowed only for
 *     the duration of the asynchronous call on `stream` (a hipStream_t passed
 *     as void*; NULL = the null stream).  The library never allocates or frees
 *     device memory and never synchronises, except in mep_get_status.
 *   - All device pointers must be 16-byte aligned (MEP_ERR_ALIGN otherwise).
 *   - Errors a host can see (null pointers, bad shapes, alignment, call order)
 *     return a negative MEP_ERR_* code synchronously and launch nothing.
 *     Data errors only the device can see (an expert id out of range, a
 *     repeated expert in one token, expert-major overflow) set bits of a
 *     sticky device status word (MEP_DEV_*), read by mep_get_status.
 *   - A handle is not thread-safe; use one handle per stream.  Calls on one
 *     handle must be issued on one stream (or externally ordered).
 *   - Layouts are row-major and dense: [T,H] means row t at offset t*H.
 *   - Apart from mep_get_status, the calls launch kernels only (no memset,
 *     copy or host wait), so a sequence of them can be captured into a HIP
 *     graph; a replay reuses the handle state of the capture (its plan).  An
 *     iteration whose plan (mep_plan, mep_plan_dispatch or
 *     mep_dispatch_standard_moe) is captured keeps its MEP_DEV_* bits apart
 *     (per planned token, and one word for the expert-major overflow that its
 *     plan clears), so every replay starts clean without an extra launch:
 *     mep_get_status returns the bits of the latest replay (of its last plan,
 *     if it holds several), mep_reset between replays is allowed and changes
 *     nothing there.  The next plan issued outside capture starts a new reset
 *     epoch.
 */
#ifndef MEP_H
#define MEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- return codes ------------------------------------------------------- */
#define MEP_OK 0
#define MEP_ERR_NULL (-1)    /* a required pointer is NULL                     */
#define MEP_ERR_CONFIG (-2)  /* config fields out of range or inconsistent      */
#define MEP_ERR_SHAPE (-3)   /* a size argument out of range                    */
#define MEP_ERR_ALIGN (-4)   /* a device pointer is not 16-byte aligned         */
#define MEP_ERR_STATE (-5)   /* call order violated (e.g. dispatch before plan) */
#define MEP_ERR_HIP (-6)     /* the HIP runtime reported an error               */
#define MEP_ERR_DEVICE (-7)  /* mep_get_status: device status word is non-zero  */
#define MEP_ERR_NOMEM (-8)   /* mep_create: the host heap could not hold a handle */

/* ---- device status bits (sticky until mep_reset) ------------------------- */
#define MEP_DEV_BAD_INDEX 1   /* an expert id outside [0, E): that token is not
                                 dispatched and combines to +0                  */
#define MEP_DEV_DUP_EXPERT 2  /* a token names one expert twice (still routed)  */
#define MEP_DEV_EM_OVERFLOW 4 /* expert-major rows exceed cap_em; rows past it
                                 are dropped                                    */

/* ---- payload and layout selectors --------------------------------------- */
#define MEP_QUANT_NONE 0              /* dispatch payload: bf16 bit copy        */
#define MEP_QUANT_FP8_E4M3_BLOCK128 1 /* dispatch payload: OCP E4M3 codes with
                                         one fp32 scale per 128 columns          */
#define MEP_QUANT_FP8_CARRY 2         /* dispatch payload arrives already as OCP
                                         E4M3 bytes with scale_dim fp32 scales
                                         per row; both are carried unchanged
                                         ("Choosing an EP API and backend": the
                                         HIP backend's dispatch can move FP8
                                         rows that arrive quantized)             */
#define MEP_QUANT_FP4_CARRY 3         /* as MEP_QUANT_FP8_CARRY for FP4 rows: H/2
                                         bytes per row (two E2M1 codes a byte),
                                         scale_dim 32-bit scale words per row,
                                         both carried unchanged (same passage) */
#define MEP_QUANT_MXFP4 4             /* dispatch payload: OCP MX FP4 -- per 32
                                         columns an E8M0 scale byte, shared
                                         exponent floor(log2(amax)) - 2 clamped
                                         to [-127, 127]; codes E2M1(x / 2^exp),
                                         round to nearest even, saturating at 6,
                                         even column in the low nibble; all-zero
                                         block: scale byte 0.  Rows of H/2
                                         bytes; the H/32 scale bytes of a row
                                         fill its H/128 scale words ("Choosing
                                         an EP API and backend": FP4 conversion
                                         kernels on gfx950; the block format is
                                         this library's reading)                */
#define MEP_RANK_MAJOR 0              /* combine input: [R, cap, H] bf16         */
#define MEP_EXPERT_MAJOR 1            /* combine input: [cap_em, H] bf16         */
#define MEP_RANK_SUM 2                /* combine input: [R, cap, H] bf16 rows from
                                         mep_convert_combine_input, which already
                                         carry the weights                       */

/*
 * Configuration.  Fields follow EpDispatchCombineConfig ("MORI-EP User Guide",
 * section 2 Configuration); the multi-node fields (gpu_per_node,
 * rdma_block_num, num_qp_per_pe, kernel_type) and launch geometry have no
 * meaning on one device and are absent.
 */
typedef struct mep_config {
  int32_t hidden_dim;                 /* H: > 0, multiple of 8; of 128 when quantising, of
                                         16 when carrying E4M3, of 32 when carrying FP4  */
  int32_t scale_dim;                  /* 32-bit scale words per row: 0 for bf16; H/128
                                         when quantising; any >= 0 when carrying         */
  int32_t num_experts_per_rank;       /* epr: 1..64                                       */
  int32_t num_experts_per_token;      /* k: 1..32, k <= R*epr                              */
  int32_t max_num_inp_token_per_rank; /* cap: receive rows per rank and the largest T, >= 1 */
  int32_t world_size;                 /* R virtual ranks: 1..64                           */
  int32_t rank;                       /* source rank used in src_token_pos: 0..R-1        */
  int32_t quant;                      /* MEP_QUANT_*  (the pages' data_type choice)        */
} mep_config;

typedef struct mep_handle mep_handle;

/* Human-readable name of a MEP_OK / MEP_ERR_* code (static string). */
const char *mep_error_string(int code);

/* Bytes of device workspace a handle needs for this config, or 0 if the config
 * is invalid.  The workspace holds the routing plan (receive row of every
 * (token, top-k slot)), the expert-major maps and the status word. */
size_t mep_workspace_bytes(const mep_config *cfg);

/* Check the config and bind it to a caller-owned device workspace of at least
 * mep_workspace_bytes(cfg) bytes, which must be zero-filled before its first
 * use (it holds the status words).  Host-only: launches nothing, makes no HIP
 * call.  *out receives a host-heap handle freed by mep_destroy.  One
 * workspace serves one handle at a time. */
int mep_create(const mep_config *cfg, void *workspace, size_t workspace_bytes,
               mep_handle **out);
int mep_destroy(mep_handle *h);

/*
 * Routing plan ("MORI-EP User Guide" section 3: dispatch() returns
 * recv_num_token; get_dispatch_src_token_pos() gives each received row's
 * origin).  For T tokens with top-k expert ids indices[T,k] (int32):
 *   - each token is sent once to each distinct rank among its experts (the
 *     first top-k position naming that rank owns the row; later positions on
 *     the same rank share it);
 *   - recv_counts[r] (int32, R entries) = rows rank r receives;
 *   - inside a rank, rows are in ascending token order, and
 *     src_token_pos[r*cap + s] (int32, [R,cap]) = rank*(R*cap) + t for the
 *     token t in slot s < recv_counts[r]; entries past the count are not
 *     written.
 * The plan is kept in the workspace and stays valid (for any number of
 * dispatch/combine calls: routing replay) until mep_reset or the next plan.
 * 0 <= T <= cap.
 */
int mep_plan(mep_handle *h, const int32_t *indices, int32_t T, int32_t *recv_counts,
             int32_t *src_token_pos, void *stream);

/*
 * Dispatch ("MORI-EP User Guide" section 3 dispatch(input, weights, scales,
 * indices)): every planned (token, rank) row receives
 *   recv_x[r, s, :]       the token row: x[T,H] bf16 copied bit for bit
 *                         (MEP_QUANT_NONE, recv_x is [R,cap,H] bf16); or its
 *                         OCP E4M3 codes (MEP_QUANT_FP8_E4M3_BLOCK128, recv_x is
 *                         [R,cap,H] bytes): per 128 columns b, scale =
 *                         amax_b / 448 (fp32) and code =
 *                         E4M3_rne_satfinite(x / scale), signed zero when
 *                         amax_b == 0; or, MEP_QUANT_FP8_CARRY, the E4M3 bytes
 *                         of x[T,H] copied;
 *   recv_scales[r, s, :]  the block scales ([R,cap,H/128] fp32), or the carried
 *                         scales[t, :] ([R,cap,scale_dim]); NULL for bf16;
 * MEP_QUANT_MXFP4 writes [R,cap,H/2] packed E2M1 bytes and [R,cap,H/32] E8M0
 * bytes (= H/128 words; x finite: NaN/Inf inputs are not supported);
 * MEP_QUANT_FP4_CARRY copies H/2 bytes of x and the
 * scale_dim words of scales[t, :];
 *   recv_weights[r, s, :] the token's k weights (fp32 [R,cap,k]);
 *   recv_indices[r, s, :] the token's k expert ids (int32 [R,cap,k]).
 * scales is the caller's [T,scale_dim] 32-bit input for the carry modes and is
 * ignored otherwise.  Rows past recv_counts[r] are not written.  Needs a
 * valid plan; x, weights, scales and indices hold the planned T tokens.
 */
int mep_dispatch(mep_handle *h, const void *x, const float *weights, const float *scales,
                 const int32_t *indices, void *recv_x, float *recv_scales, float *recv_weights,
                 int32_t *recv_indices, void *stream);

/*
 * Fused routing plan + dispatch: the same outputs as mep_plan followed by
 * mep_dispatch (recv_counts, src_token_pos, the receive rows, scales, weights
 * and ids, and a valid plan in the handle), in fewer launches -- one launch up
 * to 256 tokens, else two.  The pages pair the two steps the same way:
 * dispatch() itself returns recv_num_token ("MORI-EP User Guide" section 3).
 */
int mep_plan_dispatch(mep_handle *h, const int32_t *indices, int32_t T, int32_t *recv_counts,
                      int32_t *src_token_pos, const void *x, const float *weights,
                      const float *scales, void *recv_x, float *recv_scales,
                      float *recv_weights, int32_t *recv_indices, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * outputs as mep_plan_dispatch (recv_counts, src_token_pos, the receive rows,
 * scales, weights and ids, with the same argument layouts, alignment and
 * host-side checks) with no handle and no workspace.  The plan's scratch is a
 * 2 MiB device array inside the library, one per GPU, held until the process
 * ends; its address on the stream's GPU is looked up on the first call there
 * (hipGetSymbolAddress, no allocation).  The batch must fit it: 179 KiB
 * for 4096 tokens at top-8 on 8 ranks, roughly T*(12 + 4k) + (T/64)*R*5
 * bytes in general (each section rounded up to 256 bytes); MEP_ERR_SHAPE
 * beyond 2 MiB
 * (no launch).  Every call on one GPU shares that scratch, so calls that
 * overlap on one GPU (concurrent streams, or threads) race; calls ordered on
 * one stream do not.  Tokens with bad expert ids are not dispatched, as in
 * mep_plan_dispatch, but no status word is kept for mep_get_status.  No plan
 * is left behind: combine needs a handle and its own plan.
 */
int mep_plan_dispatch_noalloc(const mep_config *cfg, const int32_t *indices, int32_t T,
                              int32_t *recv_counts, int32_t *src_token_pos, const void *x,
                              const float *weights, const float *scales, void *recv_x,
                              float *recv_scales, float *recv_weights, int32_t *recv_indices,
                              void *stream);

/*
 * Standard-MoE layout ("MORI-EP User Guide" section 4,
 * convert_dispatch_output(): packed rows, per-expert counts, source info).
 * From the dispatch outputs (recv_x, recv_scales or NULL, recv_indices,
 * recv_counts, and the plan's src_token_pos), for every expert e in global
 * order:
 *   em_counts[e]        rows naming expert e (int32, E = R*epr entries);
 *   em_offsets[e]       first row of e's segment; segments are padded to
 *                       multiples of 128 rows (int32, E+1 entries,
 *                       em_offsets[E] = rows used);
 *   em_x[em_offsets[e] + i, :]      the i-th such receive row (ascending
 *                       receive slot), in the row format of recv_x;
 *   em_scales[...]      its scale words (scale_dim per row; NULL when 0);
 *   em_src_pos[...]     its src_token_pos.
 * Padding rows are not written.  cap_em is the row capacity of em_x /
 * em_scales / em_src_pos; T*k + 127*E always suffices.  Rows past cap_em are
 * dropped and set MEP_DEV_EM_OVERFLOW.  Needs a valid plan.  MEP_ERR_SHAPE if
 * T*k + 127*E exceeds INT32_MAX (the int32 offsets could not hold the
 * padded segments).
 */
int mep_to_expert_major(mep_handle *h, const void *recv_x, const float *recv_scales,
                        const int32_t *recv_indices, const int32_t *recv_counts,
                        const int32_t *src_token_pos, void *em_x, float *em_scales,
                        int32_t *em_counts, int32_t *em_offsets, int32_t *em_src_pos,
                        int64_t cap_em, void *stream);

/*
 * Standard-MoE dispatch ("MORI-EP User Guide" section 4,
 * dispatch_standard_moe(): dispatch and format conversion combined): the same
 * em_x / em_scales / em_counts / em_offsets / em_src_pos as mep_plan +
 * mep_dispatch + mep_to_expert_major would produce for these T tokens (rows of
 * each expert in ascending token order, segments padded to 128 rows, padding
 * not written), but written straight from x without the rank-major receive
 * buffers.  A token naming one expert twice gets one row (mapped from the
 * first position naming it).  Leaves the handle ready for
 * mep_combine(MEP_EXPERT_MAJOR) and mep_get_route(NULL, em_row); the
 * rank-major calls need a new mep_plan.  scales as for mep_dispatch.
 * 0 <= T <= cap; cap_em (and the T*k + 127*E bound) as for
 * mep_to_expert_major.
 */
int mep_dispatch_standard_moe(mep_handle *h, const int32_t *indices, int32_t T, const void *x,
                              const float *scales, void *em_x, float *em_scales,
                              int32_t *em_counts, int32_t *em_offsets, int32_t *em_src_pos,
                              int64_t cap_em, void *stream);

/*
 * Combine ("MORI-EP User Guide" section 3 combine(): expert outputs gathered
 * back to token order as a weighted combination; section 4
 * combine_standard_moe() for the expert-major input; "Choosing an EP API and
 * backend": the HIP backend's combine gathers in BF16 or FP32).  For every
 * planned token t:
 *   out[t, h] = bf16_rne(acc),  acc = +0.0f, then for j = 0..k-1 in order
 *               acc = fmaf(weights[t, j], y_j[h], acc)
 * where y_j is the bf16 expert-output row holding (t, expert j):
 *   MEP_RANK_MAJOR:   y is [R,cap,H]; y_j = y[rank of expert j, slot of t];
 *                     a row shared by two experts is used once per expert;
 *   MEP_EXPERT_MAJOR: y is [cap_em,H] in the layout mep_to_expert_major or
 *                     mep_dispatch_standard_moe produced (needs one of them
 *                     after the current plan).
 * weights are token-major fp32 [T,k]; out is [T,H] bf16.  Tokens that were
 * not dispatched (bad expert id) produce +0.
 *   MEP_RANK_SUM:     y is [R,cap,H] rows written by mep_convert_combine_input
 *                     (each already weighted); out[t, h] = bf16_rne(acc),
 *                     acc = +0, then acc = acc + y_r[h] over t's distinct
 *                     destination ranks r in the order of their first top-k
 *                     position (one fp32 rounding per addition); weights is
 *                     not read and may be NULL.  Needs a valid plan.
 */
int mep_combine(mep_handle *h, int32_t layout, const void *y, const float *weights, void *out,
                void *stream);

/*
 * FP8 direct-cast combine payload ("MORI-EP User Guide", section 10 Tuning:
 * the intra-node tuning matrix pairs quant type fp8_direct_cast with a bf16
 * combine):
 * mep_cast_fp8_direct writes y8 = OCP E4M3 of each bf16 value of the rows the
 * current plan routes (round to nearest even, saturating at +-448, no scale;
 * NaN inputs are not supported), y and y8 in the layout of mep_combine with 1
 * byte per value (y8 is [R,cap,H] or [cap_em,H] bytes; other rows are not
 * touched).  mep_combine_fp8 is mep_combine on such E4M3 rows: each value is
 * decoded exactly to fp32 and accumulated as above.  Same state rules as
 * mep_combine.
 */
int mep_cast_fp8_direct(mep_handle *h, int32_t layout, const void *y, void *y8, void *stream);
int mep_combine_fp8(mep_handle *h, int32_t layout, const void *y8, const float *weights,
                    void *out, void *stream);

/*
 * The same payload rounding without the E4M3 rows (one device: source and
 * destination of the cast are the same): mep_combine on the bf16 rows y with
 * each value cast to E4M3 and decoded back before its multiply-add.  out is
 * bit for bit what mep_cast_fp8_direct followed by mep_combine_fp8 gives, the
 * bf16 rows being read once.  Same state rules and layouts as mep_combine.
 */
int mep_combine_fp8_direct(mep_handle *h, int32_t layout, const void *y, const float *weights,
                           void *out, void *stream);

/*
 * Standard-MoE expert outputs back to the combine input ("MORI-EP User
 * Guide" section 4, convert_combine_input(packed rows, source info, layout
 * range): the experts' expert-major outputs turned into the rows combine()
 * takes).  em_y is [cap_em,H] bf16 in the layout of the last
 * mep_to_expert_major (whose source info and segments this handle keeps);
 * recv_weights is the dispatch's [R,cap,k] fp32 output.  For every received
 * row (rank r, slot s < recv_counts[r]) of token t:
 *   y[r, s, h] = bf16_rne(acc), acc = +0, then for j = 0..k-1 in order, over
 *   t's positions whose expert lives on rank r and is not named by an earlier
 *   position: acc = fmaf(recv_weights[r, s, j], em_y[row of (t, j)][h], acc).
 * The pages pass no weights to this step; applying the dispatched weights
 * here is this library's reading -- a row merging several local experts can
 * carry their weighted sum only if the weights go in before the merge -- so
 * the combine that follows is mep_combine(MEP_RANK_SUM), which adds rank rows
 * without weights.  y is [R,cap,H] bf16; rows past recv_counts[r] are not
 * written; a position whose expert-major row was dropped (MEP_DEV_EM_OVERFLOW)
 * adds nothing.  Needs a valid plan and mep_to_expert_major after it.
 */
int mep_convert_combine_input(mep_handle *h, const void *em_y, const float *recv_weights,
                              void *y, void *stream);

/*
 * Reset between iterations ("MORI-EP User Guide" section 3 reset()):
 * invalidates the plan (and the expert-major maps) and starts a new status
 * epoch, whose status word the last plan already cleared on the device, so no
 * kernel is launched and `stream` is unused.  Caller buffers are not touched:
 * the library writes a caller buffer only during the call that names it.
 */
int mep_reset(mep_handle *h, void *stream);

/* Synchronise `stream`, then copy the device status word (MEP_DEV_* bits) to
 * *device_status.  Returns MEP_ERR_DEVICE if any bit is set, else MEP_OK. */
int mep_get_status(mep_handle *h, void *stream, int32_t *device_status);

/*
 * Inspection of the current plan (for verification, "MORI-EP User Guide"
 * section 3 get_dispatch_src_token_pos()): copies, on `stream`, the flat
 * receive row r*cap + slot of every (token, top-k position) into
 * recv_row[T,k] (int32, -1 for tokens not dispatched; needs a rank-major
 * plan), and/or the expert-major row of each (token, top-k position) into
 * em_row[T,k] (-1 where none; needs mep_to_expert_major or
 * mep_dispatch_standard_moe).  Either pointer may be NULL, not both.
 */
int mep_get_route(mep_handle *h, int32_t *recv_row, int32_t *em_row, void *stream);

/* ---- router ------------------------------------------------------------ */
#define MEP_FP32 0               /* logits and their gradient: fp32               */
#define MEP_BF16 1               /* logits and their gradient: bf16               */
#define MEP_SCORE_SOFTMAX 0      /* p = softmax of the logits                      */
#define MEP_SCORE_SIGMOID 1      /* s = 1 / (1 + exp(-x)), p = s / sum of s        */
#define MEP_GROUP_MAX 0          /* a group of experts counts by its best          */
#define MEP_GROUP_TOP2 1         /* by the sum of its two best                     */

typedef struct mep_gate_config {
  int32_t num_experts; /* E: 1..4096                                             */
  int32_t top_k;       /* k: 1..32, k <= E                                       */
  int32_t score;       /* MEP_SCORE_*                                            */
  int32_t dtype;       /* MEP_FP32 or MEP_BF16                                   */
  int32_t normalize;   /* not 0: a token's k weights are divided by their sum    */
  float scale;         /* factor of every weight                                 */
  float balance_coef;  /* coef of the balance loss                               */
} mep_gate_config;

/*
 * Router: the k experts of each token and their weights, in the form the plan,
 * dispatch and combine take them.  logits is [T,E]; per token,
 *   softmax: the k largest logits; v_j = exp(x_j - max) / sum over all experts
 *            of the same (p_j);
 *   sigmoid: the k largest s_e + bias[e] (bias fp32 [E]), in the order of their
 *            64-bit values, of which those of logits above about 37 are equal;
 *            without a bias (NULL) the k largest logits, which tell apart what
 *            64 bits do not; v_j = s_j, without the bias;
 *   weights[t, j] = scale * v_j, or scale * v_j / sum_j v_j when normalizing.
 * indices (int32) and weights (fp32) are [T,k], largest first; equal values go
 * to the lower expert.  All k experts of a token are different, whatever its
 * logits: NaN ranks last, and a selected NaN gives NaN weights, as does a logit of
 * +inf under softmax; where every v_j is 0 (logits of -inf, and sigmoids of logits
 * below -708) the weights are 0.  A sum of v_j too small for fp32 is divided by
 * all the same, here and in p and the gradients below.  0 <= T <= 2^26.
 * MEP_ERR_CONFIG for a bias with softmax scores.
 */
int mep_gate(const mep_gate_config *cfg, const void *logits, const float *bias, int32_t T,
             int32_t *indices, float *weights, void *stream);

/*
 * Router over groups of experts: as mep_gate, with the k experts taken from the
 * top_groups best of num_groups equal groups (group g: experts g*E/num_groups and
 * on).  With one group per rank a token goes to at most top_groups ranks.  A group's
 * score is, of the scores of its experts (softmax: p; sigmoid: s + bias),
 *   MEP_GROUP_MAX    the largest;
 *   MEP_GROUP_TOP2   the sum of the two largest (the largest where that is +inf).
 * Groups are chosen in the order of these scores' 64-bit values (MEP_GROUP_MAX
 * without a bias: in the logits' order), equal ones the lower first; a NaN among the
 * scores counts as -inf there, and under softmax a logit of +inf puts its group first (the
 * others then go by their scores without it).  Within the chosen groups everything is as
 * in mep_gate, and so is the gradient (mep_gate_backward).  num_groups: 1..64, divides E;
 * top_groups: 1..num_groups; k at most the chosen groups' experts; for MEP_GROUP_TOP2 two
 * experts a group at least (MEP_ERR_CONFIG otherwise).
 */
int mep_gate_grouped(const mep_gate_config *cfg, int32_t num_groups, int32_t top_groups,
                     int32_t group_score, const void *logits, const float *bias, int32_t T,
                     int32_t *indices, float *weights, void *stream);

/*
 * Load-balance loss of a batch and what it is made of.  With n the tokens that
 * count (token_mask[t] != 0, uint8 [T]; NULL: all T), over those tokens
 *   counts[e]    = number of (t, j) with indices[t, j] == e (int32; ids outside
 *                  [0, E) are left out); counts[E] = n;
 *   prob_mean[e] = (1/n) sum_t p[t, e] (fp32 [E]);
 *   loss[0]      = balance_coef * E / (k n) * sum_e counts[e] prob_mean[e].
 * All are 0 when n is 0.  Rows that do not count may hold anything, NaN
 * included.  Results do not depend on timing (no floating-point atomics).
 * workspace: at least mep_balance_workspace_bytes(cfg, T) bytes (0 if cfg or T is
 * invalid), zero-filled before its first use; it serves one call at a time and
 * is ready for the next when the call has run.  0 <= T <= 2^26,
 * T*k <= INT32_MAX.
 */
size_t mep_balance_workspace_bytes(const mep_gate_config *cfg, int32_t T);
int mep_balance_loss(const mep_gate_config *cfg, const void *logits, const int32_t *indices,
                     const uint8_t *token_mask, int32_t T, int32_t *counts, float *prob_mean,
                     float *loss, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradient of the router's weights (for fixed indices) and of the balance loss
 * with respect to the logits, in one pass:
 *   grad_logits = d( sum_tj grad_weights[t, j] weights[t, j]
 *                    + grad_loss[0] * loss ) / d logits, in the logits' type.
 * grad_weights (fp32 [T,k]) may be NULL: no gradient from the weights; counts
 * (as mep_balance_loss wrote it) and grad_loss (fp32, one value on the device)
 * may be NULL together: none from the loss.  Not both groups.  Counts are
 * constants of the differentiation.  Ids outside [0, E) have no weight and no
 * gradient; an expert a token names twice collects both.  A token that does not
 * count (token_mask) gets a row of zeros.  0 <= T <= 2^26.
 */
int mep_gate_backward(const mep_gate_config *cfg, const void *logits, const int32_t *indices,
                      const uint8_t *token_mask, int32_t T, const float *grad_weights,
                      const int32_t *counts, const float *grad_loss, void *grad_logits,
                      void *stream);

/* ---- experts' products ---------------------------------------------------- */
#define MEP_ACT_NONE 0
#define MEP_ACT_GELU 1           /* z/2 (1 + erf(z / sqrt 2))                      */
#define MEP_ACT_SILU 2           /* z / (1 + exp(-z))                              */
#define MEP_ACT_SILU_GLU 3       /* silu(z[:, :N]) * z[:, N:]                      */

typedef struct mep_linear_config {
  int32_t num_experts; /* E: 1..4096 segments                                    */
  int32_t in_dim;      /* K: multiple of 8, of 128 for E4M3; at most 2^20        */
  int32_t out_dim;     /* N, columns of y: likewise                              */
  int32_t act;         /* MEP_ACT_*; Nz, rows of a weight, is 2N for
                          MEP_ACT_SILU_GLU (gate rows, then the others) and N
                          otherwise                                              */
  int32_t quant;       /* MEP_QUANT_NONE: bf16 rows and weights;
                          MEP_QUANT_FP8_E4M3_BLOCK128: E4M3 rows with one scale per
                          128 columns, as the dispatch writes them, and E4M3
                          weights with one scale per 128 x 128                   */
} mep_linear_config;

/*
 * The experts' product over an expert-major buffer (mep_to_expert_major,
 * mep_dispatch_standard_moe): for every expert e and row r of its em_counts[e]
 * rows from em_offsets[e] on,
 *   z[r, :] = em_x[r, :] . w[e]^T + bias[e, :]      (fp32 accumulation)
 *   y[r, :] = bf16_rne(act(z[r, :]) + residual[r, :])
 * em_x is [cap_em,K], w [E,Nz,K], bias fp32 [E,Nz] or NULL, residual bf16
 * [cap_em,N] or NULL, y bf16 [cap_em,N]; z, bf16 [cap_em,Nz], receives the
 * product before the activation for mep_expert_linear_backward, or is NULL.
 * E4M3: em_scales fp32 [cap_em,K/128], w_scales fp32 [E,Nz/128,K/128]; a value
 * is code * scale (the matrix instruction adds 8 neighbouring E4M3 products to
 * within 7 * 2^-13 of the largest of them, and all else in fp32); both NULL for
 * bf16. Rows outside the segments' counts (padding, rows behind the last
 * segment) are neither used nor written, and rows past cap_em are left out.
 * em_offsets[e] must be multiples of 128, em_counts[e] >= 0 and segments must
 * not overlap, as the calls above write them; their order is free, and
 * em_offsets[E] is not read. One segment over a whole batch (E = 1) is an
 * ordinary dense layer. num_rows is the number of rows to expect in all segments
 * together (T*k): it selects among kernels and sizes the launch; results are
 * complete for any value. 0 <= cap_em <= INT32_MAX. y and z overlap no input,
 * but y may be residual itself.
 */
int mep_expert_linear(const mep_linear_config *cfg, const void *em_x, const float *em_scales,
                      const int32_t *em_counts, const int32_t *em_offsets, int64_t cap_em,
                      int64_t num_rows, const void *w, const float *w_scales, const float *bias,
                      const void *residual, void *y, void *z, void *stream);

/*
 * Gradients of mep_expert_linear (bf16 only).  With grad_z = grad_y * act'(z)
 * (grad_y itself without an activation), per expert over its rows
 *   grad_x[r, :]    = grad_z[r, :] . w[e]           (bf16 [cap_em,K])
 *   grad_w[e]       = grad_z^T . em_x               (bf16 [E,Nz,K])
 *   grad_bias[e, :] = sum over rows of grad_z       (fp32 [E,Nz])
 * each NULL when not wanted, not all three.  z is the forward call's (NULL
 * allowed without an activation).  The residual's gradient is grad_y.  Rows of
 * grad_x outside the segments are not written; an expert without rows has zeros
 * in grad_w and grad_bias.  grad_z is rounded to bf16 for the two products, not
 * for grad_bias.  workspace: mep_linear_workspace_bytes(cfg, cap_em) bytes (0 if cfg
 * or cap_em is invalid), of any content; it serves one call at a time.
 * num_rows as above.  No output may overlap an input.
 */
size_t mep_linear_workspace_bytes(const mep_linear_config *cfg, int64_t cap_em);
int mep_expert_linear_backward(const mep_linear_config *cfg, const void *grad_y, const void *z,
                               const void *em_x, const void *w, const int32_t *em_counts,
                               const int32_t *em_offsets, int64_t cap_em, int64_t num_rows,
                               void *grad_x, void *grad_w, float *grad_bias, void *workspace,
                               size_t workspace_bytes, void *stream);

/* ---- norms around a block ------------------------------------------------- */
#define MEP_NORM_NONE 0          /* hat(u) = u                                     */
#define MEP_NORM_RMS 1           /* hat(u) = u / sqrt(mean u^2 + eps)              */
#define MEP_NORM_LAYER 2         /* hat(u) = (u - mean u) / sqrt(var u + eps)      */
#define MEP_BLOCK_GATE_NONE 0
#define MEP_BLOCK_GATE_TOKEN 1   /* fp32 [T]: one factor a row                     */
#define MEP_BLOCK_GATE_ELEMENT 2 /* [T,H] in the rows' type                        */

typedef struct mep_norm_config {
  int32_t hidden_dim;   /* H: multiple of 8 up to 16384, of 128 where codes are made */
  int32_t dtype;        /* MEP_FP32 or MEP_BF16: every [T,H] tensor                  */
  int32_t post;         /* MEP_NORM_* of the block's output                          */
  int32_t pre;          /* MEP_NORM_* of the new stream, the next block's input      */
  int32_t gate;         /* MEP_BLOCK_GATE_*                                          */
  int32_t gate_sigmoid; /* not 0: the gate's factor is 1 / (1 + exp(-gate))          */
  float eps;            /* > 0                                                       */
  float weight_offset;  /* o: a weight w stands for the factor o + w                 */
  float residual_scale; /* a                                                         */
  float block_scale;    /* c                                                         */
} mep_norm_config;

/*
 * What stands between two blocks, in one pass over the rows.  With x [T,H] the stream
 * before a block, y [T,H] the block's output (mep_combine's, say) and g the gate's
 * factor of a row or element (1 without a gate), per row
 *   v = hat_post(y) (o + post_weight) + post_bias
 *   s = a x + c g v
 *   n = hat_pre(s) (o + pre_weight) + pre_bias
 * in fp32, s and n rounded once each to the rows' type (n is of s before its rounding).
 * s is the new stream; n the next block's input, for its router and, as E4M3 codes with
 * a scale per 128 columns, for a dispatch with MEP_QUANT_FP8_CARRY:
 *   n_scales[t, b] = amax_b / 448 (fp32 [T,H/128]),  n_codes = E4M3_rne(n * (1 / scale))
 * of n before its rounding, the reciprocal and the product rounded to fp32's bits, n held
 * within +-448 scales (a scale of few bits may be less than amax_b / 448).  (Zeros where
 * the scale is 0; a NaN counts for no maximum and stays one; a block with an infinity in it
 * is NaN throughout, its scale being infinite.)  s, n and n_codes are NULL where not wanted,
 * not all three.  x NULL: no residual; y NULL: no block part (gate then NULL too, whatever
 * cfg->gate is), so that the call norms or only encodes rows; not both NULL.  Weights and
 * biases are fp32 [H]; a NULL weight stands for the factor 1, a NULL bias for 0.  Of a row
 * that is normed the sum of the squares must fit fp32 (of 4096 equal values: up to 2.8e17
 * each); past that the norm gives 0 or NaN.  s may be x or y itself and n may be y itself
 * (not both y); other outputs overlap nothing.
 * 0 <= T <= 2^26.
 */
int mep_block_norm(const mep_norm_config *cfg, const void *x, const void *y, const void *gate,
                   const float *post_weight, const float *post_bias, const float *pre_weight,
                   const float *pre_bias, int32_t T, void *s, void *n, void *n_codes,
                   float *n_scales, void *stream);

/*
 * Gradients of mep_block_norm from those of s and n (either may be NULL: none, not
 * both; codes pass n's through).  s is the forward call's, needed with grad_n; y and
 * gate as there.  With gs = grad_s + what hat_pre hands back of grad_n (o + pre_weight),
 *   grad_x = a gs                                       ([T,H])
 *   grad_y = what hat_post hands back of c g gs (o + post_weight)   ([T,H])
 *   grad_gate = c gs v (summed over a row for a factor a row), times the sigmoid's
 *               slope                                   (as gate)
 *   grad_post_weight = sum_t c g gs hat_post(y),   grad_post_bias = sum_t c g gs,
 *   grad_pre_weight = sum_t grad_n hat_pre(s),     grad_pre_bias = sum_t grad_n
 * (fp32 [H]); each NULL when not wanted, not all seven, and the block's four only with
 * y, the pre norm's two only with grad_n.  hat_pre is taken at s as it is given.
 * Results do not depend on timing.  workspace: mep_block_norm_workspace_bytes(cfg, T)
 * bytes (0 if cfg or T is invalid), of any content; it serves one call at a time.
 * grad_x may be grad_s itself and grad_y may be y itself; other outputs overlap
 * nothing.  0 <= T <= 2^26; the sums over no rows are 0.  Every row counts in the column
 * sums: padding among the T rows has to be finite and its gradients 0.
 */
size_t mep_block_norm_workspace_bytes(const mep_norm_config *cfg, int32_t T);
int mep_block_norm_backward(const mep_norm_config *cfg, const void *grad_s, const void *grad_n,
                            const void *s, const void *y, const void *gate,
                            const float *post_weight, const float *post_bias,
                            const float *pre_weight, int32_t T, void *grad_x, void *grad_y,
                            void *grad_gate, float *grad_post_weight, float *grad_post_bias,
                            float *grad_pre_weight, float *grad_pre_bias, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ---- gradients of many tensors --------------------------------------------- */
typedef struct mep_grad {
  const void *data; /* the gradient, dense                                           */
  void *out;        /* where mep_grad_clip puts it: data itself or a buffer of its own */
  int64_t numel;    /* >= 0; 0: pointers may be NULL                                 */
  int32_t dtype;    /* MEP_FP32 or MEP_BF16, of both                                 */
  int32_t reserved; /* 0                                                             */
} mep_grad;

/*
 * The norm of n gradients together, norm[0] = sqrt(sum of all values squared) (fp32, on
 * the device; summed in fp64, so it neither overflows nor vanishes before its rounding;
 * inf and NaN come through).  grads is a host array, read during the call.  n >= 0, at
 * most 65536.  workspace: mep_grad_workspace_bytes(grads, n) bytes (0 if grads or n is
 * invalid), of any content; it serves one call at a time.  `out` is not used.  Does not
 * depend on timing.
 */
size_t mep_grad_workspace_bytes(const mep_grad *grads, int32_t n);
int mep_grad_norm(const mep_grad *grads, int32_t n, float *norm, void *workspace,
                  size_t workspace_bytes, void *stream);

/*
 * Clipping: out = data * min(1, max_norm / (norm[0] + 1e-6)) for each of n gradients,
 * rounded to its type; norm is mep_grad_norm's, or several ranks' put together.  Where
 * the factor is 1, tensors that are their own `out` are not touched.  A NaN norm gives
 * NaN, an infinite one 0 (NaN where the gradient is not finite).  max_norm > 0; infinite: no
 * limit, the factor is 1 for every norm but NaN.
 * Outputs overlap neither each other nor other inputs.
 */
int mep_grad_clip(const mep_grad *grads, int32_t n, const float *norm, float max_norm,
                  void *stream);

/*
 * Codec probes: run, over n values, exactly the device conversions the
 * kernels use.  in is fp32 [n]; mep_probe_e4m3 writes OCP E4M3 codes (uint8
 * [n]) of in[i] (no scaling; values must satisfy |v| <= 464), mep_probe_bf16
 * writes bf16 round-to-nearest-even bits (uint16 [n]).
 */
int mep_probe_e4m3(const float *in, uint8_t *out, int64_t n, void *stream);
int mep_probe_bf16(const float *in, uint16_t *out, int64_t n, void *stream);

/*
 * FP8 block probe: the dispatch's MEP_QUANT_FP8_E4M3_BLOCK128 block encoder
 * over nblocks blocks of 128 bf16 values (in: uint16 bit patterns
 * [nblocks,128], finite values only), writing each block's 128 E4M3 codes (q:
 * uint8 [nblocks,128]) and its fp32 scale (scales [nblocks]).  in and q
 * 16-byte aligned, scales 4-byte aligned; nblocks <= 2^28.
 */
int mep_probe_fp8_block(const uint16_t *in, uint8_t *q, float *scales, int64_t nblocks,
                        void *stream);

/*
 * MX FP4 block probe: the dispatch's MEP_QUANT_MXFP4 block encoder over
 * nblocks blocks of 32 bf16 values (in: uint16 bit patterns [nblocks,32],
 * finite values only), writing each block's 16 packed E2M1 code bytes (q:
 * uint8 [nblocks,16], even column in the low nibble) and its E8M0 scale byte
 * (e8: uint8 [nblocks]).  in and q 16-byte aligned; nblocks <= 2^32.
 */
int mep_probe_mxfp4(const uint16_t *in, uint8_t *q, uint8_t *e8, int64_t nblocks, void *stream);

/*
 * Streaming probe (measurement, not part of the path): what HBM gives a mix of
 * reads and writes spread over a number of waves, for comparing a kernel with
 * plain streams of its own byte mix.  `waves` 64-lane waves share rd_units
 * reads of src and wr_units writes of dst, each unit 1 KiB (16 bytes per
 * lane), as evenly as the counts allow; each wave's share of src and of dst is
 * one contiguous run, its loads are non-temporal and all issued before its
 * non-temporal stores.  src holds rd_units KiB and dst wr_units KiB (at least
 * 16 bytes when wr_units is 0: a never-taken store keeps read-only waves'
 * loads live).  MEP_ERR_SHAPE when a wave would take more than 16 read units,
 * for more than 2^24 waves or more than 2^30 units.  The values written are
 * unspecified.
 */
int mep_probe_stream(const void *src, void *dst, int64_t waves, int64_t rd_units,
                     int64_t wr_units, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MEP_H */
