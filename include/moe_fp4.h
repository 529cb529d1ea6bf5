/*
 * moe_fp4: one block-scaled Mixture-of-Experts layer forward on an AMD MI355X
 * (gfx950), as a C ABI.
 *
 * What is computed (MegaMoE post, flashinfer.ai, "The problem" and "Our
 * approach"; FlashInfer PR #4366, "Description"; newruntime summary of
 * FlashInfer PR #5319, "Retrieval answer"):
 *
 *   S1 route     per token, the top-K of E router logits (descending, ties to
 *                the lower expert id) and weights p = softmax over the chosen K;
 *   S2 permute   routes r = t*K + k grouped by expert, tokens ascending inside a
 *                group (expert-contiguous grouped-GEMM order);
 *   S3 quantize  FC1 input: NVFP4 (E2M1 values, E4M3 scale per 16 elements,
 *                FP32 global scale per tensor or per token), MXFP8 (E4M3 values,
 *                E8M0 scale per 32) or none (W4A16: bf16 activations);
 *   S4 FC1       grouped GEMM h = x W1_e^T per route;
 *   S5           SwiGLU (silu(gate) * up) or ReLU2 (max(h,0)^2); with input-side
 *                placement the result is multiplied by p in FP32; then the FC2
 *                input is quantized (W4A4: NVFP4 per tensor or per route; MXFP8)
 *                or stored as bf16 (W4A16);
 *   S6 FC2       grouped GEMM o = a W2_e^T per route;
 *   S7 finalize  y[t] = sum_k w[t,k] o[route t*K+k] with w = p (output side) or
 *                1 (input side, the weight was applied before FC2), in fixed k
 *                order, either as its own kernel (deterministic) or fused into
 *                FC2 (the FC2 block completing a token's K routes for its
 *                columns reduces them; the same bits).
 *
 * Conventions for every entry point:
 *  - Tensor pointers are device pointers (hipMalloc'd or equivalent), row-major,
 *    owned by the caller. The library never allocates device or host memory
 *    and keeps no per-call state, except the optional stage timing below.
 *  - Every call only enqueues work on `stream` and returns; no host<->device
 *    synchronisation except in moe_check_prepared, moe_forward_status and
 *    moe_stage_times (and in moe_forward while stage timing is on, see
 *    moe_stage_timing).
 *  - Argument checks all run before any launch; on failure nothing is
 *    enqueued and a moe_status other than MOE_OK is returned, with a message in
 *    moe_last_error().
 *  - Device pointers must be 256-byte aligned where noted, else 16-byte aligned.
 */
#ifndef MOE_FP4_H
#define MOE_FP4_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_W4A4_TENSOR = 0, /* NVFP4 weights and activations, one activation global scale per tensor */
    MOE_W4A4_TOKEN = 1,  /* NVFP4 weights and activations, one activation global scale per row    */
    MOE_W4A16 = 2,       /* NVFP4 weights, bf16 activations                                         */
    MOE_MXFP8 = 3,       /* MXFP8 (E4M3 + E8M0 per 32) weights and activations                      */
    /* NVFP4 weights; activations per token under the "4-over-6" contract
     * (FlashInfer PR #4366, "Performance benchmark", named there by its
     * switches only; this library's reading): global scale amax / (6*256) per
     * row, and per 16-block the block max mapped to 6 or to 4, whichever gives
     * the smaller sum of squared errors (fp64, element order; ties to 6). The
     * GEMMs consume the result like any NVFP4 operand. */
    MOE_W4A4_TOKEN_4O6 = 4,
    /* NVFP4 W4A4 with per-token activation scales, GEMMs on the block-scaled
     * FP4 matrix cores: both operands re-blocked from NVFP4 (E4M3 per 16) to
     * MXFP4 (E8M0 per 32) by the OCP MX rule, which rounds each element a second
     * time (about 11-12 % relative Frobenius difference per GEMM operand against
     * the NVFP4 values); the FP32 global scales are applied in the epilogues.
     * Opt-in, for callers that accept that error; needs an MOE_FMT_MXFP4 blob. */
    MOE_W4A4_TOKEN_MXFP4 = 5
} moe_mode;

typedef enum { MOE_ACT_SWIGLU = 0, MOE_ACT_RELU2 = 1 } moe_act;
/* MOE_FMT_MXFP4: the weights NVFP4-quantized (per-expert FP32 global scale)
 * and re-blocked to MXFP4, in the FP4 matrix-core layout (mode 5 only). */
typedef enum { MOE_FMT_NVFP4 = 0, MOE_FMT_MXFP8 = 1, MOE_FMT_MXFP4 = 2 } moe_wfmt;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID = 1,     /* null/misaligned pointer, bad size or enum                  */
    MOE_ERR_UNSUPPORTED = 2, /* well-formed but not implemented (e.g. H % 128 != 0)       */
    MOE_ERR_WORKSPACE = 3,   /* workspace or prepared buffer too small                      */
    MOE_ERR_HIP = 4          /* a HIP call failed; moe_last_error() has hipGetErrorString */
} moe_status;

/* Layer geometry. N1 = 2*I for SwiGLU (rows [0,I) gate, [I,2I) up), I for
 * ReLU2. Limits: 1 <= E <= 1024; H and I positive multiples of 128 (the K
 * extent of one weight micro-tile); H, I <= 32768. */
typedef struct {
    int32_t E, H, I;
    int32_t act;  /* moe_act  */
    int32_t wfmt; /* moe_wfmt */
} moe_dims;

/* Size in bytes of the prepared-weight blob for `d` (0 if `d` is invalid). */
size_t moe_prepared_bytes(const moe_dims* d);

/* S0 (off the timed path): quantize and reorder the weights.
 * Weights arrive in the standard checkpoint layout and the library quantizes
 * and reorders them itself (MegaMoE post, "Usage"); one NVFP4 blob serves the
 * W4A4 and W4A16 modes (newruntime summary of PR #5319, title).
 *   w1: [E][N1][H] fp32, w2: [E][H][I] fp32 (device).
 *   prepared: device buffer of at least moe_prepared_bytes(d) bytes, 256-byte
 *   aligned; written entirely (header, per-expert FP32 global scales
 *   g = amax / (6*448) per expert per matrix for NVFP4, codes and scales in the
 *   kernel-native layout described in the design notes). Immutable afterwards;
 *   it may be shared by concurrent forwards. */
int moe_prepare_weights(const moe_dims* d, const float* w1, const float* w2, void* prepared,
                        size_t prepared_bytes, hipStream_t stream);

/* Synchronous check that a device blob's header matches `d` (reads 256 bytes
 * to the host; not for use under graph capture). */
int moe_check_prepared(const moe_dims* d, const void* prepared, hipStream_t stream);

/* Workspace bytes needed by moe_forward for up to T_max tokens and top-K. */
size_t moe_workspace_bytes(const moe_dims* d, int32_t T_max, int32_t K, int32_t mode);

/* S1..S7: one layer forward.
 *   prepared: blob from moe_prepare_weights with the same `d` (NVFP4 blob for
 *             modes 0..2, MXFP8 blob for mode 3), prepared_bytes its size in
 *             bytes (MOE_ERR_WORKSPACE below moe_prepared_bytes(d)). The blob's
 *             header is compared with `d` on the device by the forward's first
 *             kernel: on a difference (a blob prepared for other dimensions,
 *             activation or format) the forward reads no weights, leaves y
 *             unwritten and sets its status word to MOE_ERR_INVALID, which
 *             moe_forward_status returns.
 *   x:        [T][H] bf16 bit patterns.            logits: [T][E] fp32 (finite).
 *   T >= 1, 1 <= K <= min(E, 64), T*K*max(H, I)*2 < 4 GiB (MOE_ERR_UNSUPPORTED
 *   otherwise: the GEMMs address activation rows with 32-bit offsets).
 *   act must equal d->act. router_weight_on_input: 0 = output side (finalize
 *   weights p), 1 = input side (p applied to the FP32 activation output before
 *   the FC2-input quantization or bf16 store; finalize weights 1).
 *   deterministic_finalize: 1 = FC2 stores the permuted output O in fp32, then
 *   a fixed-order unpermute+reduce in fp32 (bit-identical run to run);
 *   0 = the finalize fused into the FC2 kernel: the FC2 block that completes
 *   a token's K routes for its output columns reduces them, in the same order
 *   and arithmetic, so the output is the same bits as with 1.
 *   MXFP8 quantizes the FC2 input in the FC1 epilogue (no fp32 copy).
 *   workspace: >= moe_workspace_bytes(d, T, K, mode) bytes, 256-byte aligned;
 *   afterwards it holds the forward's status word (first 4 bytes) and the
 *   intermediate views listed by moe_workspace_view.
 *   y: [T][H] bf16 bit patterns (output). */
int moe_forward(const moe_dims* d, const void* prepared, size_t prepared_bytes, const uint16_t* x,
                const float* logits, int32_t T, int32_t K, int32_t mode, int32_t act,
                int32_t router_weight_on_input, int32_t deterministic_finalize, void* workspace,
                size_t workspace_bytes, uint16_t* y, hipStream_t stream);

/* moe_forward for callers that cannot allocate: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc. The same forward, on a
 * workspace that is a device array inside the library (64 MiB; each GPU the
 * library runs on holds its own copy until the process ends) instead of a
 * caller buffer; the caller still passes the inputs and y. Arguments, their
 * checks and error codes as for moe_forward; a shape whose workspace
 * (moe_workspace_bytes) exceeds 64 MiB returns MOE_ERR_WORKSPACE before any
 * launch. No call allocates memory; the first call on a device looks up the
 * array's device address (hipGetSymbolAddress) with that device current, so
 * `stream` must belong to the current device. All calls on one GPU share the
 * array, which keeps the last call's contents (every forward rewrites what it
 * reads): forwards that overlap in time on one GPU, on different streams or
 * host threads, race and must be serialised by the caller. The status word
 * of the device-side blob check lives in that array and is not readable. */
int moe_forward_noalloc(const moe_dims* d, const void* prepared, size_t prepared_bytes,
                        const uint16_t* x, const float* logits, int32_t T, int32_t K,
                        int32_t mode, int32_t act, int32_t router_weight_on_input,
                        int32_t deterministic_finalize, uint16_t* y, hipStream_t stream);

/* Status word of the last forward enqueued on `workspace` (synchronous: waits
 * for `stream`, then reads 4 bytes): *status = 0 after a forward whose blob
 * header matched its dimensions, MOE_ERR_INVALID otherwise (y was then not
 * written). Not for use under graph capture. */
int moe_forward_status(const void* workspace, int32_t* status, hipStream_t stream);

/* S7 alone (unfused finalize, as in PR #5319): y[t][j] = sum_{k<K} w[t][k] *
 * permuted_out[route_to_row[t*K+k]][j], accumulated in fp32 in k order and
 * rounded once to bf16. Always the fixed-order (deterministic) reduction: the
 * fused variant exists only inside moe_forward, where it is the FC2
 * epilogue's scatter-add.
 *   permuted_out: [R][H] fp32 (out_is_bf16 = 0) or bf16 (1), R = T*K.
 *   route_to_row: [T*K] int32, each in [0, R).  weights: [T][K] fp32 or NULL
 *   for unit weights (input-side placement).  y: [T][H] bf16. */
int moe_finalize(const void* permuted_out, int32_t out_is_bf16, const int32_t* route_to_row,
                 const float* weights, int32_t T, int32_t K, int32_t H, uint16_t* y,
                 hipStream_t stream);

/* Standalone block quantizer (the S3/S5 quantizer as a library call).
 *   v: [rows][cols] fp32; kind: 0 = NVFP4 one global scale for the whole
 *   matrix, 1 = NVFP4 one global scale per row, 2 = MXFP8, 3 = NVFP4 per row
 *   with the 4-over-6 block choice (see MOE_W4A4_TOKEN_4O6).
 *   codes: NVFP4 [rows][cols/2] (two E2M1 codes per byte, even element in the
 *   low nibble); MXFP8 [rows][cols] E4M3.  scales: NVFP4 [rows][cols/16] E4M3;
 *   MXFP8 [rows][cols/32] E8M0.  g: NVFP4 [1] or [rows] fp32 (unused for MXFP8).
 *   scratch: 256 bytes of device memory (cleared by the call).
 *   cols % 32 == 0. */
int moe_quantize(const float* v, int32_t rows, int32_t cols, int32_t kind, uint8_t* codes,
                 uint8_t* scales, float* g, void* scratch, hipStream_t stream);

/* Location of an intermediate inside the workspace (for inspection/parity):
 *   0 topk_ids [T][K] i32        1 topk_w [T][K] f32
 *   2 counts [E] i32             3 offsets [E+1] i32
 *   4 row_to_route [R] i32       5 route_to_row [R] i32
 *   6 x codes                    7 x scales               8 x global scale(s) f32
 *   9 FC2 input, fp32 before quantization [R][I] (W4A4) or bf16 (W4A16)
 *   10 FC2-input codes           11 FC2-input scales      12 FC2-input global scale(s)
 *   13 permuted FC2 output O [R][H] f32 (either finalize)
 *   14/15 x re-blocked to MXFP4: codes [T][H/2], E8M0 scales [T][H/32] (mode 5)
 *   16/17 FC2 input re-blocked to MXFP4: codes [R][I/2], scales [R][I/32] (mode 5)
 * Returns MOE_ERR_INVALID for a view the mode does not produce. */
int moe_workspace_view(const moe_dims* d, int32_t T, int32_t K, int32_t mode, int32_t view_id,
                       size_t* offset, size_t* bytes);

/* Optional per-stage timing with HIP events recorded on the forward's stream
 * around each stage (not to be enabled under graph capture). While it is on,
 * forwards take a process-wide lock for their launches (forwards from several
 * host threads serialise), and a forward waits for the events of the oldest
 * of the last 128 timed forwards before reusing them. moe_stage_times
 * synchronises, returns the summed milliseconds per stage since the last
 * reset in ms[0..n) and the number of timed forwards, and resets. Stage ids:
 * 0 route, 1 permute, 2 quantize x, 3 FC1, 4 FC2-input quantize, 5 FC2,
 * 6 finalize. */
int moe_stage_timing(int32_t enable);
int moe_stage_times(float* ms, int32_t n, int32_t* forwards);

/* -------------------------------------------------------------------------
 * Operators around the experts, each as a call of its own
 * -------------------------------------------------------------------------
 * The routes of T tokens with K experts each (route r = t*K + k) sorted by
 * expert, token rows dispatched to the experts' rows and combined back with
 * the router's weights, the gradients of both, and products of 8-bit integer
 * matrices with a scale for each token and each output channel.
 *
 * Row strides are in elements; the elements of a row are contiguous. Pointers
 * are aligned to their element unless noted. Outputs must not share bytes with
 * inputs or with each other (MOE_ERR_INVALID; columns of one matrix that lie apart
 * are fine). T = 0 (or no rows) is valid and
 * only writes what does not depend on rows. Nothing is kept between calls, so
 * calls on different streams are independent as long as their buffers are. */
typedef enum { MOE_DT_BF16 = 0, MOE_DT_FP16 = 1, MOE_DT_FP32 = 2 } moe_dtype;

/* Workspace bytes of moe_sort_routes for up to T tokens (0 if the sizes are
 * invalid). */
size_t moe_sort_workspace_bytes(int32_t T, int32_t K, int32_t E);

/* Stable sort of the routes by expert.
 *   ids: [T][K] expert ids, int32 (ids_are_wide = 0) or int64 (1). An id
 *   outside [0, E) drops its route (an expert of another GPU, a token that is
 *   not to be routed); the same expert may appear twice in a token.
 *   row_to_route: [T*K] route of each row; routes of expert e fill the rows
 *   offsets[e] .. offsets[e+1]-1 in ascending order; -1 in the rows from
 *   offsets[E] on.   route_to_row: [T*K] the row of each route, -1 if dropped.
 *   offsets: [E+1].   workspace: >= moe_sort_workspace_bytes(T, K, E) bytes,
 *   16-byte aligned.   1 <= E <= 1024, 1 <= K <= 64, T*K <= 2^23. */
int moe_sort_routes(const void* ids, int32_t ids_are_wide, int32_t T, int32_t K, int32_t E,
                    void* workspace, size_t workspace_bytes, int32_t* row_to_route,
                    int32_t* route_to_row, int32_t* offsets, hipStream_t stream);

/* rows[route_to_row[t*K+k]] = w[t,k] * x[t] for every route that is kept.
 *   x: [T][H], rows: [T*K][H], both of type `dtype` (moe_dtype). weights:
 *   [T][K] fp32, or NULL for 1 (the rows are then copies, bit for bit). Rows
 *   that no route names are left as they were. An entry of route_to_row outside
 *   [0, T*K) counts as dropped. 1 <= H <= 2^20, T*K <= 2^23. x_stride may be
 *   anything from 0 (one row for all tokens) on. */
int moe_dispatch(const void* x, int64_t x_stride, int32_t dtype, const int32_t* route_to_row,
                 const float* weights, int32_t T, int32_t K, int32_t H, void* rows,
                 int64_t rows_stride, hipStream_t stream);

/* Gradients of moe_dispatch from the gradient of its rows:
 *   dx[t] = sum_k w[t,k] drows[row(t,k)]   (fp32 sums, k ascending, one rounding)
 *   dweights[t,k] = <x[t], drows[row(t,k)]>   (fp32; 0 for a dropped route)
 *   dweights may be NULL (x is then not read, and may be NULL); it needs weights. */
int moe_dispatch_grad(const void* drows, int64_t drows_stride, int32_t dtype,
                      const int32_t* route_to_row, const float* weights, const void* x,
                      int64_t x_stride, int32_t T, int32_t K, int32_t H, void* dx,
                      int64_t dx_stride, float* dweights, hipStream_t stream);

/* y[t] = sum_k w[t,k] rows[route_to_row[t*K+k]]: fp32 sums, k ascending, one
 * rounding to `dtype`; dropped routes are skipped (their rows, whatever they
 * hold, are not read), a token without routes gets zeros. Like moe_finalize, for
 * sorted routes with drops, every moe_dtype and strided rows. */
int moe_combine(const void* rows, int64_t rows_stride, int32_t dtype, const int32_t* route_to_row,
                const float* weights, int32_t T, int32_t K, int32_t H, void* y, int64_t y_stride,
                hipStream_t stream);

/* Gradients of moe_combine from dy: [T][H]:
 *   drows[row(t,k)] = w[t,k] dy[t]; rows that no route names are left as they were
 *   dweights[t,k] = <dy[t], rows[row(t,k)]>; may be NULL (rows is then not read). */
int moe_combine_grad(const void* dy, int64_t dy_stride, int32_t dtype, const int32_t* route_to_row,
                     const float* weights, const void* rows, int64_t rows_stride, int32_t T,
                     int32_t K, int32_t H, void* drows, int64_t drows_stride, float* dweights,
                     hipStream_t stream);

/* Symmetric 8-bit quantization of each row: scales[m] = max_j |x[m,j]| / 127 in
 * fp32, codes[m,j] = x[m,j] / scales[m] rounded to the nearest integer, ties to
 * even (the exact quotient of the fp32 scale, so the codes are reproducible bit
 * for bit), in [-127, 127]. A zero row has scale 0 and codes 0, and so has one whose
 * scale rounds to 0 (its largest value is below 64 * 2^-149); a row with an
 * infinity or a NaN has that as its scale and codes 0 (products with it are NaN).
 *   x: [rows][cols] of type dtype, codes: [rows][cols].  1 <= cols <= 2^20,
 *   rows <= 2^23. */
int moe_int_quantize(const void* x, int64_t x_stride, int32_t dtype, int32_t rows, int32_t cols,
                     int8_t* codes, int64_t codes_stride, float* scales, hipStream_t stream);

/* y[m,n] = a_scales[m] b_scales[n] sum_k a[m,k] b[n,k] + bias[n]: exact 32-bit
 * integer sums, scales and bias in fp32, one rounding to out_dtype (moe_dtype).
 *   a: [M][K], b: [N][K] int8, 16-byte aligned with strides that are multiples
 *   of 16; bias: [N] fp32 or NULL; y: [M][N].  K a multiple of 16 below 131072
 *   (MOE_ERR_UNSUPPORTED otherwise, as for strides of a and b above 2^23, N above
 *   2^20 and M above 2^23). */
int moe_int_matmul(const int8_t* a, int64_t a_stride, const float* a_scales, const int8_t* b,
                   int64_t b_stride, const float* b_scales, const float* bias, int32_t M, int32_t N,
                   int32_t K, int32_t out_dtype, void* y, int64_t y_stride, hipStream_t stream);

/* The same product expert by expert on sorted rows: the rows offsets[e] ..
 * offsets[e+1]-1 of y use b[e] ([E][N][K], experts b_expert_stride bytes
 * apart: a multiple of 16 from 0, one matrix for all, to 2^48), b_scales[e] ([E][N])
 * and bias[e] ([E][N] or NULL). Rows of y outside the offsets are left as they were.
 *   row_to_route NULL: row r of y uses row r of a (a_rows = M).
 *   Otherwise row r uses row row_to_route[r] / topk of a, the token's (a_rows =
 *   M / topk tokens, below 4 GiB): FC1 needs no dispatched copy. Rows whose
 *   entry names no token are left as they were. */
int moe_int_grouped_matmul(const int8_t* a, int64_t a_stride, const float* a_scales, int32_t a_rows,
                           const int8_t* b, int64_t b_stride, int64_t b_expert_stride,
                           const float* b_scales, const float* bias, const int32_t* offsets,
                           const int32_t* row_to_route, int32_t topk, int32_t M, int32_t N,
                           int32_t K, int32_t E, int32_t out_dtype, void* y, int64_t y_stride,
                           hipStream_t stream);

/* -------------------------------------------------------------------------
 * Operators in front of, between and beside the experts' products
 * -------------------------------------------------------------------------
 * Under the same conventions: strides in elements, contiguous rows, any stride from 0
 * on for an input's rows, outputs apart from inputs and from each other. */

/* Root-mean-square norm of each row, with the residual's addition before it:
 *   h = x + residual, rounded to `dtype` and stored in total (x itself where
 *   residual is NULL; the two come together);
 *   r = 1 / sqrt(mean_j h_j^2 + eps);   y_j = h_j r weight_j, rounded once.
 * The norm reads h as it is stored. 8-bit output (codes and scales come together,
 * beside y or instead of it; for moe_int_matmul): p_j = h_j weight_j rounded to fp32,
 * s = max_j |p_j| / 127 in fp32, codes[j] = p_j / s as moe_int_quantize rounds it,
 * scales = s r. So the codes do not depend on r and are reproducible bit for bit. A row
 * whose p has an infinity or a NaN has codes 0 and a scale that is not finite.
 *   x, residual, total, y: [rows][cols] of type dtype; weight: [cols] of type
 *   weight_dtype (dtype or fp32), or NULL for ones. total may be residual itself
 *   (same address and stride). 1 <= cols <= 32768, rows <= 2^23, eps >= 0 (a zero
 *   row with eps = 0 is NaN). */
int moe_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                 int32_t dtype, const void* weight, int32_t weight_dtype, int32_t rows,
                 int32_t cols, float eps, void* total, int64_t total_stride, void* y,
                 int64_t y_stride, int8_t* codes, int64_t codes_stride, float* scales,
                 hipStream_t stream);

/* Workspace bytes of moe_rms_norm_grad with dweight (0 if the sizes are invalid). */
size_t moe_rms_norm_grad_workspace_bytes(int32_t rows, int32_t cols);

/* Gradients of moe_rms_norm from dy, the gradient of y, and h (x, or total): with
 * n = h r, g = dy weight
 *   dx = r (g - n mean_j(g n)) + dtotal    (also the residual's gradient; dtotal: the
 *                                           gradient of total, or NULL)
 *   dweight = sum over the rows of dy n    (fp32, rows in a fixed order; or NULL)
 *   workspace: >= moe_rms_norm_grad_workspace_bytes(rows, cols) bytes, 16-byte
 *   aligned; may be NULL without dweight. */
int moe_rms_norm_grad(const void* dy, int64_t dy_stride, const void* h, int64_t h_stride,
                      int32_t dtype, const void* weight, int32_t weight_dtype, const void* dtotal,
                      int64_t dtotal_stride, int32_t rows, int32_t cols, float eps, void* workspace,
                      size_t workspace_bytes, void* dx, int64_t dx_stride, float* dweight,
                      hipStream_t stream);

/* The activation between an expert's two products, on sorted rows (moe_act):
 *   swiglu: a_j = silu(h_j) h_{I+j}, h: [rows][2I];  relu2: a_j = max(h_j, 0)^2, h: [rows][I]
 *   out[m][j] = w a_j, in fp32 and rounded once to dtype, with w = weights[row_to_route[m]] (the
 *   router's weight on the input side of the second product), 1 where weights is NULL.
 *   offsets ([E+1]): only the rows below offsets[E] are read and written; NULL: all rows.
 *   weights ([rows], i.e. [T][K]) need offsets and row_to_route; rows whose entry names
 *   no route are then left as they were. 1 <= I <= 32768, rows <= 2^23. */
int moe_activate(const void* h, int64_t h_stride, int32_t dtype, int32_t act, int32_t rows,
                 int32_t I, const int32_t* offsets, int32_t E, const int32_t* row_to_route,
                 const float* weights, void* out, int64_t out_stride, hipStream_t stream);

/* The same with an 8-bit result for moe_int_grouped_matmul: codes of a by
 * moe_int_quantize's rule, s = max_j |a_j| / 127 rounded to fp32, codes[j] = a_j / s to the
 * nearest integer, both of the a_j in 64 bits (so the codes are reproducible bit for
 * bit), and scales[m] = w s. A row with a value beyond fp32 or a NaN has codes 0 and a
 * scale that is not finite. codes: [rows][I], scales: [rows]. */
int moe_activate_int(const void* h, int64_t h_stride, int32_t dtype, int32_t act, int32_t rows,
                     int32_t I, const int32_t* offsets, int32_t E, const int32_t* row_to_route,
                     const float* weights, int8_t* codes, int64_t codes_stride, float* scales,
                     hipStream_t stream);

/* Gradients of moe_activate from da ([rows][I], the gradient of out): dh, of h's shape, and
 * dweights[route] = <da, a> in fp32, 0 for a route without a row (NULL, or with weights
 * and route_to_row). The same rows are read and written. */
int moe_activate_grad(const void* da, int64_t da_stride, const void* h, int64_t h_stride,
                      int32_t dtype, int32_t act, int32_t rows, int32_t I, const int32_t* offsets,
                      int32_t E, const int32_t* row_to_route, const int32_t* route_to_row,
                      const float* weights, void* dh, int64_t dh_stride, float* dweights,
                      hipStream_t stream);

/* The router's choice of K experts for each token.
 *   score s = softmax over the token's logits, or sigmoid (moe_score); choice c = s + bias
 *   (bias: [E] fp32 or NULL; it takes part in the choice only). The experts lie in
 *   `groups` groups of E / groups; a group's score is the sum of its group_top (1 or 2)
 *   largest choices, and the top_groups best groups take part. ids[t]: the K experts
 *   with the largest c, descending, ties (of groups too) to the lower index.
 *   weights[t][k] = scale s[ids[t][k]], divided by the sum of the chosen s if renormalize.
 * Choices are compared as if computed exactly (in 64 bits), not in rounded scores. An
 * expert whose logit or bias is -inf is never chosen; where fewer than K are left the
 * other ids are -1 (moe_sort_routes drops them) with weight 0. A NaN among a token's
 * logits makes its weights NaN (as a choice it counts as the lowest finite value), a NaN
 * in the bias every token's.
 *   logits: [T][E] of type dtype. 1 <= E <= 1024, 1 <= K <= min(E, 64), T*K <= 2^23,
 *   groups divides E. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
int moe_route(const void* logits, int64_t logits_stride, int32_t dtype, const float* bias,
              int32_t T, int32_t E, int32_t K, int32_t score, int32_t groups, int32_t top_groups,
              int32_t group_top, int32_t renormalize, float scale, int32_t* ids, float* weights,
              hipStream_t stream);

/* Gradient of moe_route's weights to the logits, from dweights [T][K]: dlogits [T][E] of
 * type dtype, written entirely. An id outside [0, E) and one whose logit is -inf add
 * nothing; the choice itself (and so the bias) has no gradient. */
int moe_route_grad(const float* dweights, const void* logits, int64_t logits_stride, int32_t dtype,
                   const int32_t* ids, int32_t T, int32_t E, int32_t K, int32_t score,
                   int32_t renormalize, float scale, void* dlogits, int64_t dlogits_stride,
                   hipStream_t stream);

/* Workspace bytes of moe_adapt (0 if the sizes are invalid). */
size_t moe_adapt_workspace_bytes(int32_t T, int32_t adapters, int32_t H, int32_t rank);

/* Low-rank adapters of many requests beside a shared projection:
 *   out[t] = base[t] + scales[e] b[e] (a[e] x[t]), e the adapter of token t, and
 *   out[t] = base[t] (bit for bit) for a token without one. Sums and a[e] x[t] in fp32
 *   (with fp16 operands to 2^-37 of the token's largest |a[e] x[t]|), one rounding. (An
 *   infinity in b makes its column infinite or NaN.)
 *   base, out: [T][N], x: [T][H], a: [adapters][rank][H], b: [adapters][N][rank], all of
 *   type dtype (bf16 or fp16); rows of a and b a_stride and b_stride apart, adapters
 *   a_adapter_stride and b_adapter_stride (0: one for all, to 2^48). scales: [adapters]
 *   fp32, or NULL for 1.
 *   row_to_token, token_to_row [T], offsets [adapters + 1]: the tokens sorted by adapter, as
 *   moe_sort_routes gives them for ids [T][1] (an id outside [0, adapters): no adapter).
 *   Entries of the maps that name no row or token stay in range; damaged maps leave rows
 *   of out unwritten.
 *   out may be base itself (same address and stride).
 *   workspace: >= moe_adapt_workspace_bytes(T, adapters, H, rank) bytes, 16-byte aligned.
 *   H a multiple of 16, rank a multiple of 8 up to 256 (MOE_ERR_UNSUPPORTED otherwise),
 *   1 <= adapters <= 1024, T <= 2^22, H, N <= 2^20. */
int moe_adapt(const void* base, int64_t base_stride, const void* x, int64_t x_stride, int32_t dtype,
              const int32_t* row_to_token, const int32_t* token_to_row, const int32_t* offsets,
              const void* a, int64_t a_adapter_stride, int64_t a_stride, const void* b,
              int64_t b_adapter_stride, int64_t b_stride, const float* scales, int32_t T,
              int32_t adapters, int32_t H, int32_t rank, int32_t N, void* workspace,
              size_t workspace_bytes, void* out, int64_t out_stride, hipStream_t stream);

/* Message for the last non-OK status returned on this thread. */
const char* moe_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_FP4_H */
