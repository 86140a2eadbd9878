/*
 * moe_fp4.h - C ABI of the MI355X (gfx950) library for the routed
 * mixture-of-experts FFN over block-scaled FP4 expert weights.
 *
 * The method (sources cited by title and section):
 *  [Q] "Running a 133 GB MoE model on an 8 GB GPU at 11 tokens/s by streaming
 *      experts from NVMe" (aiwithghost.com)
 *  [D] "Running the 510 GB DeepSeek-V4.1-Flash on an 8 GB GPU, and three bugs
 *      that never raise an error" (dev.to)
 *
 * One MoE layer: a router picks k of E experts per token from fp32 logits
 * (softmax, top-k, weights renormalised over the chosen k; [Q] "Why this
 * model, of all models": top-10 of 512; [D] "Bytes per token decide
 * everything": 6 of 384). Each chosen expert is a SwiGLU FFN
 * y = down(silu(gate x) * (up x)) whose three matrices are stored as 4-bit
 * e2m1 codes with one scale per group of G codes ([Q] "The engine", item 4:
 * NVFP4; [D] "Three bugs", item 2: ue8m0 scales). The layer output is the
 * weighted sum of the chosen experts' outputs (plus an optional dense bf16
 * shared expert). Decode runs one token; prefill runs the whole prompt
 * through the layer at once with tokens grouped by expert ([Q] "The engine",
 * item 5).
 *
 * Conventions for every entry point:
 *  - All buffers are DEVICE memory owned by the caller unless stated. The
 *    library never allocates, never synchronises, never reads device data on
 *    the host and never copies to the host; every call only enqueues work on
 *    `stream` (a hipStream_t; NULL = the default stream) and returns.
 *  - Return value: MOE_OK (0) or a negative MOE_ERR_* code. Arguments are
 *    validated on the host before anything is launched; on error nothing is
 *    launched and moe_last_error() describes the problem (thread-local).
 *  - A shape the library has no tuned kernel for returns
 *    MOE_ERR_UNSUPPORTED; there is no slow or silent fallback.
 *  - Faults inside kernels surface at the caller's next synchronisation.
 *  - Workspace `ws`: device memory of at least moe_workspace_bytes() bytes,
 *    256-byte aligned. Its contents on entry do not matter and nothing in it
 *    carries over from one call to the next (its first 4096 bytes are
 *    reserved and never written). Calls that share one workspace must not
 *    run concurrently.
 *  - The library keeps no mutable global state and is reentrant.
 */
#ifndef MOE_FP4_H
#define MOE_FP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Expert weight formats. Both use e2m1 codes (OCP MX FP4: magnitudes 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and a sign bit); they differ in the scale. */
#define MOE_FMT_NVFP4 1 /* one E4M3 (OCP FP8 E4M3FN) scale per 16 codes */
#define MOE_FMT_MXFP4 2 /* one UE8M0 (power-of-two) scale per 32 codes  */

#define MOE_OK 0
#define MOE_ERR_ARG (-1)         /* null / misaligned pointer, bad size or shape */
#define MOE_ERR_UNSUPPORTED (-2) /* valid, but no tuned kernel for this shape */
#define MOE_ERR_HIP (-3)         /* a HIP launch failed */
#define MOE_ERR_WORKSPACE (-4)   /* workspace missing or too small */

#define MOE_MODE_ROUTE 0
#define MOE_MODE_DECODE 1
#define MOE_MODE_PREFILL 2
#define MOE_MODE_DECODE_BATCH 3

#define MOE_OUT_F32 0
#define MOE_OUT_BF16 1

/* Layer shape. H = hidden size, I = expert intermediate size, E = experts,
 * k = experts per token, format = MOE_FMT_*. H and I must be multiples of
 * the format's group size G (16 or 32). */
typedef struct moe_desc {
    int32_t H, I, E, k, format;
} moe_desc;

/* Dense bf16 shared expert (bit patterns, row-major): gate [I][H], up [I][H],
 * down [H][I]. It is added to the layer output unweighted. */
typedef struct moe_shared {
    const uint16_t *gate;
    const uint16_t *up;
    const uint16_t *down;
} moe_shared;

/* Optional debug outputs of moe_expert_prefill (any member may be NULL).
 * Rows in "grouped order" are indexed by position p in perm (rows of one
 * expert are contiguous, see moe_expert_prefill). */
typedef struct moe_prefill_debug {
    uint16_t *x_bf16;   /* [T][H] x~ = bf16(x), NVFP4 layers */
    uint8_t *x_codes;   /* [T][H/2] x~ e2m1 codes, MXFP4 layers (element 2i in the low nibble) */
    uint8_t *x_scales;  /* [T][H/32] x~ UE8M0 scale bytes, MXFP4 layers */
    float *h_pre;       /* [T*k][I] silu(g)*u before rounding, grouped order */
    float *h_q;         /* [T*k][I] h~ (the rounded h, as fp32), grouped order */
    int32_t *perm;      /* [T*k] assignment id t*k+j at each grouped position */
    int32_t *off;       /* [E+1] first grouped position of each expert; off[E] = T*k */
    /* Controls of the NVFP4 GEMM launch's bounded wait (down tiles wait for
     * their gate/up tiles; a wait that ends unmet writes NaN over the tile's
     * outputs). 0 and 0: the library's behaviour. */
    int32_t tile_wait_polls;  /* > 0: poll limit instead of the library's (about 0.4 s) */
    int32_t tile_wait_unmet;  /* nonzero: every wait asks for one more gate/up tile than exists */
} moe_prefill_debug;

/* ---------------------------------------------------------------------- */
/* Expert block layout                                                     */
/* ---------------------------------------------------------------------- */

/* Bytes of one expert block: 3*H*I/2 code bytes + 3*H*I/G scale bytes.
 * Region order gate | up | down | gate_scale | up_scale | down_scale, as the
 * expert repack of [Q] "The engine", item 1 (2,764,800 B for the Qwen shape,
 * H=2560, I=640, NVFP4; 18,800,640 B = 17.93 MiB for the DeepSeek shape,
 * H=4096, I=2880, MXFP4, [D] "Bytes per token decide everything").
 * gate/up are [I][H] and down is [H][I]; every matrix is row-major with the
 * 4-bit codes packed along the row (element 2c in the low nibble of byte c of
 * the row); scales are row-major [rows][cols/G] bytes. Returns 0 for an
 * invalid descriptor. */
size_t moe_block_bytes(const moe_desc *d);

/* Byte offsets of the six regions (off[0..5]) and the block size (off[6]).
 * Returns MOE_OK or MOE_ERR_ARG. Host memory. */
int moe_block_layout(const moe_desc *d, int64_t off[7]);

/* Workspace bytes needed by one call of the given mode for T tokens. */
size_t moe_workspace_bytes(const moe_desc *d, int32_t T, int32_t mode);

/* ---------------------------------------------------------------------- */
/* Router                                                                  */
/* ---------------------------------------------------------------------- */

/* For each token t < T: logits[t][e] = sum_h Wr[e][h] * x[t][h] (fp32
 * accumulate); S = the k experts with the largest logits (ties: lower expert
 * index first), written to idx[t][0..k) in that order; w[t][j] =
 * softmax(logits[t])[S_j] / sum over S, i.e. the softmax weights
 * renormalised over the chosen k ([Q] "Where the time actually goes": the
 * router's chosen experts). Nothing is read back to the host.
 *   x          [T][H] fp32, 16-B aligned
 *   Wr         [E][H] fp32, 16-B aligned
 *   idx        [T][k] int32 (out);  w [T][k] fp32 (out)
 *   logits_out [T][E] fp32 (out) or NULL
 * Errors: MOE_ERR_ARG for an invalid descriptor (k > E, sizes not positive
 * or not multiples of G), a null or misaligned pointer, T < 1;
 * MOE_ERR_UNSUPPORTED unless H % 256 == 0, H <= 8192, E <= 1024 and k <= 32;
 * MOE_ERR_WORKSPACE for a workspace below moe_workspace_bytes(d, T,
 * MOE_MODE_ROUTE). */
int moe_route(const moe_desc *d, const float *x, int32_t T, const float *Wr, int32_t *idx, float *w,
              float *logits_out, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Decode: one token                                                       */
/* ---------------------------------------------------------------------- */

/* The single-token expert computation of one MoE layer ([Q] "The engine",
 * item 4: a single-token SwiGLU expert kernel over NVFP4 weights, decoding
 * the e2m1 codes on the fly; [Q] "Why this model, of all models": gate, up
 * and down matrices per expert, and a shared expert kept in bf16):
 * y = sum_{j<k} w[j] * expert_{idx[j]}(x)  (+ shared(x) if shared != NULL)
 * where expert_e(x) = down_e( silu(gate_e x) * (up_e x) ), silu(z) =
 * z / (1 + exp(-z)), weights decoded on the fly from the block at
 * expert_ptrs[e] (format per d->format), fp32 activations and fp32
 * accumulation. The combine runs in increasing j (then the shared
 * expert), so results are bit-identical from run to run.
 *   x           [H] fp32, 16-B aligned
 *   expert_ptrs DEVICE array of E pointers (8-B aligned), each to one
 *               256-B-aligned expert block (resident layers:
 *               base + e * moe_block_bytes)
 *   idx [k] int32, w [k] fp32: the routing (e.g. from moe_route)
 *   shared      host struct of device pointers, or NULL
 *   y           [H] fp32 (out)
 * Requires H % 512 == 0, H <= 4096, 16 <= I <= 4096 (a multiple of G), and
 * k <= 32; other shapes return MOE_ERR_UNSUPPORTED. */
int moe_expert_decode(const moe_desc *d, const float *x, const void *const *expert_ptrs, const int32_t *idx,
                      const float *w, const moe_shared *shared, float *y, void *ws, size_t ws_bytes, void *stream);

/* One decode layer in one call: moe_route (T = 1) followed by
 * moe_expert_decode, with the same results (bit-identical chosen experts,
 * weights and y), in three launches instead of four: the router GEMV shares
 * a launch with the shared expert's gate/up (neither depends on the
 * routing), and the top-k is recomputed at the start of every routed
 * gate/up workgroup. idx_out [k] int32 and w_out [k] fp32 receive the
 * routing. Requirements: those of moe_route and of moe_expert_decode;
 * workspace: moe_workspace_bytes(d, 1, MOE_MODE_DECODE). */
int moe_layer_decode(const moe_desc *d, const float *x, const float *Wr, const void *const *expert_ptrs,
                     const moe_shared *shared, float *y, int32_t *idx_out, float *w_out, void *ws, size_t ws_bytes,
                     void *stream);

/* ---------------------------------------------------------------------- */
/* Decode: a few tokens                                                    */
/* ---------------------------------------------------------------------- */

/* One layer for T tokens at once (sequences decoded side by side, a draft of
 * several tokens checked at once): for every token what moe_layer_decode
 * computes for one, in fp32 with fp32 accumulation; each chosen expert's block
 * is read for all of its tokens together. Results are bit-identical from run to
 * run, but not to moe_layer_decode's, except for T = 1 without a mask, which
 * runs its kernels (otherwise the sums run in another order; the chosen experts
 * agree unless two logits differ by less than their rounding). Two tokens of
 * many small experts take less time in two calls of moe_layer_decode (512
 * experts of 2560 x 640: 32 us against 42), three as much, more take less here.
 *   x    [T][H] fp32, 16-B aligned;  Wr [E][H] fp32
 *   mask [T] uint8 or NULL: a token with mask[t] == 0 (an empty slot of a
 *        serving batch) is left out: its rows of y, idx_out and w_out stay as
 *        they were, and its row of x does not matter
 *   y    [T][H] fp32 (out);  idx_out [T][k] int32 (out);  w_out [T][k] fp32 (out)
 * expert_ptrs, shared and the supported shapes as for moe_layer_decode, and
 * T <= 64 (MOE_ERR_UNSUPPORTED above; moe_expert_prefill takes longer
 * batches). T = 0 enqueues nothing. Outputs overlap neither inputs nor each
 * other. Workspace: moe_workspace_bytes(d, T, MOE_MODE_DECODE_BATCH), which
 * never falls as T grows. */
int moe_layer_decode_batch(const moe_desc *d, const float *x, int32_t T, const uint8_t *mask, const float *Wr,
                           const void *const *expert_ptrs, const moe_shared *shared, float *y, int32_t *idx_out,
                           float *w_out, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Decode without a workspace                                              */
/* ---------------------------------------------------------------------- */

/* Bytes of the static scratch array behind moe_layer_decode_noalloc. Every
 * shape moe_layer_decode supports needs at most 549,120 bytes. */
#define MOE_NOALLOC_SCRATCH_BYTES 1048576

/* moe_layer_decode for callers that cannot allocate memory: code being
 * captured into a HIP graph, tight serving loops, harnesses that forbid
 * allocation. Same arguments minus the workspace, same kernels, bit-identical
 * results. The workspace is a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES bytes that the library holds on every GPU it runs
 * on until the process ends; its address on the current device is looked up
 * on the first call there (hipGetSymbolAddress). No call allocates or frees
 * memory. Nothing in the array carries over from one call to the next, but
 * all calls on one GPU share it: calls that may overlap on one GPU (other
 * streams, other host threads) race and must not be issued; calls ordered on
 * one stream are fine. Errors: those of moe_layer_decode (apart from the
 * workspace ones); MOE_ERR_WORKSPACE if a layer would need more than
 * MOE_NOALLOC_SCRATCH_BYTES; MOE_ERR_HIP if the lookup fails. */
int moe_layer_decode_noalloc(const moe_desc *d, const float *x, const float *Wr, const void *const *expert_ptrs,
                             const moe_shared *shared, float *y, int32_t *idx_out, float *w_out, void *stream);

/* ---------------------------------------------------------------------- */
/* Prefill: T tokens grouped by expert                                     */
/* ---------------------------------------------------------------------- */

/* out[t] = sum_{j<k} w[t][j] * down_e( Q( silu(gate_e x~_t) * (up_e x~_t) ) ),
 * e = idx[t][j], for every token at once ([Q] "The engine", item 5: the
 * whole prompt through each layer). Assignments a = t*k + j are grouped by
 * expert with a stable counting sort (count, exclusive prefix scan, scatter;
 * within an expert in increasing a) and each expert's rows are multiplied
 * as one ragged GEMM. Activation rounding points:
 *   NVFP4: x~ = bf16(x) and h~ = bf16(h) (round to nearest even); the
 *          weights are dequantised to bf16 exactly; bf16 MFMA, fp32 accumulate.
 *   MXFP4: x~ and h~ are converted to MXFP4 per 32 consecutive elements
 *          (OCP MX: shared exponent floor(log2 max|v|) - 2, e2m1 codes by
 *          round-to-nearest-even with saturation); scaled FP4 MFMA, fp32
 *          accumulate.
 * The combine runs in increasing j in fp32; out is fp32 [T][H] or, with
 * out_dtype = MOE_OUT_BF16, bf16 [T][H] rounded from that fp32 sum.
 *   x [T][H] fp32; idx, w [T][k]; expert_ptrs as for decode; dbg optional.
 * Requires H % 256 == 0 and I % 128 == 0 (NVFP4) or H % 512 == 0 and
 * I % 64 == 0 (MXFP4), H and I <= 16384, E <= 1024, k <= 32. */
int moe_expert_prefill(const moe_desc *d, const float *x, int32_t T, const void *const *expert_ptrs,
                       const int32_t *idx, const float *w, void *out, int32_t out_dtype, void *ws,
                       size_t ws_bytes, const moe_prefill_debug *dbg, void *stream);

/* ---------------------------------------------------------------------- */
/* FP8 beside the MoE path                                                 */
/* ---------------------------------------------------------------------- */

#define MOE_SCALE_FLOOR 0 /* OCP MX: X = floor(log2 amax) - 8; quotients above 448 saturate */
#define MOE_SCALE_CEIL 1  /* smallest X with amax <= 448 * 2^X; never saturates */

/* Activation quantiser: FP8 E4M3 codes with one UE8M0 (power-of-two) scale
 * per block of `block` consecutive values of a row ([D] "Three bugs", item
 * 2: DeepSeek's activation quantiser, ue8m0 scales, FP8 out, checked
 * bit-exact at 1, 17, 300 and 1024 rows; OCP MX: MXFP8 uses blocks of 32).
 *   x       fp32 [rows][cols], 16-byte aligned
 *   block   32 or 128; cols a positive multiple of block
 *   rule    MOE_SCALE_FLOOR or MOE_SCALE_CEIL (shared exponent X of a block
 *           from its largest magnitude amax, clamped to [-127, 127])
 *   codes   out: uint8 [rows][cols], 4-byte aligned: E4M3 (OCP E4M3FN) of
 *           v / 2^X rounded to nearest even, magnitudes clamped to 448;
 *           negative values that round to zero give 0x80
 *   scales  out: uint8 [rows][cols/block]: X + 127 (0 for an all-zero block)
 * rows == 0 enqueues nothing and returns MOE_OK. No workspace. Inputs must be
 * finite. Errors: MOE_ERR_ARG (pointers, sizes, block, rule). */
int moe_act_quant_fp8(const float *x, int32_t rows, int32_t cols, int32_t block, int32_t rule, uint8_t *codes,
                      uint8_t *scales, void *stream);

/* Row-scaled FP8 matrix-vector product ([Q] "The engine", item 4: the FP8
 * row-scaled matrix-vector kernel; [Q] "Why this model, of all models": the
 * large dense matrices stored in FP8 with one scale per row):  y[r] = row_scale[r] * sum_c e4m3(W[r][c]) * x[c],
 * accumulated in fp32.
 *   W          uint8 E4M3 codes [rows][cols], row-major, 16-byte aligned
 *   row_scale  fp32 [rows];  x  fp32 [cols], 16-byte aligned;  y  fp32 [rows]
 * cols must be 512 * d with d in 1..8, 10, 12 or 16 (MOE_ERR_UNSUPPORTED
 * otherwise); rows >= 0 (0 enqueues nothing). No workspace. */
int moe_gemv_fp8(const uint8_t *W, const float *row_scale, const float *x, int32_t rows, int32_t cols, float *y,
                 void *stream);

/* ---------------------------------------------------------------------- */
/* Training the router                                                     */
/* ---------------------------------------------------------------------- */

/* The router's balance loss, its z loss, the per-expert counts and the
 * gradient of the logits. A batch is T tokens in S sequences: sequence s
 * holds the tokens seq_off[s] <= t < seq_off[s + 1] with mask[t] != 0 (its
 * counted tokens, n_s of them); tokens before seq_off[0], behind seq_off[S]
 * or with mask[t] == 0 are not counted, and their values do not matter. With
 * p_t = softmax(logits[t]) over all E, lse_t its log-sum-exp, live = the
 * sequences with n_s > 0 and N = sum n_s:
 *   counts[s][e] = #{(t, j): t counted in s, idx[t][j] = e}
 *   probs[s][e]  = mean of p_t[e] over the counted tokens of s (0 if none)
 *   balance = 1/live sum_s E sum_e counts[s][e] / (n_s k) * probs[s][e]
 *   z       = 1/N sum_t lse_t^2
 *   loss    = { balance_coef * balance + z_coef * z, balance, z }
 *   dlogits = dloss[0] * d loss[0] / d logits, the counts taken as constants;
 *             0 in the rows of tokens that are not counted
 * A term whose coefficient is 0 does not enter loss[0] or dlogits. A counted
 * token whose logits are all -inf has p = 0 and lse = 0. A batch without
 * counted tokens has the loss 0. Softmax and sums in fp32, in a fixed order:
 * results are bit-identical from run to run.
 *   logits  [T][E] fp32, 16-B aligned (e.g. logits_out of moe_route)
 *   idx     [T][k] int32 (the routing)
 *   mask    [T] uint8, or NULL: every token counts
 *   seq_off [S + 1] int32, not decreasing, in [0, T]; or NULL: one sequence
 *           of T tokens (S must be 1)
 *   dloss   [1] fp32, or NULL: 1
 *   loss    [3] fp32 (out)
 *   counts  [S][E] int32 (out) or NULL;  probs [S][E] fp32 (out) or NULL
 *   dlogits [T][E] fp32 (out), 16-B aligned, or NULL; not logits itself
 * If seq_off decreases or leaves [0, T], or a counted token names an expert
 * outside [0, E), every fp32 output is NaN and every count -1. T = 0 gives
 * the loss 0 (logits, idx and dlogits are not used). Outputs overlap neither
 * inputs nor each other. Workspace: moe_balance_workspace_bytes(d, T, S),
 * which never falls as T grows. Errors: MOE_ERR_ARG (descriptor,
 * pointers, T < 0, S < 1, coefficients that are not finite);
 * MOE_ERR_UNSUPPORTED unless E <= 1024, k <= 32, S <= 65535 and T <= 2^24;
 * MOE_ERR_WORKSPACE. d->H, d->I and d->format only have to be valid. */
size_t moe_balance_workspace_bytes(const moe_desc *d, int32_t T, int32_t S);
int moe_balance_loss(const moe_desc *d, const float *logits, int32_t T, const int32_t *idx, const uint8_t *mask,
                     const int32_t *seq_off, int32_t S, float balance_coef, float z_coef, const float *dloss,
                     float *loss, int32_t *counts, float *probs, float *dlogits, void *ws, size_t ws_bytes,
                     void *stream);

#define MOE_ACC_DX 1  /* add to dx instead of writing it */
#define MOE_ACC_DWR 2 /* add to dWr instead of writing it */
#define MOE_FP32_PRODUCTS 8 /* fp32 operands in batches of any length */

/* The backward pass of moe_route: from dw, the loss's gradient at the
 * routing weights w, and dlogits_in, a gradient that reaches the logits
 * directly (moe_balance_loss), to the logits, the layer input and the router.
 *   ds[t][j] = w[t][j] * (dw[t][j] - sum_i w[t][i] dw[t][i])
 *   G[t][e]  = dlogits_in[t][e] + sum_{j: idx[t][j] = e} ds[t][j]
 *   dx = G Wr ([T][H]),  dWr = G^T x ([E][H])
 * Tokens with mask[t] == 0 have G = 0, and their values do not matter. A token
 * with an index outside [0, E) (dw given) has G = NaN in its whole row. Sums in
 * fp32; results are bit-identical from run to run. Below 2^29 multiplications
 * (T E H), with up to 64 experts, and where the caller asks for it
 * (MOE_FP32_PRODUCTS), the products have fp32 operands. Otherwise each operand is a pair of fp16 values under a power of two for its
 * row or column, h + l with h = fp16(v), l = fp16(v - h), and the product of
 * the two l is left out: off by at most 3 * 2^-22 of each product, and for
 * values below 2^-17 of their row's (Wr, x: column's) largest by 2^-39 of that
 * largest, whatever the exponents. An infinity or a NaN there makes every sum
 * that it enters infinite or NaN.
 *   x [T][H], Wr [E][H] fp32, 16-B aligned (x may be NULL without dWr, Wr
 *   without dx);  idx [T][k] int32, w [T][k], dw [T][k] fp32 (dw NULL: only
 *   dlogits_in; idx and w are then not used);  mask [T] uint8 or NULL;
 *   dlogits_in [T][E] fp32 or NULL (one of dw and dlogits_in is needed);
 *   dlogits_out [T][E] fp32 (out): G, or NULL; may be dlogits_in;
 *   dx [T][H], dWr [E][H] fp32 (out), 16-B aligned, or NULL
 *   accumulate  a sum of MOE_ACC_* and MOE_FP32_PRODUCTS
 * Outputs overlap neither inputs nor each other, but for dlogits_out ==
 * dlogits_in. T = 0 writes zeros to dWr (unless it accumulates). Workspace:
 * moe_route_backward_workspace_bytes(d, T), which never falls as T grows.
 * Errors: MOE_ERR_ARG (also where an output is an input or another output);
 * MOE_ERR_UNSUPPORTED unless moe_route supports the descriptor and
 * T <= 2^20; MOE_ERR_WORKSPACE. */
size_t moe_route_backward_workspace_bytes(const moe_desc *d, int32_t T);
int moe_route_backward(const moe_desc *d, const float *x, int32_t T, const float *Wr, const int32_t *idx,
                       const float *w, const float *dw, const uint8_t *mask, const float *dlogits_in,
                       float *dlogits_out, float *dx, float *dWr, int32_t accumulate, void *ws, size_t ws_bytes,
                       void *stream);

/* ---------------------------------------------------------------------- */
/* Low-rank adapters beside a shared projection                            */
/* ---------------------------------------------------------------------- */

/* Types of activations (x, base, y and their gradients) and of the factors:
 * F32: fp32 activations, bf16 factors; BF16: both bf16; F16: both fp16. */
#define MOE_ACT_F32 0
#define MOE_ACT_BF16 1
#define MOE_ACT_F16 2

/* K = input size, N = output size of the projection, n = adapters in the
 * tables, max_rank = the largest rank among them, dtype = MOE_ACT_*. */
typedef struct moe_lora_desc {
    int32_t K, N, n, max_rank, dtype;
} moe_lora_desc;

/* Many requests share one projection (moe_gemv_fp8, a shared expert's
 * matrix, any other), each with a low-rank adapter of its own: with
 * a = ids[t],
 *   y[t] = base[t] + scales[a] * B_a^T (A_a x[t])        (a < 0: y[t] = base[t])
 * where base is the projection's output. y may be base (the same rows and
 * stride). Products and sums in fp32 (16-bit operands multiply exactly, fp32
 * activations enter with all their bits); the intermediate A_a x stays fp32;
 * y is rounded once. Infinities and NaN enter the sums as in fp32 arithmetic;
 * an fp32 value's bits below 2^-133 may count as 0. Results are bit-identical
 * from run to run.
 *   x     [T] rows of K, stride ldx elements;  base (or NULL: zeros) and y
 *         [T] rows of N, strides ldbase and ldy. 16-B aligned, strides
 *         multiples of 8 and at least the row.
 *   ids   [T] int32: the token's adapter; negative: none
 *   a_ptrs, b_ptrs  DEVICE arrays of n pointers, 16-B-aligned each: A_a
 *         [r_a][K] and B_a [r_a][N] (rank-major: B_a is the transpose of the
 *         usual [N][r]), dense
 *   ranks [n] int32, 0 .. max_rank;  scales [n] fp32
 * A token whose id is n or more, or whose adapter's rank is not in
 * 0 .. max_rank or has a NULL factor beside a rank above 0, gets NaN in its
 * row. Only rows of x whose tokens have an adapter are read. T = 0 enqueues
 * nothing. y overlaps no input, but for y == base. Workspace:
 * moe_lora_workspace_bytes(l, T, 0), which never falls as T grows. Errors: MOE_ERR_ARG (descriptor: sizes
 * not positive, K or N not a multiple of 8, unknown dtype; pointers, strides,
 * T < 0); MOE_ERR_UNSUPPORTED unless K, N <= 65536, n <= 1024,
 * max_rank <= 128 and T <= 2^20; MOE_ERR_WORKSPACE. */
size_t moe_lora_workspace_bytes(const moe_lora_desc *l, int32_t T, int32_t backward);
int moe_lora_apply(const moe_lora_desc *l, const void *x, int64_t ldx, int32_t T, const int32_t *ids,
                   const void *const *a_ptrs, const void *const *b_ptrs, const int32_t *ranks, const float *scales,
                   const void *base, int64_t ldbase, void *y, int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* The backward pass of moe_lora_apply: with v_t = scales[a] * B_a dy[t] and
 * u_t = scales[a] * A_a x[t],
 *   dx[t] = dx_base[t] + A_a^T v_t     (dx_base: the projection's own
 *           gradient of x, or NULL: zeros; dx may be dx_base; dx may be NULL)
 *   dA_a  = sum_{t: ids[t] = a} v_t x[t]^T   ([r_a][K] fp32)
 *   dB_a  = sum_{t: ids[t] = a} u_t dy[t]^T  ([r_a][N] fp32)
 * Tables, types, arithmetic, alignment and strides as for moe_lora_apply; dy
 * [T] rows of N. da_ptrs and db_ptrs are DEVICE arrays of n pointers to fp32 memory (16-B
 * aligned each, no two the same), or NULL; an entry that is NULL skips that
 * adapter's factor (an adapter that is served but not trained). An adapter
 * without tokens gets zeros. accumulate != 0 adds to dA and dB instead of
 * writing them. A token whose id is n or more, or whose adapter has no usable
 * rank (not in 0 .. max_rank, or above 0 beside a NULL factor), gets NaN in
 * its row of dx and enters no gradient; the gradients of an adapter with such
 * a rank are left as they are (one without tokens may have NULL factors). Sums
 * over tokens run in a fixed order: results are bit-identical from run to run.
 * Outputs overlap neither inputs nor each other, but for dx == dx_base.
 * Workspace: moe_lora_workspace_bytes(l, T, 1), which never falls as T grows.
 * Errors as for moe_lora_apply. */
int moe_lora_backward(const moe_lora_desc *l, const void *x, int64_t ldx, const void *dy, int64_t lddy, int32_t T,
                      const int32_t *ids, const void *const *a_ptrs, const void *const *b_ptrs, const int32_t *ranks,
                      const float *scales, const void *dx_base, int64_t lddx_base, void *dx, int64_t lddx,
                      float *const *da_ptrs, float *const *db_ptrs, int32_t accumulate, void *ws, size_t ws_bytes,
                      void *stream);

/* ---------------------------------------------------------------------- */
/* 4-bit matrices: quantisation and products                               */
/* ---------------------------------------------------------------------- */

#define MOE_SCALE_NEAREST 2 /* NVFP4: the E4M3 value nearest to amax / 6 */

/* A matrix to block-scaled e2m1 codes, laid out as in an expert block (codes
 * [rows][cols / 2], element 2c in the low nibble of byte c; scales
 * [rows][cols / G]): three calls fill the regions of one block.
 *   MOE_FMT_MXFP4, rule MOE_SCALE_FLOOR: shared exponent X = floor(log2 amax) - 2
 *     (OCP MX; quotients above 6 saturate); MOE_SCALE_CEIL: the smallest X with
 *     amax <= 6 * 2^X. X is clamped to [-127, 125]; byte X + 127, 0 for an
 *     all-zero block. row_exp must be NULL.
 *   MOE_FMT_NVFP4, rule MOE_SCALE_NEAREST: scale = the E4M3 value nearest to
 *     amax / 6 (ties to even, at most 448) of the row's values times 2^-e.
 *     e = row_exp[r] (out) is the smallest with the row's largest finite
 *     magnitude <= 2688 * 2^e, in [-100, 116], 0 for a row of zeros; with
 *     row_exp NULL (expert blocks) e = 0.
 *   codes: v / (scale 2^e) to the nearest e2m1 value, ties to the even code,
 *     magnitudes above 6 saturate; a negative value that rounds to zero keeps
 *     its sign. A block that holds an infinity or a NaN gets a NaN scale (0xFF;
 *     E4M3 0x7F) and codes 0.
 * Every step is exact: the codes and scales are those of the definition.
 *   x      [rows] rows of cols elements of dtype (MOE_ACT_*), stride ldx
 *          elements; 16-B aligned, strides multiples of 8
 *   cols   a positive multiple of G
 *   codes  (out) 4-B aligned, or NULL;  scales (out) or NULL
 *   values (out) the values that the codes stand for, in dtype (in fp16 at most
 *          65504 in magnitude), stride ldv; or NULL; may be x with its stride
 * At least one output. rows == 0 enqueues nothing. No workspace. Errors:
 * MOE_ERR_ARG; MOE_ERR_UNSUPPORTED above 2^33 elements. */
int moe_fp4_quant(const void *x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype, int32_t format, int32_t rule,
                  int8_t *row_exp, uint8_t *codes, uint8_t *scales, void *values, int64_t ldv, void *stream);

/* K = input size, N = output size, format = MOE_FMT_*, dtype = MOE_ACT_* of
 * the activations on both sides. */
typedef struct moe_fp4_desc {
    int32_t K, N, format, dtype;
} moe_fp4_desc;

/* y[t] = base[t] + W x[t] with W [N][K] stored as moe_fp4_quant writes it:
 * W[n][k] = e2m1(code) * scale * 2^row_exp[n]. The activations keep all their
 * bits (fp32 ones down to 2^-133), products are exact, sums are in fp32 and y
 * is rounded once. The sums of moe_fp4_apply take the row's power of two at
 * their end, and have to be within fp32 before it (they are for activations of
 * magnitudes 2^-100 to 2^100); in moe_fp4_backward each product takes it. With
 * round_x != 0 (MOE_FMT_MXFP4 only) the activations are first rounded to MXFP4
 * per 32 elements (MOE_SCALE_FLOOR) and multiplied as codes on the FP4 matrix
 * units. Results are bit-identical from run to run.
 *   x     [T] rows of K, stride ldx;  base (or NULL: zeros; may be y, with its
 *         stride) and y [T] rows of N, strides ldbase and ldy. 16-B aligned,
 *         strides multiples of 8, at least the row and at most 2^22 elements
 *   codes [N][K / 2], 16-B aligned; scales [N][K / G];
 *   row_exp [N] in [-100, 116], or NULL: zeros (MOE_FMT_MXFP4: must be NULL)
 * An infinity or a NaN among the activations enters the sums as in fp32
 * arithmetic. A NaN scale in W makes every output that it enters NaN; a value
 * of W above the largest fp32 (scale bytes 253 and 254, which moe_fp4_quant
 * does not write) makes them infinite or NaN, or, with round_x, where codes
 * are multiplied as they are, enters as that value. T = 0 enqueues nothing. y
 * overlaps no input, but for base. Workspace:
 * moe_fp4_workspace_bytes(f, T, 0), which never falls as T grows. Errors:
 * MOE_ERR_ARG (K not a multiple of 32, N not of 8, pointers, strides, round_x
 * with NVFP4); MOE_ERR_UNSUPPORTED unless K, N <= 65536, T <= 2^20, strides
 * <= 2^22 and, with round_x, T * K <= 2^33; MOE_ERR_WORKSPACE. */
size_t moe_fp4_workspace_bytes(const moe_fp4_desc *f, int32_t T, int32_t backward);
int moe_fp4_apply(const moe_fp4_desc *f, const void *x, int64_t ldx, int32_t T, const uint8_t *codes,
                  const uint8_t *scales, const int8_t *row_exp, int32_t round_x, const void *base, int64_t ldbase,
                  void *y, int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* The activations' gradient: dx[t] = dx_base[t] + W^T dy[t] (W is frozen; a
 * rounding of x counts as the identity). dy [T] rows of N, dx_base (or NULL)
 * and dx [T] rows of K; dx may be dx_base, e.g. to add to what
 * moe_lora_backward takes as its own dx_base. Arithmetic, alignment, strides,
 * limits and errors as for moe_fp4_apply; workspace:
 * moe_fp4_workspace_bytes(f, T, 1). */
int moe_fp4_backward(const moe_fp4_desc *f, const void *dy, int64_t lddy, int32_t T, const uint8_t *codes,
                     const uint8_t *scales, const int8_t *row_exp, const void *dx_base, int64_t lddx_base, void *dx,
                     int64_t lddx, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* The norms around a block                                                */
/* ---------------------------------------------------------------------- */

#define MOE_GATE_NONE 0
#define MOE_GATE_CHANNEL 1 /* gate [H]: one learned value a channel */
#define MOE_GATE_TOKEN 2   /* gate [T]: one value a token */

/* H = hidden size; r_dtype, y_dtype, x_dtype = MOE_ACT_* of the residual
 * stream, the block's output and the next block's input; gate = MOE_GATE_*;
 * scale = residual scale; eps > 0. */
typedef struct moe_norm_desc {
    int32_t H, r_dtype, y_dtype, x_dtype, gate;
    float scale, eps;
} moe_norm_desc;

/* Behind a block and before the next one, in one pass: with
 * rms(v) = v / sqrt(mean(v^2) + eps),
 *   s     = r + scale * gate * (rms(y) * post)
 *   r_out = s rounded to r_dtype
 *   x     = rms(s) * pre rounded to x_dtype (from s before its rounding)
 * in fp32. y NULL: s = r (the norm before the first block); post NULL: y
 * enters without a norm; pre NULL: no x.
 *   r, y  [T] rows of H with strides ldr, ldy;  r_out (or NULL; may be r, with
 *         its stride) and x (NULL without pre) [T] rows of H. 16-B aligned,
 *         strides multiples of 8 and at least H
 *   mask  [T] uint8 or NULL: rows with mask[t] == 0 are not read, and their
 *         rows of r_out and x stay as they were
 *   post, pre [H] fp32, 16-B aligned;  gate [H] or [T] fp32 (channel: 16-B
 *         aligned)
 * T = 0 enqueues nothing. Outputs overlap neither inputs nor each other, but
 * for r_out == r. Errors: MOE_ERR_ARG (H not a multiple of 8, eps not above 0,
 * scale not finite, pointers, strides); MOE_ERR_UNSUPPORTED unless H <= 16384
 * and T <= 2^20. */
int moe_block_norm(const moe_norm_desc *n, const void *r, int64_t ldr, const void *y, int64_t ldy, int32_t T,
                   const uint8_t *mask, const float *post, const float *gate, const float *pre, void *r_out,
                   int64_t ldr_out, void *x, int64_t ldx, void *stream);

/* Its backward pass, from the stored sum r_out (all of the forward pass that
 * it needs beside y): dr_out is the gradient that reaches r_out from behind
 * (NULL: zeros), dx the gradient of x (NULL: zeros; needed with dpre). With
 * n = rms(r_out), q = rms(y) (y itself without post) and the root mean squares
 * S and Y that they were divided by:
 *   a = dx * pre,  d = dr_out + (a - n * mean(a n)) / S,  dr = d
 *   dpre = sum_t dx * n;  u = scale * gate * d;  dpost = sum_t u * q
 *   dgate = scale * d * q * post summed over the tokens (channel) or the
 *           channels (token)
 *   b = u * post,  dy = (b - q * mean(b q)) / Y   (without post: dy = u)
 * A row with mask[t] == 0 has dr = dy = 0, dgate[t] = 0 and enters no sum.
 *   dr [T] rows of H (r_dtype; may be dr_out, with its stride), dy [T] rows of
 *   H (y_dtype), dpost, dpre [H], dgate [H] or [T] fp32 (out); any may be NULL.
 *   accumulate != 0 adds to dpost, dpre and dgate instead of writing them.
 * Sums over tokens run in a fixed order: results are bit-identical from run to
 * run. T = 0 writes zeros to dpost, dpre and a channel's dgate (unless it
 * accumulates). Outputs overlap neither inputs nor each other, but for
 * dr == dr_out. Workspace: moe_block_norm_workspace_bytes(n, T), which never
 * falls as T grows. Errors as for moe_block_norm; MOE_ERR_WORKSPACE. */
size_t moe_block_norm_workspace_bytes(const moe_norm_desc *n, int32_t T);
int moe_block_norm_backward(const moe_norm_desc *n, const void *r_out, int64_t ldr_out, const void *y, int64_t ldy,
                            int32_t T, const uint8_t *mask, const float *post, const float *gate, const float *pre,
                            const void *dr_out, int64_t lddr_out, const void *dx, int64_t lddx, void *dr, int64_t lddr,
                            void *dy, int64_t lddy, float *dpost, float *dgate, float *dpre, int32_t accumulate,
                            void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Speculative expert prefetch                                             */
/* ---------------------------------------------------------------------- */

/* ([Q] "The engine", item 3: guess the next layer's experts and read them
 * while the GPU is busy; [D] "Making it faster": predicting the next layer's
 * experts.) Reads the whole blocks of experts idx[0..n) (device int32; an
 * index outside [0, E) is skipped) through expert_ptrs so that they sit in
 * the GPU's last-level cache when a following launch needs them. The guess is
 * the caller's: typically moe_route with the next layer's router on this
 * layer's input, on a second stream. The read is made observable: sink
 * (device, 4-byte aligned, at least moe_prefetch_sink_bytes(d, n) bytes)
 * receives, for expert j and 64 KiB chunk c of its block, the XOR of the
 * chunk's 32-bit words at sink[j * nchunks + c] (0 for a skipped index).
 * n in 1..1024. Errors: MOE_ERR_ARG. */
size_t moe_prefetch_sink_bytes(const moe_desc *d, int32_t n);
int moe_expert_prefetch(const moe_desc *d, const void *const *expert_ptrs, const int32_t *idx, int32_t n,
                        uint32_t *sink, size_t sink_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Expert tier: pinned host blocks with an HBM slot cache                  */
/* ---------------------------------------------------------------------- */

/* ([Q] "The engine", items 2-3: an LRU cache of experts in front of the slow
 * tier, GPU slots, and copies into them overlapped with compute; [D] "Making
 * it faster".) Every expert block of `layers` layers lives in pinned host
 * memory; n_slots HBM slots hold the most recently routed ones. The tier owns
 * the per-layer pointer tables the decode entry points take
 * (expert_ptrs = table + layer * E): each entry points at the expert's HBM
 * slot or, for experts not in HBM, at its pinned host block, which the
 * kernels then read in place over PCIe (no copy, no host synchronisation).
 *
 * Unlike the compute entry points, the tier is a resource-owning object: it
 * creates one copy stream and a few events, allocates a small pinned staging
 * array and host-side state, and moe_tier_create synchronises once (initial
 * table). Every decode launch that reads the table must be on the
 * compute_stream given to moe_tier_update (the tier orders its table writes
 * with those launches); not for use under graph capture. */
typedef struct moe_tier moe_tier;
typedef struct {
    int64_t resident;   /* experts whose table entry points at their HBM slot */
    int64_t pending;    /* experts being copied (entry switches at the next update) */
    int64_t hits;       /* routed (layer, slot) uses found resident, over all updates */
    int64_t misses;     /* routed uses read from host memory */
    int64_t promotions; /* blocks copied into slots */
    int64_t evictions;  /* experts moved back to their host blocks */
} moe_tier_stats;

/*   host_blocks  pinned host memory (hipHostMalloc or equivalent, mapped at the
 *                same address on the device): layers * E blocks of
 *                moe_block_bytes(d), layer-major, 256-byte aligned
 *   slots        device memory for n_slots blocks (NULL if n_slots == 0)
 *   table        device memory for layers * E pointers, 8-byte aligned;
 *                filled by the tier (all entries start at the host blocks)
 * Errors: MOE_ERR_ARG (sizes, alignment, memory not pinned / not on the
 * device), MOE_ERR_HIP. */
int moe_tier_create(const moe_desc *d, int32_t layers, void *host_blocks, void *slots, int32_t n_slots, void **table,
                    moe_tier **out);

/* Waits for the tier's own copies, then frees its streams, events and state
 * (not the caller's buffers). Work the caller enqueued that reads the table
 * must be finished first. */
int moe_tier_destroy(moe_tier *t);

/* After a decode step: idx_host [layers][k] is that step's routing (host
 * memory, e.g. read back asynchronously by the caller; indices outside
 * [0, E) are ignored). Enqueued on compute_stream, in this order: the table
 * entries of the previous update's newcomers switch to their slots (after
 * their copies, by event); up to max_promote experts of this step that are
 * not in HBM take a free slot or the slot of the least recently used expert
 * that this step did not use, whose entry first returns to its host block;
 * then, on the tier's copy stream, once the compute stream has passed those
 * entries, the newcomers' blocks are copied into their slots (overlapping the
 * compute stream). Nothing here waits on the host except for a staging
 * buffer four updates old. */
int moe_tier_update(moe_tier *t, const int32_t *idx_host, int32_t max_promote, void *compute_stream);

/* Counters and residency (host state, no device access). */
int moe_tier_get_stats(const moe_tier *t, moe_tier_stats *out);

/* Slot of (layer, expert) if its table entry points at HBM, else -1. */
int32_t moe_tier_slot_of(const moe_tier *t, int32_t layer, int32_t expert);

/* ---------------------------------------------------------------------- */
/* Test support and errors                                                 */
/* ---------------------------------------------------------------------- */

/* Dequantise one expert block to fp32 gate [I][H], up [I][H], down [H][I]
 * (each weight is e2m1(code) * scale, exact in fp32). For bit-exact checks
 * of the decode used by every kernel. */
int moe_dequant_block(const moe_desc *d, const void *block, float *gate, float *up, float *down, void *stream);

/* Static description of a status code. */
const char *moe_status_string(int status);

/* Detail of the last error returned on the calling thread ("" if none). */
const char *moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP4_H */
