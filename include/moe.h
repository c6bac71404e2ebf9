/*
 * moe.h -- C ABI of the routed mixture-of-experts FFN layer over block-quantized
 * expert weights, for one AMD Instinct MI355X (gfx950).
 *
 * The layer is the one the Strata pages describe: a router scores the 512
 * experts of a layer and each token is sent to the 10 best; shared experts run
 * for every token ("Strata - the details", section "How it works"; the Strata
 * README, "How does it work?"); every expert is three matrices, its gate, up and
 * down rows ("Strata - the details", "Low-RAM mode without experts.bin"), stored
 * as 2-bit or 3-bit block-quantized packs ("Speed (measured)", "Which model?").
 * It runs over decode verify windows of a few tokens ("How it works":
 * speculation) and over prefill chunks of up to 8,192 tokens ("Faster prompts").
 *
 * Conventions shared by every call
 *   - Every buffer pointer is a DEVICE pointer (HBM), unless a comment says
 *     otherwise. The caller allocates and owns every buffer; the library never
 *     allocates device memory and keeps no pointer after a call returns, except
 *     the weight planes a moe_experts handle refers to.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls validate their arguments on the host, enqueue kernels on `stream`
 *     and return without synchronising. Results are ready when the stream is.
 *   - Return value: MOE_OK, or a negative moe_status. Argument errors are
 *     detected on the host before anything is enqueued; nothing is written then.
 *     MOE_ERR_HIP means a kernel launch failed (hipGetLastError); faults inside
 *     a kernel surface at the caller's next synchronisation of the stream.
 *   - Element counts are int32; sizes in bytes are size_t.
 *   - No compute call keeps global state (the opt-in launch profiler below is
 *     the one exception); calls on different streams may run concurrently as
 *     long as they do not share output or workspace buffers.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------- */
#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1) /* a size, pointer or enum is out of range     */
#define MOE_ERR_UNSUPPORTED (-2) /* valid, but outside what the kernels handle */
#define MOE_ERR_WORKSPACE (-3)   /* workspace smaller than the *_size() query  */
#define MOE_ERR_HIP (-4)         /* a HIP runtime call or launch failed         */

/* ---- enums -------------------------------------------------------------- */
#define MOE_F32 0  /* activations x and output y are float32               */
#define MOE_BF16 1 /* activations x and output y are bfloat16 (uint16 bits) */
#define MOE_MX4 4  /* rows of microscaled 4-bit blocks (moe_mx4_* calls only)  */

#define MOE_Q2 2 /* 2-bit codes, w = d*q + m, q in 0..3, 32-weight blocks */
#define MOE_Q3 3 /* 3-bit codes, w = d*q + m, q in 0..7, 32-weight blocks */

/* FFN compute modes.
 * MOE_FAST: matrix cores with fp32 accumulation. Gate/up: weights dequantised
 *   to fp16 (one rounding of d*q + m) times the activations in fp16, each token
 *   row first scaled by its own power of two 2^-e (its largest |x| lands in
 *   [4, 8)), which is exact for bf16 rows; the epilogue multiplies g and u by
 *   2^e again before SwiGLU. h = silu(g) * u is rounded to bf16. Down: weights
 *   dequantised to bf16 times bf16 h. y is rounded to the activation dtype.
 *   So neither x nor h is limited to fp16's range: every finite bf16 or fp32
 *   activation row is handled at its own scale (values below 2^-12 of their
 *   row's largest turn fp16-subnormal and lose low bits). Some experts of
 *   batches of up to 256 tokens run an exact-code dot on bf16 activations
 *   instead. Expected agreement with an exact evaluation: a few 1e-3 relative
 *   L2 per token row.
 * MOE_CHECK_F32: every step in fp32 on the vector ALUs (parity mode); y is
 *   always float32. Agreement about 1e-6. */
#define MOE_FAST 0
#define MOE_CHECK_F32 2

/* ---- limits ------------------------------------------------------------- */
#define MOE_MAX_E 2048 /* routed experts per layer */

/* ---- routing ------------------------------------------------------------ */

/* Router scores in front of the top-k: the product of each token's hidden
 * state with every expert's router row ("Strata - the details", "How it
 * works": routers stay on the GPU and pick the experts that score highest).
 *   logits[t][e] = sum_h x[t][h] * w[e][h] (+ bias[e] when bias != NULL)
 * x: [T][H], float32 (xdtype MOE_F32) or bf16 (MOE_BF16), 16-byte aligned.
 * w: [E][H] bf16 (row e = expert e's router row), 16-byte aligned.
 * bias: [E] float32 or NULL.  logits: [T][E] float32.
 * Products of bf16 values are exact in float32; sums are float32 in a fixed
 * order (reproducible run to run; with bf16 x, at least 256 tokens and E a
 * multiple of 128 the order is the matrix cores', else a lane split of H).
 * Requires H % 256 == 0, H <= 4096, 1 <= E <= MOE_MAX_E, T >= 0 (T == 0: no
 * launch). The result feeds moe_route_topk, moe_route_group or moe_layer. */
int moe_router_logits(const void *x, int32_t xdtype, int32_t T, int32_t H, const uint16_t *w,
                      const float *bias, int32_t E, float *logits, void *stream);

/* Top-k expert selection and gates, per token.
 *
 * Per token t (the router step of "How it works"; 10 of 512 experts per token):
 *   idx[t][0..k-1]  = the k experts with the largest logits, in descending rank;
 *                     equal logits (IEEE equality, +0 == -0) go to the lower
 *                     expert index; NaN ranks below every number.
 *   gates[t][j]     = exp(l_j - l_0) / sum_{j'<k} exp(l_j' - l_0), l_j the
 *                     logit of idx[t][j]: a softmax over the selected logits,
 *                     equal to a softmax over all E renormalised over the top k.
 * logits: [T][E] float32, row-major.  idx: [T][k] int32.  gates: [T][k] float32.
 * Requires 1 <= E <= MOE_MAX_E, 1 <= k <= E, T >= 0 (T == 0: no launch).
 * Gates are finite when the selected logits are finite. */
int moe_route_topk(const float *logits, int32_t T, int32_t E, int32_t k, int32_t *idx,
                   float *gates, void *stream);

/* ---- grouping ----------------------------------------------------------- */

/* Workspace bytes moe_group needs for these sizes (device memory, any content). */
size_t moe_group_workspace_size(int32_t T, int32_t k, int32_t E);

/* Stable grouping of the token-to-expert assignments by expert (a counting sort;
 * the pages' prefill groups the chunk's tokens per expert before the expert
 * matrices run: "Faster prompts").
 *
 * Assignment ids: routed assignment (t, j) has id t*k + j; with has_shared, the
 * shared expert's assignment of token t has id T*k + t and belongs to group E.
 * A = T*(k + has_shared) assignments in all.
 *   counts [E+1]  : assignments per expert (counts[E] = T with a shared expert, else 0)
 *   offsets[E+2]  : exclusive prefix sum of counts; offsets[E+1] = A
 *   perm   [A]    : the assignment ids of group e at perm[offsets[e] .. offsets[e+1]),
 *                   in ascending id order (so ascending token order)
 *   slot_of[A]    : inverse of perm: perm[slot_of[a]] == a
 * idx [T][k] int32, every entry in [0, E). Entries outside that range are not
 * detected; the kernels stay in bounds and skip them, and the affected outputs
 * are unspecified.
 * ws: device scratch of at least moe_group_workspace_size(T, k, E) bytes. */
int moe_group(const int32_t *idx, int32_t T, int32_t k, int32_t E, int32_t has_shared,
              int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *slot_of, void *ws,
              size_t ws_bytes, void *stream);

/* Top-k routing followed by the grouping, in one call: the same results as
 * moe_route_topk then moe_group (idx, gates, counts, offsets, perm, slot_of as
 * defined there). Small batches (T <= 16 and T*k <= 1024, e.g. decode verify
 * windows) run as one workgroup in a single launch; larger ones run the two
 * steps' kernels back to back. ws: at least moe_group_workspace_size(T, k, E)
 * bytes. T == 0 writes the empty grouping (counts, offsets) only. */
int moe_route_group(const float *logits, int32_t T, int32_t E, int32_t k, int32_t has_shared,
                    int32_t *idx, float *gates, int32_t *counts, int32_t *offsets, int32_t *perm,
                    int32_t *slot_of, void *ws, size_t ws_bytes, void *stream);

/* ---- experts ------------------------------------------------------------ */

/* An immutable description of one layer's packed experts. The handle is a small
 * host object; it refers to the caller's device planes, which must stay alive
 * and unchanged until moe_experts_destroy.
 *
 * Packed layout (fixed by this library; the pages publish none):
 *   experts 0..E-1 routed, then the shared expert (index E) when has_shared;
 *   each expert holds NB = 3*H*I/32 blocks of 32 weights: its gate matrix [I][H],
 *   then up [I][H], then down [H][I], each row-major with blocks along a row.
 *   codes: NB * 8 bytes per expert. Weight j (0..31) of a block is in byte j/4 at
 *          bits 2*(j%4) (the low two bits of the code for Q3).
 *   hi   : Q3 only, NB * 4 bytes per expert; bit j of the block's little-endian
 *          32-bit word is bit 2 of code j. Pass NULL for Q2.
 *   dm   : NB * 2 uint16 per expert: fp16 bits of d, then of m, per block.
 *   Weight value: w = d*q + m.
 * Plane bases must be 16-byte aligned. Requires H a multiple of 256 and I a
 * multiple of 128 (the matrix-core tile: 256 output rows of the down
 * projection, 128 rows each of gate and up), 1 <= E <= MOE_MAX_E; other
 * shapes return MOE_ERR_UNSUPPORTED. The decode GEMV kernels cover H/32 and
 * I/32 in {4, 8, 16, 32, 64}; other shapes run every expert on the
 * matrix-core tiles. */
typedef struct moe_experts moe_experts;

int moe_experts_create(moe_experts **out, int32_t qtype, int32_t E, int32_t has_shared,
                       int32_t H, int32_t I, const void *codes, const void *hi,
                       const void *dm);
int moe_experts_destroy(moe_experts *ex);

/* Optional second copy of the weights, in the order in which the prefill
 * matrix-core tiles read them, so that every wave's weight loads are
 * contiguous (the canonical planes give one 16-byte piece per weight row).
 * The pages' prompt path likewise runs on quantised expert data in kernel-
 * friendly form ("Strata - the details", "Faster prompts"); the arrangement
 * here is this library's own.
 *
 * moe_experts_tiled_size: bytes of the copy (the same as the codes, hi and dm
 *   planes together), or 0 for a null handle.
 * moe_experts_attach_tiled: enqueues on `stream` a device kernel that writes
 *   the copy into buf (device memory owned by the caller, at least
 *   moe_experts_tiled_size bytes, 16-byte aligned) from the canonical planes,
 *   and records buf in the handle; from then on moe_ffn_q and moe_layer run
 *   their matrix-core tiles on it (same results up to fp32 summation order).
 *   buf == NULL detaches. The caller keeps buf alive and unchanged until it
 *   detaches or destroys the handle, and must not call this while other calls
 *   on the handle are in flight on other streams.
 * Layout of the copy: codes [E_tot][3 matrices][R][64 lanes][16 bytes], then
 *   dm [E_tot][3][R][64][4 uint16], then (Q3) hi [E_tot][3][R][64][8 bytes],
 *   R = H*I/4096 records per matrix: for 32-row group g (rows 32g..32g+31 of
 *   the matrix) and block quad p (blocks 4p..4p+3 of each row), record
 *   g * (K/128) + p (K = the matrix's row length) holds for lane l the blocks
 *   4p + l/32 and 4p + 2 + l/32 of row 32g + l%32.
 * Errors: MOE_ERR_INVALID_ARG for a null handle, a misaligned buf or
 *   bytes below the size; MOE_ERR_HIP if the kernel launch fails. */
size_t moe_experts_tiled_size(const moe_experts *ex);
int moe_experts_attach_tiled(moe_experts *ex, void *buf, size_t bytes, void *stream);

/* ---- expert FFN and combine ---------------------------------------------- */

/* Workspace bytes moe_ffn_q needs for T tokens, k experts per token, `mode`,
 * including room for the grouping when the caller does not pass one. */
size_t moe_ffn_q_workspace_size(const moe_experts *ex, int32_t T, int32_t k, int32_t mode);

/* The routed expert FFN with gate-weighted combine, for T tokens.
 *
 * For every token t (expert = gate/up/down rows, "Low-RAM mode without
 * experts.bin"; shared experts for every token, "How it works"):
 *   o(e, x) = Wd_e . ( silu(Wg_e . x) * (Wu_e . x) ),   silu(z) = z / (1 + e^-z)
 *   y[t]    = sum_{j<k} gates[t][j] * o(idx[t][j], x[t])  +  o(shared, x[t])
 * with every weight dequantised as w = d*q + m from the handle's planes.
 *
 * x     : [T][H], dtype xdtype (MOE_F32 or MOE_BF16).
 * idx   : [T][k] int32 in [0, E); gates: [T][k] float32 (any values).
 * counts/offsets/perm/slot_of: a grouping of idx exactly as moe_group writes
 *         it, or all four NULL to have it computed inside `ws`.
 * y     : [T][H]; dtype xdtype in MOE_FAST, float32 in MOE_CHECK_F32.
 * ws    : device scratch of at least moe_ffn_q_workspace_size(ex, T, k, mode).
 * T == 0 is valid and launches nothing.
 *
 * Execution (fast mode; results agree within the FFN tolerance whichever form
 * runs): below 256 tokens with H 1024 or 2048 and I 256 or 512, every touched
 * expert runs on the small-batch matrix-core kernels (work items of expert,
 * output rows and 16 of its tokens); other batches below 256 tokens run
 * experts with 1..4 assignments on the GEMV kernels and the rest on the
 * matrix-core tiles; from 256 tokens on every expert runs on the tiles. */
int moe_ffn_q(const void *x, int32_t xdtype, int32_t T, const moe_experts *ex,
              const int32_t *idx, const float *gates, int32_t k, const int32_t *counts,
              const int32_t *offsets, const int32_t *perm, const int32_t *slot_of, void *y,
              int32_t mode, void *ws, size_t ws_bytes, void *stream);

/* ---- whole layer ---------------------------------------------------------- */

/* Workspace bytes moe_layer needs (device scratch). */
size_t moe_layer_workspace_size(const moe_experts *ex, int32_t T, int32_t k, int32_t mode);

/* The whole routed MoE layer in one call: top-k routing of `logits` ([T][E]
 * f32), the grouping, the expert FFN and the combine, writing idx and gates
 * ([T][k]) and y ([T][H]). Results match moe_route_group followed by
 * moe_ffn_q within the FFN tolerance (idx and gates identically).
 *
 * A decode verify window ("Strata - the details", "How it works": the drafted
 * tokens are checked in one pass) is fast mode with T <= 4, k <= 64 and H/32,
 * I/32 in {4..64}. With H a multiple of 1024 up to 4096, I 256 or 512,
 * E <= 512, T k <= 64 and T k + T (with a shared expert; T k without) at most
 * 32768 / I - 1 (the routed rows of h that the down rows hold at once: 63 at
 * I = 512, so k <= 14 at T = 4) it runs as ONE kernel: every workgroup routes the
 * window itself; the first workgroups compute gate/up rows, the others down
 * rows once counters at the head of `ws` show every gate/up row released; y is
 * reproducible run to run. Other windows run as two kernels (gate/up, then
 * down); other calls run moe_route_group then moe_ffn_q inside the workspace.
 *
 * ws: at least moe_layer_workspace_size(ex, T, k, mode) bytes. Its first 8192
 * bytes (the head) must be zero before the first call that uses it (a
 * zero-filled allocation). The one-kernel window keeps counters there that
 * count over all calls on the workspace; every call leaves them in a state the
 * next call can start from, also when a wait timed out; no other form of the
 * call writes the head, so one zeroed workspace serves every shape. Calls that
 * overlap in time must not share a workspace. A head whose first 128 bytes are
 * not zero shows as NaN in the window's y; a down row that waits longer than
 * about 0.2 s for the gate/up rows gives up and becomes NaN. Bytes 128..131 of
 * the head may hold a shorter bound on that wait, in ticks of the 100 MHz wall
 * clock (0 = the default); this exists for testing the timeout path. */
int moe_layer(const float *logits, const void *x, int32_t xdtype, int32_t T, const moe_experts *ex,
              int32_t k, int32_t *idx, float *gates, void *y, int32_t mode, void *ws,
              size_t ws_bytes, void *stream);

/* Router product and top-k in one launch, for many bf16 tokens: the logits of
 * moe_router_logits (written to `logits` [T][E] when not NULL) and their top-k
 * and gates as moe_route_topk ("Strata - the details", "How it works": the
 * router picks the experts that score highest), with no logits round trip
 * through memory between the two. x: [T][H] bf16 (xdtype MOE_BF16), w: [E][H]
 * bf16, both 16-byte aligned; bias: [E] float32 or NULL; idx, gates: [T][k].
 * The logits are f32 sums of exact bf16 products (matrix cores, a fixed
 * order), so idx and gates are exactly moe_route_topk of the logits written.
 * Each workgroup takes 32 tokens against every expert, so it reads the whole
 * router matrix from cache: measured at 8,192 tokens x 512 experts x 2,048 it
 * takes about 1.7 times as long as moe_router_logits followed by
 * moe_route_topk (which read the matrix once per 128 tokens); the layer calls
 * use those two.
 * Requires H % 256 == 0, H <= 4096, E 256 or 512, 1 <= k <= 64 (else
 * MOE_ERR_UNSUPPORTED); T == 0: no launch. */
int moe_router_topk(const void *x, int32_t xdtype, int32_t T, int32_t H, const uint16_t *w,
                    const float *bias, int32_t E, int32_t k, int32_t *idx, float *gates, float *logits,
                    void *stream);

/* ---- whole layer from hidden states --------------------------------------- */

/* Workspace bytes moe_layer_hidden needs: moe_layer's plus room for the
 * logits ([T][E] float32). */
size_t moe_layer_hidden_workspace_size(const moe_experts *ex, int32_t T, int32_t k, int32_t mode);

/* The layer from the tokens' hidden states: the router product
 * (moe_router_logits: logits[t][e] = x[t] . w_router[e] (+ bias[e]); "Strata -
 * the details", "How it works": each layer's router runs on the GPU in front
 * of its experts), then moe_layer on those logits. x: [T][H] as for moe_layer
 * (also the router's input); w_router: [E][H] bf16 (16-byte aligned); bias:
 * [E] float32 or NULL; logits: [T][E] float32 output, or NULL to keep them in
 * the workspace. idx, gates, y, mode and the workspace head as moe_layer; ws at
 * least moe_layer_hidden_workspace_size bytes.
 *
 * A decode window that moe_layer runs as one kernel runs here as one kernel
 * too: its first E / 16 workgroups compute the logits (an f32 sum of H
 * products per entry, in a fixed order) and store them; the other workgroups
 * wait for them through counters in the head (bounded like the window's other
 * wait; a wait that runs out makes y NaN and idx 0 .. k-1) and route from
 * them. Other calls launch the router product and then moe_layer (for many
 * tokens that is faster than moe_router_topk's single launch, see there). In
 * every form idx and gates are the top-k of the logits written.
 * Requires what moe_router_logits requires of H and E (else
 * MOE_ERR_UNSUPPORTED); other errors as moe_layer. */
int moe_layer_hidden(const void *x, int32_t xdtype, int32_t T, const uint16_t *w_router,
                     const float *bias, const moe_experts *ex, int32_t k, int32_t *idx, float *gates,
                     void *y, float *logits, int32_t mode, void *ws, size_t ws_bytes, void *stream);

/* ---- one expert's gate/up on the FP8 matrix cores (measured variant) -------- */

/* Workspace bytes moe_expert_gateup_fp8 needs for T tokens. */
size_t moe_expert_gateup_fp8_workspace_size(const moe_experts *ex, int32_t T);

/* h[t][r] = silu(g) * u of expert `expert` (0 .. E + has_shared - 1) for every
 * token row of x ([T][H] bf16, 16-byte aligned), g and u its gate and up
 * products: the analogue of the pages' 8-bit tensor-core prompt kernels
 * ("Strata - the details", "Speed (measured)") on the gfx950 FP8 matrix
 * cores, kept as a measured variant beside the layer's fp16 prefill tiles.
 * The codes enter the matrix cores as exact E4M3 values; each token row is
 * scaled by a power of two and split into two E4M3 parts (hi + lo, about 8
 * significant bits together); one product per 32-weight block, and d and m are
 * applied per block in fp32. h: [T][I] float32. Requires H % 64 == 0,
 * H <= 4096 and I % 32 == 0 (else MOE_ERR_UNSUPPORTED). ws: at least
 * moe_expert_gateup_fp8_workspace_size bytes (no zeroing needed); it holds the
 * E4M3 operands. Other errors as moe_ffn_q. */
int moe_expert_gateup_fp8(const void *x, int32_t T, const moe_experts *ex, int32_t expert, float *h,
                          void *ws, size_t ws_bytes, void *stream);

/* ---- microscaled 4-bit operands ------------------------------------------- */

/* A matrix of R rows of K values as microscaled 4-bit blocks, B = ceil(K / 32)
 * blocks a row, each 32 consecutive values of it (the last may hold fewer):
 *   codes : [R][B][16] bytes. Value j (0..31) of a block is in byte j/2, at bits
 *           4*(j%2); bit 3 of its code is the sign, bits 0..2 pick the magnitude
 *           0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   scales: [R][B] bytes. Byte s stands for 2^(s - 127); the value is the signed
 *           magnitude times that. s = 255: every value of the block is NaN.
 * Codes past K in a row's last block are zero. codes is 16-byte aligned.
 * In every moe_mx4_* call results and workspace share no memory with one another
 * or with the operands (MOE_ERR_INVALID_ARG). N and K are at most 2^19, the rows
 * of a product at most 2^22, and row distances at most 2^40 elements
 * (MOE_ERR_UNSUPPORTED). */

/* Quantises x ([rows][K], MOE_F32 or MOE_BF16, ld elements from row to row,
 * ld >= K). The scale of a block is the power of two that brings its largest
 * magnitude into [4, 8): byte floor(log2 max) - 2 + 127, at least 0 (also for a
 * block of zeros). Magnitudes over the scale go to the nearest of the eight,
 * ties to the even code, past 6 to 6; zeros keep their sign. A block that holds
 * a NaN or an infinity becomes NaN (byte 255, codes 0). rows == 0: no launch. */
int moe_mx4_quantize(const void *x, int32_t xdtype, int64_t ld, int32_t rows, int32_t K,
                     uint8_t *codes, uint8_t *scales, void *stream);

/* The values that codes and scales stand for: y [rows][K], MOE_F32 or MOE_BF16,
 * both exact (magnitudes from 2^128 on are infinite). */
int moe_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t K,
                       int32_t ydtype, void *y, void *stream);

/* y[t][n] = sum_k x[t][k] * W[n][k] for T rows and one microscaled matrix W of
 * N rows of K values.
 *   x  : [T][K], MOE_F32 or MOE_BF16, ldx elements from row to row (>= K), or
 *        MOE_MX4: codes, with their scales in x_scales (ldx is not used).
 *        x_scales is NULL for the other types.
 *   y  : [T][N], MOE_F32 or MOE_BF16.
 * Every product is exact (float32 x enters the matrix cores as three bf16
 * parts; |x| below 2^-110 loses its bits below 2^-133); sums are float32 in a
 * fixed order, with one rounding to y's type. So results are reproducible run to
 * run. Weights of 2^128 and more (scale bytes 253 and 254, which moe_mx4_quantize
 * never writes) are infinite: results that they reach are infinite or NaN with
 * MOE_BF16 rows, as the arithmetic of infinities has it, and one of the two with
 * MOE_F32 rows. With MOE_MX4 rows they are what they are. T == 0: no launch. */
int moe_mx4_matmul(const void *x, const uint8_t *x_scales, int32_t xdtype, int64_t ldx, int32_t T,
                   const uint8_t *w_codes, const uint8_t *w_scales, int32_t N, int32_t K, void *y,
                   int32_t ydtype, void *stream);

/* The gradient of moe_mx4_matmul for its rows: dx[t][k] = sum_n dy[t][n] *
 * W[n][k]. dy: [T][N], MOE_F32 or MOE_BF16, ldd elements from row to row (>= N);
 * dx: [T][K], MOE_F32 or MOE_BF16. The matrix is not trained: it has no
 * gradient. */
int moe_mx4_matmul_backward(const void *dy, int32_t dtype, int64_t ldd, int32_t T,
                            const uint8_t *w_codes, const uint8_t *w_scales, int32_t N, int32_t K,
                            void *dx, int32_t dxdtype, void *stream);

/* Workspace bytes moe_mx4_experts_matmul needs (0 for a few rows). */
size_t moe_mx4_experts_matmul_workspace_size(int32_t T, int32_t k, int32_t has_shared);

/* The same products for rows grouped by expert (moe_group, moe_route_group):
 * row s of [offsets[e], offsets[e+1]) is multiplied by matrix e of the E_tot =
 * E + has_shared matrices (w_codes [E_tot][N][B][16], w_scales [E_tot][N][B];
 * the shared expert's last). A = T*(k + has_shared) rows.
 *   gather == 0: x holds the A rows in the groups' order.
 *   gather == 1: x holds T rows, one a token; row s of the groups is the row of
 *                the token of assignment perm[s].
 *   y     : [A][N] in the groups' order. Rows that are in no group (from
 *           offsets[E_tot] on) are left as they were.
 * E_tot is at most MOE_MAX_E + 1.
 * offsets: [E_tot + 1] (moe_group writes one more), perm: [A]; perm may be NULL
 * when gather == 0. Values of perm outside [0, A) are not detected; the kernels
 * stay in bounds and the results of those rows are unspecified. offsets must not
 * decrease; each counts as cut to [0, A]. Types and rounding as
 * moe_mx4_matmul. ws: at least ..._workspace_size bytes (any content, 16-byte
 * aligned); calls that overlap in time must not share it. Results do not depend
 * on which workgroup takes which rows. */
int moe_mx4_experts_matmul(const void *x, const uint8_t *x_scales, int32_t xdtype, int64_t ldx,
                           int32_t T, int32_t k, int32_t E, int32_t has_shared, int32_t gather,
                           const int32_t *offsets, const int32_t *perm, const uint8_t *w_codes,
                           const uint8_t *w_scales, int32_t N, int32_t K, void *y, int32_t ydtype,
                           void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes moe_mx4_experts_matmul_backward needs. */
size_t moe_mx4_experts_matmul_backward_workspace_size(int32_t T, int32_t k, int32_t has_shared,
                                                      int32_t K, int32_t gather);

/* The gradient of moe_mx4_experts_matmul for its rows. dy: [A][N] in the
 * groups' order, ldd elements from row to row.
 *   gather == 0: dx [A][K]; rows in no group are left as they were.
 *   gather == 1: dx [T][K]; the sum over the token's assignments, in the order
 *                j = 0 .. k-1, then the shared expert's, kept in float32 in ws
 *                ([A][K]) and rounded once. slot_of: [A] as moe_group writes it
 *                (else it may be NULL); values outside [0, A), and rows in no
 *                group, add nothing.
 * ws: at least ..._workspace_size bytes (any content, 16-byte aligned); calls
 * that overlap in time must not share it. */
int moe_mx4_experts_matmul_backward(const void *dy, int32_t dtype, int64_t ldd, int32_t T, int32_t k,
                                    int32_t E, int32_t has_shared, int32_t gather,
                                    const int32_t *offsets, const int32_t *slot_of,
                                    const uint8_t *w_codes, const uint8_t *w_scales, int32_t N,
                                    int32_t K, void *dx, int32_t dxdtype, void *ws, size_t ws_bytes,
                                    void *stream);

/* ---- balance loss ------------------------------------------------------------ */

/* Workspace bytes moe_balance_loss needs (device memory, any content). */
size_t moe_balance_loss_workspace_size(int32_t T, int32_t k, int32_t E);

/* Per-expert counts of a routed batch, and the two losses that keep a router in
 * shape. Over the n tokens that `mask` keeps (mask [T] bytes, 0 = left out;
 * NULL: all T), p[t] the softmax of the token's E logits, lse[t] the logarithm
 * of the sum of their exponentials:
 *   counts[e] = entries of idx[t][0..k-1] equal to e, over the kept tokens
 *               (entries outside [0, E) count nowhere)
 *   kept[0]   = n
 *   losses[0] = E * sum_e (counts[e] / (n k)) * (sum_t p[t][e] / n)   (balance)
 *   losses[1] = sum_t lse[t]^2 / n                                    (z)
 * n == 0: both are 0. A token whose logits are all -inf has no distribution: its
 * p and lse count as 0. NaN and +inf logits of a kept token make the losses
 * NaN; those of a token left out are not looked at.
 * logits: [T][E], MOE_F32 or MOE_BF16, ld elements from row to row (>= E); idx:
 * [T][k] int32 (moe_route_topk); counts: [E] int32; kept: [1] int32; losses: [2]
 * float32. Sums are float32 in a fixed order: reproducible run to run.
 * Requires 1 <= E <= MOE_MAX_E, k >= 1, T*k <= 2^30; T == 0 writes n = 0 and zeros.
 * ws: at least moe_balance_loss_workspace_size bytes, any content; calls that
 * overlap in time must not share it. */
int moe_balance_loss(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t k,
                     const int32_t *idx, const uint8_t *mask, float *losses, int32_t *counts,
                     int32_t *kept, void *ws, size_t ws_bytes, void *stream);

/* The gradient for the logits: dlogits [T][E] (type and rows as `dtype`, rows E
 * elements apart), from counts and kept as moe_balance_loss wrote them and the
 * gradients d_losses [2] (float32, device) of the two losses:
 *   dlogits[t][e] = p[t][e] * (d_losses[0] * E / n * (f[e] - sum_j f[j] p[t][j])
 *                              + d_losses[1] * 2 * lse[t] / n),
 * f[e] = counts[e] / (n k) (counts depend on idx alone and pass no gradient).
 * Rows of tokens that mask leaves out are 0. dlogits may be the logits themselves
 * (where ld == E), and shares no memory with them otherwise. T == 0: no launch. */
int moe_balance_loss_backward(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                              int32_t k, const uint8_t *mask, const int32_t *counts,
                              const int32_t *kept, const float *d_losses, void *dlogits,
                              void *stream);

/* ---- routing by scores -------------------------------------------------------- */

#define MOE_SIGMOID 0 /* score of an expert: 1 / (1 + exp(-logit))          */
#define MOE_SOFTMAX 1 /* exp(logit) / sum of exp(logit) over all E experts  */

/* Top-k selection and gates from scores, with a bias that takes part in the
 * selection alone and with groups of experts. Per token:
 *   s[e] = the score of logits[t][e];  c[e] = s[e] + bias[e] (bias NULL: 0)
 *   The E experts lie in `groups` groups of E / groups neighbours. A group's value
 *   is the sum of its group_top (1 or 2) largest c; the `keep` groups of the
 *   largest values stay, equal values in favour of the lower group.
 *   idx[t][0..k-1]  = the k experts of the kept groups with the largest c, in
 *                     descending rank, equal c in favour of the lower index.
 *   gates[t][j]     = scale * s[idx_j], with renorm != 0 over the sum of the k
 *                     selected scores (0 where that sum is 0; small scores are taken in 64
 *                     bits, in which a sigmoid is 0 from a logit of about -709 down, and a
 *                     softmax from about 745 below the row's largest logit down).
 * Groups and experts are ranked by values in 64 bits, so that the order does not
 * depend on how scores are rounded to 32 (without a bias by the logits themselves,
 * which have the same order). An expert whose logit or bias is -inf is switched off:
 * it comes behind every other (in a group's sum it is left out; a group that has no other
 * comes behind every other group), with its score, 0 where the logit is -inf. A
 * c that is NaN ranks below -inf. Of a token whose logits are all -inf every score
 * is 0. Softmax scores of a token with a NaN or +inf logit are NaN: its gates
 * are NaN, its indices distinct and in range.
 * logits: [T][E], MOE_F32 or MOE_BF16, ld elements from row to row (>= E); bias:
 * [E] float32 or NULL; idx: [T][k] int32; gates: [T][k] float32.
 * Requires E % groups == 0, 1 <= keep <= groups <= 64, group_top 1 or 2,
 * 1 <= k <= keep * E / groups, E <= MOE_MAX_E, T <= 2^22, scale finite. Results share no
 * memory with one another or with the operands (MOE_ERR_INVALID_ARG), here and in every
 * call down to moe_fp8_experts_matmul_backward, where nothing else is said. T == 0: no launch. */
int moe_route_scores(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                     const float *bias, int32_t score, int32_t groups, int32_t keep,
                     int32_t group_top, int32_t k, int32_t renorm, float scale, int32_t *idx,
                     float *gates, void *stream);

/* The gradient of moe_route_scores' gates for the logits, from idx as it wrote
 * them and the gates' gradient d_gates [T][k] (float32). The selection itself, and so
 * the bias, passes none. With S the sum of the selected scores, d = scale * d_gates, and for
 * renorm d := (d_j - sum_i d_i s_i / S) / S (0 where S is 0: of sigmoids as in moe_route_scores, of
 * a softmax, whose ratios the selected logits alone give, where those are all -inf):
 *   sigmoid: dlogits[t][idx_j] = d_j s_j (1 - s_j), 0 elsewhere
 *   softmax: dlogits[t][e]     = s_e ((sum of d_j over idx_j = e) - sum_i d_i s_i)
 * An index that appears twice in a row counts twice; one outside [0, E) is not
 * there. dlogits: [T][E] in the logits' type, rows E elements apart. A token's
 * NaN logits make its gradient NaN where they enter. k <= MOE_MAX_E. */
int moe_route_scores_backward(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                              int32_t k, int32_t score, int32_t renorm, float scale,
                              const int32_t *idx, const float *d_gates, void *dlogits, void *stream);

/* ---- 8-bit rows and matrices ---------------------------------------------------- */

/* Values in 8 bits: E4M3 codes (sign, 4 exponent bits with bias 7, 3 bits of
 * mantissa; largest 448, 0x7F and 0xFF are NaN, no infinities) and a float32
 * scale for each block; a value is its code's times the scale. B = ceil(K / 128).
 *   codes : rows of 128 B bytes, one a value; codes past K are zero. 16-byte aligned.
 *   scales: of rows (activations) [R][B], one for 128 consecutive values of a row;
 *           of a matrix [ceil(N / 128)][B], one for 128 rows by 128 columns.
 * Several matrices ([E_tot][N][K]) have codes [E_tot][N][128 B] and scales
 * [E_tot][ceil(N / 128)][B]. N and K are at most 2^19, the rows of a product at most
 * 2^22, and row distances at most 2^40 elements (MOE_ERR_UNSUPPORTED). */

/* Quantises x (`mats` matrices of [rows][K], MOE_F32 or MOE_BF16, ld elements from row
 * to row, rows * ld from matrix to matrix). block_rows is 1 (rows) or 128
 * (matrices). scale = max(largest magnitude of the block, 2^-116) / 448 in float32;
 * code = x / scale, the exact quotient rounded once to the nearest code, ties to
 * the even one; zeros keep their sign. A block that holds a NaN or an infinity becomes
 * NaN (scale NaN, codes 0). Matrices of 2^24 blocks and more together: MOE_ERR_UNSUPPORTED.
 * mats == 0 or rows == 0: no launch. */
int moe_fp8_quantize(const void *x, int32_t xdtype, int64_t ld, int32_t mats, int32_t rows, int32_t K,
                     int32_t block_rows, uint8_t *codes, float *scales, void *stream);

/* The values that codes and scales stand for, rounded once to ydtype: y [mats][rows][K],
 * MOE_F32 or MOE_BF16. */
int moe_fp8_dequantize(const uint8_t *codes, const float *scales, int32_t mats, int32_t rows, int32_t K,
                       int32_t block_rows, int32_t ydtype, void *y, void *stream);

/* y[t][n] = sum_k x[t][k] W[n][k] for T 8-bit rows and one 8-bit matrix of N rows of
 * K values. y: [T][N], MOE_F32 or MOE_BF16. Blocks of 128 columns are added up in
 * float32, each scaled by its two scales, in a fixed order (reproducible run to
 * run). For MOE_F32 results every product of two codes is exact and their sum is float32; for
 * MOE_BF16 the 8-bit matrix cores add up a block's 128 products, which drop of each what
 * lies under 2^-13 of the binade of the block's largest product: less than 2^-12 of that one a
 * product, 2^-5 a block (2e-4 of the norm of rows of normal values, an eighth of what bf16's
 * rounding does). Blocks whose large products cancel may lose their small ones; where they
 * count, ask for MOE_F32. A block's sum is multiplied by the float32 product of its two scales, so
 * blocks whose largest values' product passes 2^145 give infinities or NaN, and where it is
 * below 2^-108 lose bits. T == 0: no launch. */
int moe_fp8_matmul(const uint8_t *x_codes, const float *x_scales, int32_t T, const uint8_t *w_codes,
                   const float *w_scales, int32_t N, int32_t K, void *y, int32_t ydtype, void *stream);

/* The gradient of moe_fp8_matmul for its rows: dx[t][k] = sum_n dy[t][n] W[n][k].
 * dy: 8-bit rows of N values (a scale for 128 of them), dx: [T][K], MOE_F32 or MOE_BF16.
 * Codes of dy past N are zero. Products and sums as in moe_fp8_matmul. The matrix is not
 * trained in 8 bits: it has no gradient here. */
int moe_fp8_matmul_backward(const uint8_t *dy_codes, const float *dy_scales, int32_t T,
                            const uint8_t *w_codes, const float *w_scales, int32_t N, int32_t K,
                            void *dx, int32_t dxdtype, void *stream);

/* The same products for rows grouped by expert: arguments, groups, `gather`, rows in no
 * group and bad ids as in moe_mx4_experts_matmul. x: [A] 8-bit rows in the groups'
 * order (gather == 0), or [T], one a token (gather == 1). It needs no workspace. */
int moe_fp8_experts_matmul(const uint8_t *x_codes, const float *x_scales, int32_t T, int32_t k,
                           int32_t E, int32_t has_shared, int32_t gather, const int32_t *offsets,
                           const int32_t *perm, const uint8_t *w_codes, const float *w_scales,
                           int32_t N, int32_t K, void *y, int32_t ydtype, void *stream);

/* Workspace bytes moe_fp8_experts_matmul_backward needs. */
size_t moe_fp8_experts_matmul_backward_workspace_size(int32_t T, int32_t k, int32_t has_shared,
                                                      int32_t K, int32_t gather);

/* The gradient of moe_fp8_experts_matmul for its rows, as moe_mx4_experts_matmul_backward:
 * dy: [A] 8-bit rows of N values in the groups' order; gather == 0: dx [A][K]; gather == 1:
 * dx [T][K], the sum over the token's assignments in the order j = 0 .. k-1, then the
 * shared expert's, kept in float32 in ws and rounded once. */
int moe_fp8_experts_matmul_backward(const uint8_t *dy_codes, const float *dy_scales, int32_t T, int32_t k,
                                    int32_t E, int32_t has_shared, int32_t gather,
                                    const int32_t *offsets, const int32_t *slot_of,
                                    const uint8_t *w_codes, const float *w_scales, int32_t N,
                                    int32_t K, void *dx, int32_t dxdtype, void *ws, size_t ws_bytes,
                                    void *stream);

/* ---- RMS norm --------------------------------------------------------------------- */

#define MOE_MAX_NORM_H 32768 /* values of a row of moe_rms_norm */

/* The residual's addition and the root-mean-square norm in front of a router and its
 * experts. Per row t of T:
 *   r = x[t] + residual[t] (residual NULL: x[t]), in float32
 *   total[t] = r, rounded once to dtype (total NULL: not written)
 *   v = weight * r / sqrt(mean(r^2) + eps), from r before its rounding
 *   y[t] = v rounded once to dtype (y NULL: not written)
 *   codes[t], scales[t] = v as an 8-bit row, as moe_fp8_quantize writes it (both NULL: not)
 * x, residual: [T][H], MOE_F32 or MOE_BF16, ldx and ldr elements from row to row; weight:
 * [H], MOE_F32 or MOE_BF16 (wdtype); total, y: [T][H], rows H elements apart. One of total,
 * y and codes at least is written. total may be x or residual themselves where their
 * rows are H apart. Up to 32 squares are added up in float32, their sums in 64 bits, in a fixed
 * order: magnitudes up to 2^61 stay in range. A row where squares pass float32's range
 * has mean infinity and gives 0 (and NaN where r is infinite); squares below it count as 0, and
 * with eps 0 a row of nothing else gives infinities and NaN; a NaN makes its whole row NaN. H <= MOE_MAX_NORM_H, T <= 2^22 (else
 * MOE_ERR_UNSUPPORTED), eps >= 0 and finite. T == 0: no launch. */
int moe_rms_norm(const void *x, int32_t dtype, int64_t ldx, const void *residual, int64_t ldr,
                 const void *weight, int32_t wdtype, float eps, int32_t T, int32_t H, void *total,
                 void *y, uint8_t *codes, float *scales, void *stream);

/* Workspace bytes moe_rms_norm_backward needs. */
size_t moe_rms_norm_backward_workspace_size(int32_t T, int32_t H);

/* The gradients of the norm at the rows h (moe_rms_norm's total, or its x where there was no
 * residual). With q = 1 / sqrt(mean(h^2) + eps) and dy the gradient of v (an 8-bit row passes
 * its values' gradient straight through):
 *   dh[t]   = d_total[t] + q (weight dy - h q^2 mean(weight dy h))   (d_total NULL: 0)
 *   dweight = sum over t of dy h q
 * dh is the gradient of x and of the residual alike. dy, h, d_total: [T][H] of `dtype`, ldd, ldh
 * and ldt elements from row to row; dh: [T][H] of `dtype`; dweight: [H] float32. dweight NULL: only
 * dh, no workspace. T == 0 writes dweight = 0. A row's sums are taken as in moe_rms_norm (products
 * weight dy h up to 2^122 stay in range), those over rows in float32, in a fixed order. ws: at least
 * moe_rms_norm_backward_workspace_size bytes (any content, 16-byte aligned); calls that
 * overlap in time must not share it. */
int moe_rms_norm_backward(const void *dy, int64_t ldd, const void *h, int64_t ldh, int32_t dtype,
                          const void *weight, int32_t wdtype, const void *d_total, int64_t ldt,
                          float eps, int32_t T, int32_t H, void *dh, float *dweight, void *ws,
                          size_t ws_bytes, void *stream);

/* ---- whole layer without allocation --------------------------------------- */

/* Bytes of the library's own scratch array per GPU (moe_layer_static). */
#define MOE_STATIC_SCRATCH_BYTES (16u << 20)

/* moe_layer for callers that cannot allocate device memory or pass a
 * workspace: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc. The same computation, results and kernels as moe_layer
 * (same arguments without ws/ws_bytes); the workspace is a 16 MiB array inside
 * the library, one per GPU, held until the process ends. The first call on a
 * device resolves that device's array and enqueues a small kernel on `stream`
 * that zeroes its first 8192 bytes; no call allocates or frees anything.
 * Calls whose moe_layer_workspace_size exceeds MOE_STATIC_SCRATCH_BYTES return
 * MOE_ERR_WORKSPACE before launching anything (decode windows and batches of a
 * few dozen tokens fit; 1,024-token prefill chunks do not). Every call on a GPU
 * uses that GPU's one array: calls that overlap in time on one GPU (other
 * streams, other threads) race and give undefined results; serialise them.
 * Returns MOE_ERR_HIP if the device's array cannot be resolved. */
int moe_layer_static(const float *logits, const void *x, int32_t xdtype, int32_t T,
                     const moe_experts *ex, int32_t k, int32_t *idx, float *gates, void *y,
                     int32_t mode, void *stream);

/* ---- launch profiling ------------------------------------------------------ */

/* A measurement aid for the caller's own timing (per-kernel GPU durations).
 * moe_profile_begin: from now on every kernel the library launches carries
 *   two HIP events attached to its dispatch on its launch stream, which record
 *   the start and end of the kernel's execution, for up to max_launches
 *   launches (later launches are not recorded). Clears earlier records.
 *   Creates the events on first use (host-side objects, no device memory).
 * moe_profile_end: stops recording, waits for the recorded events and sums the
 *   elapsed time per kernel name.
 * moe_profile_count / moe_profile_get: the summary, one entry per kernel name:
 *   name (static string owned by the library), launches, total milliseconds.
 * The profiling state is process-global and not thread-safe; it is off unless
 * moe_profile_begin is called. */
int moe_profile_begin(int32_t max_launches);
int moe_profile_end(void);
int32_t moe_profile_count(void);
int moe_profile_get(int32_t i, const char **name, int32_t *launches, double *total_ms);

/* A static, human-readable description of a status code (host string). */
const char *moe_status_string(int32_t status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
