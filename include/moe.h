/*
 * moe.h - C ABI of the MI355X (gfx950) routed-expert MoE FFN layer library
 * (libmoe.so).
 *
 * The layer, for every token t of x[T, H]:
 *   1. router: logits l = x_t . router_w^T (+ router_bias), accumulated in
 *      fp32 and never rounded to bf16; the top_k experts by logit (descending,
 *      ties to the lower expert index); weights w = softmax of the k selected
 *      logits (equal to the full softmax renormalised over the selection).
 *      Pages: "MoE prefill quantum" (cause section: each token uses k of E
 *      experts); "DeepSeek V4.1F Q4 with native DSpark MTP" (decode
 *      paragraph: the router as a single fused dispatch).
 *   2. permutation: the (t, j) pairs grouped by expert, stably (t, then j
 *      ascending within an expert).
 *   3. per expert e: h = silu(x W_gate[e]^T) * (x W_up[e]^T)  (SwiGLU with the
 *      SiLU on the gate branch; "Jetson Orin Nano MoE ... expert cache",
 *      re-check section and gate-first section).
 *   4. o = h W_down[e]^T, scaled by w[t, j]; y_t = sum over j = 0..k-1 of the
 *      scaled rows in that fixed order (same page, nondeterminism section:
 *      each expert owns its output rows, so the order of the sum is fixed),
 *      plus, if present, the always-on shared expert's output with weight 1
 *      ("DeepSeek V4.1F" decode paragraph).
 *
 * Layouts (row-major, K-contiguous):
 *   x [T, H], y [T, H]              act_dtype (MOE_F32 or MOE_BF16)
 *   router_w [E, H]                 act_dtype
 *   router_bias [E]                 float, or NULL
 *   w_gate, w_up [E, I, H]          w_dtype
 *   w_down [E, H, I]                w_dtype
 *     MXFP4 (OCP MX v1.0): the matrices as moe_pack_mxfp4 lays them out
 *     (below), from the OCP row-major form: codes [E, N, K/2], two E2M1
 *     codes per byte, even element in the low nibble, and E8M0 scales
 *     [E, N, K/32], one per 32 consecutive K elements ([N, K] = [I, H] for
 *     gate and up, [H, I] for down).
 *   sh_gate, sh_up [I_shared, H], sh_down [H, I_shared]   act_dtype
 *     BF16 expert matrices (routed and shared) are passed as moe_pack_bf16
 *     lays them out (below); F32 and FP8 ones row-major as listed.  The caller
 *     states which in moe_weights_t.layout: MOE_LAYOUT_PACKED is required for
 *     BF16 and MXFP4 expert matrices, MOE_LAYOUT_ROWMAJOR for F32 and FP8; any
 *     other combination is refused with MOE_EINVAL (a zero-initialised
 *     struct says ROWMAJOR, so row-major bf16 weights never reach a kernel).
 *     FP8 (E4M3 codes, one float scale per 128 x 128 block): row-major codes
 *     and scales [E, N/128, K/128] in s_gate, s_up, s_down, as
 *     moe_quant_fp8 makes them; x is quantised in the call (1 x 128 blocks),
 *     and so is h, from its fp32 values.
 *   topk_idx [T, top_k] int32, topk_w [T, top_k] float
 *
 * Packed MXFP4 (what the kernels read: each wave's weights are whole
 * contiguous kilobytes).  Rows go in blocks of 16 (n = 16*nb + r) and K in
 * steps of 128 (q = K/128 steps); the lane index l = r + 16*b, b = 0..3:
 *   codes  [E][N/16][q][64 lanes][16 B]: lane l of step s holds the 32 codes
 *          of row n at K = 128*s + 32*b .. +31 (OCP byte order);
 *   scales [E][N/16][64 lanes][q]: byte s of lane l is the scale of row n
 *          at K = 128*s + 32*b .. +31.
 * The packed matrices have the same sizes as the OCP ones.
 *
 * Packed BF16 (what the kernels read: a wave's weight fragment of one MFMA
 * step is a contiguous kilobyte).  Rows go in groups of 32 (g = n / 32) and
 * K in steps of 32 (s = k / 32); each (g, s) is two 1 KB blocks c = 0, 1;
 * lane l = r + 16*b (r = 0..15, b = 0..3) of block c holds the 8 elements
 * of row n = 32*g + 8*(r/4) + 4*c + r%4 at K = 32*s + 8*b .. +7:
 *   [E][N/32][K/32][2][64 lanes][8 bf16].
 *
 * Supported combinations: act F32 with w F32; act BF16 with w BF16, MXFP4 or
 * FP8.  FP8 needs H and I multiples of 128, at most 32768, and no shared
 * expert (MOE_EINVAL / MOE_EUNSUPPORTED otherwise).  MXFP4 needs H and I multiples of 128, at most 4096, and no shared expert
 * (MOE_EINVAL / MOE_EUNSUPPORTED otherwise).  One pass (chunk) of Tc tokens
 * must keep Tc * H, Tc * E * 8 and rows * max(H, I, I_shared) below 2^31,
 * rows = Tc * top_k (+ Tc with a shared expert); larger passes are refused
 * with MOE_EINVAL (split them with chunk_T).
 * Every pointer except router_bias, topk_w and the unused ones is a device
 * pointer, 16-byte aligned.  The caller owns all memory; the library
 * allocates nothing per call and keeps no state between calls other than
 * cached device properties.  Calls are asynchronous on `stream` (a
 * hipStream_t, NULL = the default stream): outputs are valid once the stream
 * has synchronised.  Nothing is read back to the host inside a call.
 *
 * Error handling: every entry point returns MOE_OK (0) or a negative code;
 * no exception crosses the boundary.  On MOE_EINVAL / MOE_EWORKSPACE nothing
 * has been launched.  On MOE_EHIP a launch failed; moe_last_error() gives the
 * HIP error text of the calling thread's last failure.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_MXFP4 = 2, MOE_FP8 = 3 } moe_dtype_t;

/* Layout of the expert matrices in moe_weights_t (see Layouts above). */
enum { MOE_LAYOUT_ROWMAJOR = 0, MOE_LAYOUT_PACKED = 1 };

enum {
    MOE_OK = 0,
    MOE_EINVAL = -1,       /* null/misaligned pointer, bad size or dtype  */
    MOE_EWORKSPACE = -2,   /* ws_bytes < moe_workspace_bytes(shape)       */
    MOE_EUNSUPPORTED = -3, /* device is not gfx950, or dtype combination  */
    MOE_EHIP = -4          /* HIP launch/runtime error                    */
};

/* Sizes of one call.
 *  - top_k is a run-time value, not a property of the weights: a caller may
 *    run a layer with fewer experts per token than it was trained with ("Jetson
 *    Orin Nano MoE: GPU clock floor and expert cache", section on decode time
 *    as a fixed part plus a read part, where the model's experts-per-token
 *    count is overridden from 8 to 4).
 *  - chunk_T is the prefill quantum: the number of tokens the layer is handed
 *    at a time ("MoE prefill quantum", the one-line summary and the inverse
 *    equation quantum = target tokens per expert x E / top_k).  Passes of
 *    chunk_T tokens run one after the other on one workspace; tokens are
 *    independent, so y does not depend on it. */
typedef struct {
    int32_t T;         /* tokens                                             */
    int32_t H;         /* hidden size (multiple of 64)                       */
    int32_t E;         /* routed experts, 1..1023                            */
    int32_t top_k;     /* experts per token, 1..min(E, 16)                   */
    int32_t I;         /* expert intermediate size (multiple of 64)          */
    int32_t I_shared;  /* shared expert intermediate size, 0 = none          */
    int32_t chunk_T;   /* tokens per internal pass, 0 = all T at once        */
    int32_t act_dtype; /* moe_dtype_t of x, y, router_w and shared weights   */
    int32_t w_dtype;   /* moe_dtype_t of the routed expert weights           */
} moe_shape_t;

typedef struct {
    const void *router_w;
    const float *router_bias;                /* nullable                     */
    const void *w_gate, *w_up, *w_down;      /* codes when w_dtype == MXFP4  */
    const uint8_t *s_gate, *s_up, *s_down;   /* MXFP4: E8M0; FP8: the floats */
    const void *sh_gate, *sh_up, *sh_down;   /* I_shared > 0 only            */
    int32_t layout;  /* MOE_LAYOUT_* of the expert and shared matrices       */
} moe_weights_t;

/* Bytes of device workspace moe_forward / moe_route need for `shape`
 * (sized for one chunk of min(T, chunk_T) tokens); 0 if the shape is
 * invalid. */
size_t moe_workspace_bytes(const moe_shape_t *shape);

/* The whole layer: y [T, H] and the routing (topk_idx required, topk_w
 * nullable).  The routing is returned because callers keep it: per-layer
 * logs of the experts the router chose are what an expert cache's policy is
 * chosen from ("Jetson Orin Nano MoE: GPU clock floor and expert cache",
 * section on choosing what to cache from the router's records).  `ws` is device memory of at least moe_workspace_bytes(shape)
 * bytes, 256-byte aligned, owned by the caller; its contents on entry do not
 * matter.  The result does not depend on chunk_T beyond rounding order: each
 * chunk is processed independently in token order. */
int moe_forward(const moe_shape_t *shape, const moe_weights_t *w,
                const void *x, void *y, int32_t *topk_idx, float *topk_w,
                void *ws, size_t ws_bytes, void *stream);

/* Bytes of the static device scratch moe_forward_noalloc uses (per GPU). */
#define MOE_NOALLOC_SCRATCH_BYTES (64ull << 20)

/* moe_forward for callers that cannot allocate device memory: code under
 * HIP graph capture, serving loops and harnesses that must not call
 * hipMalloc.  Same arguments and results as moe_forward, without the
 * workspace: the scratch comes from a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES (64 MiB) that each GPU the library runs on holds
 * from the library's first use there until the process ends; its address on
 * a device is looked up on the first call on that device.  Allocates nothing
 * (no hipMalloc/hipFree, no allocating library routine).  A shape whose pass
 * (min(T, chunk_T) tokens) needs more scratch than that is refused with
 * MOE_EWORKSPACE before anything is launched (moe_workspace_bytes gives the
 * need; a smaller chunk_T lowers it: 52 MiB for 1024 tokens at H=2048, E=256,
 * top-8, I=768).  Every call on a GPU shares that GPU's scratch and leaves
 * its contents behind (no call needs it cleared): calls that overlap on one
 * GPU, from several streams or threads, race. */
int moe_forward_noalloc(const moe_shape_t *shape, const moe_weights_t *w,
                        const void *x, void *y, int32_t *topk_idx, float *topk_w,
                        void *stream);

/* Router and permutation only (analysis / test export).  For the tokens of
 * one pass (chunk_T must be 0 or >= T): topk_idx [T, k], topk_w [T, k],
 * counts [E] (pairs per expert), offsets [E+1] (exclusive prefix of counts)
 * and row_src [T*k] (the pair t*k+j at each grouped position).  All device
 * pointers; topk_w, counts, offsets and row_src are nullable. */
int moe_route(const moe_shape_t *shape, const moe_weights_t *w,
              const void *x, int32_t *topk_idx, float *topk_w,
              int32_t *counts, int32_t *offsets, int32_t *row_src,
              void *ws, size_t ws_bytes, void *stream);

/* ---- Routing and experts apart --------------------------------------------
 * The layer in three calls, for routing other than moe_forward's:
 *   moe_logits  -> moe_select -> moe_experts
 * (any of them may be replaced by the caller's own: moe_experts takes whatever
 * routing it is given).  The general rules above hold for them: device
 * pointers, nothing allocated, nothing read back, asynchronous on `stream`.
 */

/* The router's logits alone: logits[T, E] (fp32) = x . router_w^T
 * (+ router_bias).  Only the shape's T, H, E, top_k and act_dtype and the
 * weights' router_w and router_bias are used (the shape must be valid as a
 * whole).  Any T: the limits of a pass do not hold here.  x and logits 16-byte
 * aligned. */
int moe_logits(const moe_shape_t *shape, const moe_weights_t *w, const void *x, float *logits,
               void *stream);

enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 };

/* Selection of experts from logits [T, E]:
 *   score  s_e = softmax(l)_e over all E, or 1 / (1 + exp(-l_e))
 *   key    s_e + bias_e (the bias balances the experts' loads: it counts in
 *          the selection, not in the weights)
 *   groups n_group > 1: groups of E / n_group consecutive experts, valued by
 *          their largest key or the sum of their two largest; only experts of
 *          the topk_group best groups (equal ones: the lower group) remain
 *   top-k  the k remaining experts by key, descending, equal keys to the lower
 *          index: topk_idx, in that order
 *   weights topk_w = s of the selected, divided by their sum if renorm, times
 *          scale; all 0 where the sum is 0
 * The order is that of the keys in 64 bits, whatever type the logits have.
 * An expert is masked by a logit of -inf or NaN or a bias of -inf or NaN: it
 * ranks behind all others (masked ones by index) and has weight 0, and a masked
 * logit has no share of the softmax.  A group of masked experts only ranks last.  +inf
 * counts as the largest finite float. */
typedef struct {
    int32_t T;            /* tokens                                             */
    int32_t E;            /* experts, 1..1024                                   */
    int32_t top_k;        /* 1..min(E, 16), at most the open groups' experts    */
    int32_t n_group;      /* 1 = no groups; at most 64, divides E               */
    int32_t topk_group;   /* 1..n_group                                         */
    int32_t score;        /* MOE_SCORE_*                                        */
    int32_t group_score;  /* MOE_GROUP_*                                        */
    int32_t renorm;       /* nonzero: weights divided by their sum              */
    int32_t logit_dtype;  /* MOE_F32 or MOE_BF16                                */
    float scale;          /* factor of the weights                              */
    int64_t ld;           /* row stride of the logits in elements, 0 = E        */
} moe_select_t;

/* logits [T, E] (row stride ld), bias [E] float or NULL, topk_idx [T, top_k],
 * topk_w [T, top_k] or NULL; pointers aligned to their elements. */
int moe_select(const moe_select_t *select, const void *logits, const float *bias,
               int32_t *topk_idx, float *topk_w, void *stream);

/* The routed experts with given routing: y_t = sum over j of topk_w[t, j] *
 * FFN of expert topk_idx[t, j] on x_t, in j order.  Every weight type of
 * moe_forward; the weights' router_w and router_bias are not used (NULL is
 * fine) and I_shared must be 0 (MOE_EUNSUPPORTED otherwise).  A slot whose
 * index is outside 0..E-1 (say -1) is empty: it adds nothing, whatever its
 * weight, and a token with empty slots only gets zeros.  An expert may occur more than once
 * in a token.  Workspace and chunk_T as for moe_forward; x and y 16-byte
 * aligned, topk_idx and topk_w 4-byte. */
int moe_experts(const moe_shape_t *shape, const moe_weights_t *w, const void *x,
                const int32_t *topk_idx, const float *topk_w, void *y, void *ws,
                size_t ws_bytes, void *stream);

/* ---- FP8 (E4M3) with block scales ------------------------------------------ */

/* Rows [R, K] to E4M3 codes and float scales, one per block of block_rows x
 * 128 (1: activations, 128: weights):
 *   top = max(max |x| over the block, 2^-100), scale = top / 448,
 *   code = the E4M3 value nearest to 448 x / top, ties to the even one
 * so x is about code * scale.  The last blocks of a row or column are cut off
 * at K and R.  NaN elements are passed over by the maximum and get the NaN
 * code; every code of a block with an infinity is NaN. */
typedef struct {
    int32_t R, K;        /* rows and columns                                    */
    int32_t block_rows;  /* 1 or 128                                            */
    int32_t src_dtype;   /* MOE_F32 or MOE_BF16                                 */
    int64_t ld;          /* row stride of x in elements, 0 = K                  */
} moe_quant_t;

/* codes [R, Kp] bytes, Kp = K rounded up to a multiple of 128, the columns
 * behind K zero; scales [R, Kp / 128] (block_rows 1) or [R / 128 rounded up,
 * Kp / 128] (128).  x and scales element aligned, codes 16-byte aligned; the
 * outputs overlap neither x nor each other.  Fewer than 2^31 blocks, 2^24 of
 * 128 rows.  A stack of matrices [E, N, K]
 * with N a multiple of 128 is one call with R = E * N. */
int moe_quant_fp8(const moe_quant_t *quant, const void *x, void *codes, float *scales,
                  void *stream);

/* Product of such codes, y[m, n] = sum over blocks q of 128 K of sa[m, q] *
 * sb[n / 128, q] * sum over k in q of a[m, k] * b[n, k]: the sums in fp32, y
 * rounded once.  With G > 1 the rows of a are grouped: rows offsets[g] ..
 * offsets[g + 1] - 1 meet matrix b[g] (groups may be empty); rows outside
 * offsets[0] .. offsets[G] - 1 of y stay as they were.  offsets is a device array, not
 * decreasing; parts of it outside 0..M are cut off. */
typedef struct {
    int32_t M, N, K;     /* rows of a, rows of each b, depth (at most 32768)    */
    int32_t G;           /* matrices b, 1..65535                                */
    int32_t out_dtype;   /* MOE_F32 or MOE_BF16                                 */
    int64_t lda, ldb;    /* row strides in bytes, multiples of 16, 0 = Kp       */
    int64_t ldy;         /* row stride of y in elements, 0 = N                  */
} moe_matmul_t;

/* a [M, Kp] codes (Kp = K rounded up to a multiple of 128; the columns behind
 * K must hold zero codes, as moe_quant_fp8 writes them), sa [M, Kp / 128],
 * b [G, N, Kp] codes, sb [G, N / 128 rounded up, Kp / 128], offsets [G + 1]
 * (G = 1: NULL takes all rows), y [M, N].  a and b 16-byte aligned, the others
 * element aligned; y overlaps none of the operands. */
int moe_matmul_fp8(const moe_matmul_t *matmul, const void *a, const float *sa, const void *b,
                   const float *sb, const int32_t *offsets, void *y, void *stream);

/* ---- Rows by expert, and gradients ------------------------------------------
 * For callers whose step through the experts is their own (training, adapters,
 * other activations), and for the backward pass of the routed layer.  Forward:
 *   moe_logits -> moe_select -> moe_dispatch -> moe_matmul_bf16 (gate, up) ->
 *   moe_swiglu -> moe_matmul_bf16 (down) -> moe_combine
 * and backward:
 *   moe_combine_grad -> moe_matmul_bf16_dx / _dw (down) -> moe_swiglu_grad ->
 *   moe_matmul_bf16_dx / _dw (gate, up) -> moe_combine without weights (the
 *   gradient of moe_dispatch) and moe_select_grad
 * The general rules above hold.  Element types: rows of moe_dispatch, moe_combine
 * and moe_swiglu are MOE_F32 or MOE_BF16, operands of the products bf16.
 * Pointers are aligned to their elements, codes to 16 bytes, unless said
 * otherwise; strides are in elements, at most 2^31; an output overlaps neither an
 * input nor another output (spans from the first to the last element count). */

/* The pairs (t, j) sorted by expert, stably (t, then j within an expert), and
 * the tokens' rows in that order:
 *   offsets [E + 1]     first place of each expert's pairs; offsets[E] pairs in all
 *   row_src [T * top_k] pair t * top_k + j at each place (nullable; the places from
 *                       offsets[E] on stay as they were)
 *   row_of [T, top_k]   place of each pair, -1 for an empty slot (an index outside
 *                       0..E-1)
 *   rows [T * top_k, H] rows[row_of[t, j]] = x[t]; the rows from offsets[E] on stay
 *                       as they were
 * x holds MOE_F32 or MOE_BF16 values, which are copied bit by bit, or MOE_FP8: codes
 * and scales of moe_quant_fp8 in 1 x 128 blocks (an 8-bit checkpoint of x), which
 * are multiplied in fp32 and rounded once to row_dtype. */
typedef struct {
    int32_t T, H;        /* tokens and columns (at most 2^30, as every number of rows, tokens and columns here) */
    int32_t E, top_k;    /* experts, 1..1024; slots of a token, 1..16           */
    int32_t x_dtype;     /* MOE_F32, MOE_BF16 or MOE_FP8                        */
    int32_t row_dtype;   /* x_dtype; MOE_F32 or MOE_BF16 where x is MOE_FP8     */
    int64_t ldx;         /* row stride of x, 0 = H (codes: H rounded up to 128; a multiple of 16) */
    int64_t ldr;         /* row stride of rows, 0 = H                           */
} moe_dispatch_t;

/* Bytes of workspace of moe_dispatch, 0 if the sizes are invalid. */
size_t moe_dispatch_workspace_bytes(const moe_dispatch_t *dispatch);

/* At most 2^30 pairs.  x and rows NULL: the order alone.  sx: scales of MOE_FP8
 * [T, H / 128 rounded up], else not used.  ws 256-byte aligned, one for each call
 * that may run at the same time. */
int moe_dispatch(const moe_dispatch_t *dispatch, const int32_t *topk_idx, const void *x, const float *sx,
                 void *rows, int32_t *offsets, int32_t *row_src, int32_t *row_of, void *ws, size_t ws_bytes,
                 void *stream);

/* The rows alone, by a row_of [T, top_k] that moe_dispatch has made: places outside
 * 0 .. T * top_k - 1 take no row.  (E has to be in its range, and is not used.) */
int moe_gather(const moe_dispatch_t *dispatch, const int32_t *row_of, const void *x, const float *sx, void *rows,
               void *stream);

/* The way back: y[t] = sum over j of topk_w[t, j] * rows[row_of[t, j]] in j order
 * (fp32, rounded once); a slot whose row_of is outside 0 .. R - 1 adds nothing,
 * whatever its weight, and a token of empty slots gets zeros.  topk_w NULL: weights of 1,
 * which is the gradient of moe_gather. */
typedef struct {
    int32_t T, H, top_k; /* tokens, columns, slots of a token (1..16)           */
    int32_t R;           /* rows there are                                      */
    int32_t dtype;       /* MOE_F32 or MOE_BF16, of rows and y                  */
    int64_t ldr, ldy;    /* row strides of rows and y, 0 = H                    */
} moe_combine_t;

int moe_combine(const moe_combine_t *combine, const void *rows, const int32_t *row_of, const float *topk_w,
                void *y, void *stream);

/* Its gradient: drows[row_of[t, j]] = topk_w[t, j] * dy[t] and dtopk_w[t, j] = sum
 * over the columns of dy[t] * rows[row_of[t, j]] (fp32), 0 for an empty slot.  Rows
 * that no slot names stay as they were; a row may be named once.  drows or dtopk_w may
 * be NULL (rows then too, without dtopk_w).  drows lies as rows do, dy as y. */
int moe_combine_grad(const moe_combine_t *combine, const void *dy, const void *rows, const int32_t *row_of,
                     const float *topk_w, void *drows, float *dtopk_w, void *stream);

/* h = silu(gate) * up of rows [R, I], in fp32 and rounded once, and with codes an
 * 8-bit checkpoint of gate and up: per row the codes of gate, then those of up, each
 * Ip = I rounded up to a multiple of 128 wide (codes [R, 2 * Ip]), and their scales
 * [R, 2 * Ip / 128], by the definition of moe_quant_fp8 in 1 x 128 blocks.  `used`:
 * a device count of the rows in use (offsets + E of moe_dispatch, say), NULL: all; the
 * rows behind stay as they were, in every output.  gate and up may be columns of one
 * matrix (ld 2 * I or more). */
typedef struct {
    int32_t R, I;        /* rows and columns                                    */
    int32_t dtype;       /* MOE_F32 or MOE_BF16                                 */
    int64_t ld;          /* row stride of gate, up, dgate and dup, 0 = I        */
    int64_t ldh;         /* row stride of h and dh, 0 = I                       */
} moe_swiglu_t;

int moe_swiglu(const moe_swiglu_t *swiglu, const void *gate, const void *up, const int32_t *used, void *h,
               void *codes, float *scales, void *stream);

/* Its gradient, with s = 1 / (1 + exp(-gate)):
 *   dgate = dh * up * s * (1 + gate * (1 - s)),  dup = dh * gate * s
 * and, if h is not NULL, h again.  gate and up are read from the checkpoint where
 * codes and scales are given (gate and up are then not used), each output rounded
 * once. */
int moe_swiglu_grad(const moe_swiglu_t *swiglu, const void *gate, const void *up, const void *codes,
                    const float *scales, const void *dh, const int32_t *used, void *dgate, void *dup, void *h,
                    void *stream);

/* Gradient of moe_select to the logits: dlogits [T, E] (dense, dlogit_dtype MOE_F32 or
 * MOE_BF16) of a loss whose gradient to the weights is dtopk_w [T, top_k] and to every
 * token's score s_e is dscore[e] (NULL: none; a balance loss c * sum_e f_e * mean_t
 * s_te has dscore[e] = c * f_e / T; one over scores that each token divides by their
 * sum has gradients that differ from token to token and is not covered).  The selection
 * itself, the bias and the groups are constants: T, E, top_k, score, renorm,
 * logit_dtype, scale and ld of `select` are used.  topk_idx as moe_select wrote it.
 * Masked experts (by logit or bias) have score 0 and pass no gradient from dtopk_w or
 * dscore, nor do experts whose score is 0 in 64 bits; what passes through a score, its
 * rest to 1 or a ratio of selected scores below 2^-126 loses digits, and below 2^-149 it
 * is 0 (fp32).  An index outside 0..E-1 counts as no slot: it is left out of the
 * renormalising sum as well (a slot dropped after the selection keeps its index here,
 * with dtopk_w 0). */
int moe_select_grad(const moe_select_t *select, const void *logits, const float *bias, const int32_t *topk_idx,
                    const float *dtopk_w, const float *dscore, void *dlogits, int dlogit_dtype, void *stream);

/* Grouped products of bf16 rows with bf16 matrices w [G, N, K] (row-major), sums in
 * fp32, rounded once to out_dtype:
 *   moe_matmul_bf16     y [M, N]     = x w[g]^T   for the rows of each group g
 *   moe_matmul_bf16_dx  dx [M, K]    = dy w[g]
 *   moe_matmul_bf16_dw  dw [G, N, K] = dy^T x     over the rows of each group
 * (+ add, as the output lies and of its type, or NULL; it may be the output itself:
 * a gradient summed over several calls).  Rows offsets[g] .. offsets[g + 1] - 1
 * belong to group g; groups may be empty (their dw is 0, or add).  Rows of y and dx
 * outside offsets[0] .. offsets[G] - 1 stay as they were, those of x and dy are not
 * used.  offsets is a device array, not decreasing; parts of it outside 0..M are cut
 * off (of offsets that decrease it is not defined which rows are taken, but nothing
 * outside 0..M is); with G = 1 NULL takes all rows.  Any sizes, strides and element alignment are
 * taken; sizes and strides that are multiples of 8 elements (rows: any number), strides below
 * 2^20 and pointers aligned to 16 bytes are fast. */
typedef struct {
    int32_t M, N, K;     /* rows; rows and columns of each w; at most 2^30 each */
    int32_t G;           /* matrices w, 1..65535                                */
    int32_t out_dtype;   /* MOE_F32 or MOE_BF16                                 */
    int64_t ldx, ldw, ldy; /* row strides of x and dx, w and dw, y and dy, 0: K, K, N */
} moe_matmul_bf16_t;

int moe_matmul_bf16(const moe_matmul_bf16_t *matmul, const void *x, const void *w, const int32_t *offsets,
                    const void *add, void *y, void *stream);
int moe_matmul_bf16_dx(const moe_matmul_bf16_t *matmul, const void *dy, const void *w, const int32_t *offsets,
                       const void *add, void *dx, void *stream);
int moe_matmul_bf16_dw(const moe_matmul_bf16_t *matmul, const void *dy, const void *x, const int32_t *offsets,
                       const void *add, void *dw, void *stream);

/* The tile that such a product takes, for analysis and tests (nothing is launched): way
 * 0, 1 or 2 for y, dx or dw, off16 not 0 where a pointer is not at a multiple of 16
 * bytes.  tile[0], tile[1]: rows and columns of the output; tile[2]: groups of waves that
 * share the depth of the sums; tile[3]: 1 if the operands are copied in pieces of 16
 * bytes, 0 for the tiles of any alignment. */
int moe_matmul_bf16_tile(const moe_matmul_bf16_t *matmul, int way, int off16, int32_t *tile);

/* Repack E MXFP4 matrices of N rows and K columns (N a multiple of 16, K of
 * 128) from the OCP row-major form (codes [E, N, K/2], scales [E, N, K/32])
 * into the layout moe_forward reads (above); E * N * K / 2 code bytes and
 * E * N * K / 32 scale bytes out.  Device pointers, 16-byte aligned, the
 * outputs not overlapping the inputs; asynchronous on `stream`.  A one-time
 * step when weights are loaded.  MOE_EINVAL on bad sizes or pointers. */
int moe_pack_mxfp4(int E, int N, int K, const void *codes, const uint8_t *scales,
                   void *codes_out, uint8_t *scales_out, void *stream);

/* Repack E bf16 matrices of N rows and K columns (multiples of 32) from the
 * row-major form [E, N, K] into the layout moe_forward reads (above); the
 * same number of bytes out.  Device pointers, 16-byte aligned, not
 * overlapping; asynchronous on `stream`.  A one-time step when weights are
 * loaded.  MOE_EINVAL on bad sizes or pointers. */
int moe_pack_bf16(int E, int N, int K, const void *w, void *w_out, void *stream);

/* Stage timing for measurement (not needed for computing).  While enabled,
 * moe_forward records a pair of HIP events on its stream around each of its
 * stages - 0 router, 1 permutation, 2 gate+up, 3 down, 4 combine - for up to
 * 4096 calls; moe_stage_timing_read waits for them, writes the summed
 * milliseconds per stage into ms[0..n_stages) and the number of recorded
 * calls into *n_calls, and clears the record.  Enabling or disabling also
 * clears it.  Process-wide; returns MOE_OK or MOE_EHIP. */
int moe_stage_timing_enable(int on);
int moe_stage_timing_read(float *ms, int n_stages, int *n_calls);

/* Measurement aids (not part of the layer): the ceilings its kernels are
 * compared with on this device.  Asynchronous on `stream`; time them with
 * events around the call.
 * moe_probe_read reads `bytes` (a positive multiple of 16) at the device
 * pointer buf with 16-byte loads from every CU and discards the data, so a
 * buffer much larger than the caches gives the achievable HBM read rate.
 * moe_probe_mfma runs `iters` rounds of 8 independent bf16 16x16x32 MFMA
 * chains in each of `waves` waves (a positive multiple of 4): 8 * 16384
 * floating-point operations per wave and round, the matrix cores' sustained
 * bf16 rate.  sink is a device int (or NULL) that may receive a value
 * derived from the results.  MOE_EINVAL for bad sizes or a NULL buffer,
 * MOE_EHIP if the launch fails. */
int moe_probe_read(const void *buf, size_t bytes, void *stream);
int moe_probe_mfma(int waves, int iters, int *sink, void *stream);

/* Scattered expert-block reads ("MoE prefill quantum", the section ruling
 * out the hardware, which times a random read of 300 blocks of 13.3 MB
 * beside a sequential read).  pool: a device buffer of pool_bytes holding
 * pool_bytes / chunk_bytes chunks of chunk_bytes (a positive multiple of 16;
 * one expert's weight block); order: a device int32 array of nchunks chunk
 * numbers (entries outside the pool read the nearest chunk); the chunks are
 * read whole in that order by `wgs` workgroups of 256 threads (1..65536;
 * fewer workgroups than CUs gives the read rate of that many CUs), 16-byte
 * non-temporal loads, data discarded: nchunks * chunk_bytes bytes.
 * moe_probe_mxfp4 streams nblocks MXFP4 blocks in the OCP row-major form
 * (codes: 16 bytes per block, 32 E2M1 codes, the even element in the low
 * nibble, 16-byte aligned; scales: one E8M0 byte per block), decodes every
 * value as code x 2^(scale - 127) with the scaled fp4 conversion and adds
 * them up: out[w] (a device float array of wgs entries) receives workgroup
 * w's fp32 sum, so the stream is checkable; 17/32 byte per value ("MoE
 * prefill quantum", the same section: unpacking and scaling MXFP4 streams
 * at the raw read rate).  Both asynchronous on `stream`; MOE_EINVAL for bad
 * sizes or NULL / misaligned pointers (checked before any launch), MOE_EHIP
 * if the launch fails. */
int moe_probe_gather(const void *pool, size_t pool_bytes, size_t chunk_bytes,
                     const int32_t *order, int nchunks, int wgs, void *stream);
int moe_probe_mxfp4(const void *codes, const uint8_t *scales, size_t nblocks, int wgs,
                    float *out, void *stream);

/* Static text for a return code. */
const char *moe_strerror(int code);

/* Detail of the calling thread's last failure (argument name or HIP error). */
const char *moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
