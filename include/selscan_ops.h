/*
 * libselscan: the operators around the selective scan (same library and conventions as
 * selscan.h, whose ss_dtype and ss_status are used here).
 *
 *   ss_glr_fwd, ss_glr_bwd, ss_glr_step   a gated linear recurrence: forward over whole
 *                                         sequences, its gradients, one decode token
 *   ss_quant_q8                           rounding to 8-bit floating point with block scales
 *   ss_norm_q8                            the same behind a residual's addition and RMS norm
 *   ss_gemm_q8                            the product of two such matrices
 *   ss_block_q8_fwd, ss_block_q8_step     the block around the scan with such projections
 *
 * Ownership, ordering, errors: as in selscan.h. Every pointer inside a struct is a DEVICE
 * pointer owned by the caller, arguments are validated on the host before anything is
 * enqueued, all work is asynchronous on `stream` of the current device, the library
 * allocates no device memory and never synchronises. Workspace contents on entry do not
 * matter; calls that share a workspace must be ordered on one stream. Results are
 * deterministic for a given shape (no floating-point atomics).
 */
#ifndef SELSCAN_OPS_H
#define SELSCAN_OPS_H

#include "selscan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Gated linear recurrence, one state per channel. Per batch row b, channel d and token t,
 * with r (recurrence gate) and i (input gate) given before their sigmoids:
 *
 *   s_t = sigmoid(r_t)
 *   a_t = exp(A[d] * s_t)                     0 where reset[b,t] != 0
 *   w_t = sqrt(1 - a_t^2)                     1 there
 *   h_t = a_t * h_{t-1} + w_t * sigmoid(i_t) * x_t
 *   y_t = h_t
 *
 * A[d] <= 0 (not checked; a positive value gives NaN through the square root; minus infinity
 * is a channel without memory, a = 0 but where the sigmoid is 0 itself). A reset
 * token starts a new document: the state before it is not read, so that not even a NaN
 * passes it. Elsewhere non-finite values propagate to the later tokens of their channel.
 *
 * Layout: x, r and i are [B, L, D] views whose channels are contiguous and whose batch
 * rows and tokens lie at any strides (columns of one projection's output, rows of a padded
 * batch); every other tensor is contiguous row-major. x, r, i, y and the gradients of x, r
 * and i have the I/O dtype (fp32 or bf16); A, states, checkpoints and the gradient of A
 * are fp32, and so is all arithmetic. */

#define SS_GLR_CKPT 64    /* tokens between two checkpoints */

typedef struct {
    int64_t batch;      /* B (streams for ss_glr_step), >= 1                            */
    int64_t seqlen;     /* 1 <= L < 2^31; ignored by ss_glr_step                         */
    int64_t d;          /* 1 <= D <= 2^26 channels                                       */
    int32_t io_dtype;   /* ss_dtype of x, r, i, y and their gradients                    */
    int32_t reserved;   /* 0                                                             */
} ss_glr_dims;

typedef struct {          /* [B, L, D] view: element (b, t, d) at p + b batch_stride + t token_stride + d */
    const void* p;        /* aligned to its element                                          */
    int64_t batch_stride; /* in elements, >= 0; ignored where B = 1                          */
    int64_t token_stride; /* in elements, >= 0; ignored where L = 1 and by ss_glr_step       */
} ss_view;

typedef struct {
    ss_view        x, r, i;  /* inputs                                                       */
    const float*   A;        /* [D]                                                          */
    const uint8_t* reset;    /* [B,L] ([B] for ss_glr_step) or NULL (no resets)              */
    void*          y;        /* [B,L,D] io OUT; must not overlap any input                   */
    float*         state;    /* [B,D] IN/OUT, or NULL: zero initial state, final not returned.
                                Required by ss_glr_step; not used by ss_glr_bwd              */
    float*         ckpt;     /* [B, ceil(L / SS_GLR_CKPT), D]: the state before tokens 0, 64, 128, ...
                                OUT of ss_glr_fwd (NULL: not written), IN of ss_glr_bwd      */
} ss_glr_args;

/* Bytes of device workspace of ss_glr_fwd (backward = 0) or ss_glr_bwd; 0 is possible for
 * the forward, and returned for invalid dims. */
size_t ss_glr_workspace_bytes(const ss_glr_dims* dims, int backward);

ss_status ss_glr_fwd(const ss_glr_dims* dims, const ss_glr_args* args, void* workspace, size_t workspace_bytes,
                     void* stream);

/* One token for every stream: x, r, i [B,D] views, y [B,D]; state updated in place. */
ss_status ss_glr_step(const ss_glr_dims* dims, const ss_glr_args* args, void* stream);

typedef struct {
    const void*  dy;           /* [B,L,D] io: gradient of y (required)                           */
    const float* dstate_final; /* [B,D] or NULL (zero): gradient of the returned state            */
    void*  dx;                 /* [B,L,D] io OUT (required)                                       */
    void*  dr;                 /* [B,L,D] io OUT (required)                                       */
    void*  di;                 /* [B,L,D] io OUT (required)                                       */
    float* dA;                 /* [D] OUT (required), summed over batch and time                  */
    float* dstate_init;        /* [B,D] OUT or NULL: gradient of the initial state                */
} ss_glr_grads;

/* Gradients of sum(dy * y) + sum(dstate_final * state_out) for the forward's inputs in
 * `args`, whose ckpt are the checkpoints that forward wrote (y and state are ignored, and
 * the initial state is read from the first checkpoint). With g_t the gradient of h_t,
 *   g_t = dy_t + a_{t+1} g_{t+1},        v_t = sigmoid(i_t) x_t,
 *   d(A s_t) = g_t (a_t h_{t-1} - (a_t^2 / w_t) v_t)   (0 at a reset; without the second
 *                                        term where w_t^2 is 0 or below the smallest normal fp32).
 * Outputs are overwritten; none may overlap an input, another output or the workspace. */
ss_status ss_glr_bwd(const ss_glr_dims* dims, const ss_glr_args* args, const ss_glr_grads* grads, void* workspace,
                     size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * 8-bit floating point with block scales. A matrix v [M, K] is held as q [M, K], one e4m3
 * byte a value (4 exponent bits, 3 stored mantissa bits, largest finite value 448, no
 * infinity), and fp32 scales; it stands for scale * q. A scale covers 128 consecutive
 * columns of one row (scale [M, ceil(K/128)], activations) or of 128 consecutive rows
 * ("square": scale [ceil(M/128), ceil(K/128)], weights); blocks at the ends are smaller.
 *   scale = max(max |v| / 448, 2^-126),   q = e4m3(v / scale), to nearest, ties to even
 * (of the quotient 448 v / max |v| itself: neither it nor the scale is rounded to fp32 first.
 * With fp32 v, and behind the norm, quotients below 2^-6 that lie within two fp32 steps of the
 * middle between two e4m3 values may go to either).
 * A NaN becomes a NaN and leaves its block's scale alone; an infinity makes its block's scale
 * infinite (its finite values stand for NaN then). All matrices are contiguous row-major. */
typedef struct {
    int64_t rows;       /* M, >= 1                                                      */
    int64_t cols;       /* K, 1 <= K < 2^31                                              */
    int32_t io_dtype;   /* ss_dtype of x (and residual, sum)                             */
    int32_t square;     /* ss_quant_q8: 0 = blocks of 1 x 128, 1 = 128 x 128             */
    float   eps;        /* ss_norm_q8: > 0                                               */
    int32_t reserved;   /* 0                                                             */
} ss_q8_dims;

ss_status ss_quant_q8(const ss_q8_dims* dims, const void* x, void* q, float* scale, void* stream);

/* The norm in front of a layer: with s = x + residual (in fp32),
 *   n = s / sqrt(mean over the row of s^2 + eps) * w,
 * rounded in blocks of 1 x 128. The norm takes s before it is rounded to the I/O dtype. */
typedef struct {
    const void*  x;         /* [M,K] io                                                     */
    const void*  residual;  /* [M,K] io or NULL: s = x                                      */
    const float* w;         /* [K]                                                          */
    void*        q;         /* [M,K] bytes OUT                                              */
    float*       scale;     /* [M, ceil(K/128)] OUT                                         */
    void*        sum;       /* [M,K] io OUT: s; required with a residual, else NULL.
                               May be x or residual itself (in place)                       */
} ss_norm_q8_args;

ss_status ss_norm_q8(const ss_q8_dims* dims, const ss_norm_q8_args* args, void* stream);

/* y[m,n] = sum_k (xs[m, k/128] xq[m,k]) (ws[n/128, k/128] wq[n,k])  (+ residual[m,n]).
 * Products and sums of a block on the matrix cores in fp32, blocks added in fp32 in order
 * of k (in a fixed order of several such sums where M is small). */
typedef struct {
    int64_t m, n;       /* rows of X and of W, 1 <= m, n < 2^31                          */
    int64_t k;          /* a multiple of 16, <= 2^23                                     */
    int32_t y_dtype;    /* ss_dtype of y and residual                                    */
    int32_t reserved;   /* 0                                                             */
} ss_gemm_q8_dims;

typedef struct {
    const void*  xq;        /* [M,K] e4m3, 16-byte aligned                                  */
    const float* xs;        /* [M, ceil(K/128)]                                             */
    const void*  wq;        /* [N,K] e4m3, 16-byte aligned                                  */
    const float* ws;        /* [ceil(N/128), ceil(K/128)]                                   */
    const void*  residual;  /* [M,N] of y_dtype, 16-byte aligned, or NULL; may be y itself  */
    void*        y;         /* [M,N] OUT, 16-byte aligned                                   */
} ss_gemm_q8_args;

ss_status ss_gemm_q8(const ss_gemm_q8_dims* dims, const ss_gemm_q8_args* args, void* stream);

/* ---------------------------------------------------------------------------
 * The block around the scan (ss_block_fwd, ss_block_step) with its input and output
 * projections as 8-bit products: RMSNorm(x) and the scan's output y are rounded in blocks of
 * 1 x 128, W_in [2 Di, d_model] and W_out [d_model, Di] are e4m3 with scales of 128 x 128 (as
 * ss_quant_q8 with square = 1 makes them). Everything else, and the types of x, out, W_x, W_dt
 * and the states, is as there. d_model and d_inner are multiples of 16. */
typedef struct {
    ss_block_weights w;     /* W_in and W_out point to e4m3 bytes, 16-byte aligned          */
    const float* S_in;      /* [ceil(2 Di/128), ceil(d_model/128)]                          */
    const float* S_out;     /* [ceil(d_model/128), ceil(Di/128)]                            */
} ss_block_q8_weights;

/* Bytes of workspace; 0 for invalid sizes. */
size_t ss_block_q8_workspace_bytes(const ss_block_dims* dims, int step);

/* x, out [B,L,d_model]; states as for ss_block_fwd (NULL: zero, not returned). out may be x
 * (in place); nothing else that is written may overlap anything. */
ss_status ss_block_q8_fwd(const ss_block_dims* dims, const ss_block_q8_weights* weights, const void* x, void* out,
                          float* ssm_state, float* conv_state, void* workspace, size_t workspace_bytes, void* stream);

/* One token of each stream: x, out [B,d_model]; both states required and updated. */
ss_status ss_block_q8_step(const ss_block_dims* dims, const ss_block_q8_weights* weights, const void* x, void* out,
                           float* ssm_state, float* conv_state, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_OPS_H */
