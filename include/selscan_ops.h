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
 *   ss_gdr_fwd, ss_gdr_bwd, ss_gdr_step   the gated delta rule: forward over whole sequences, its
 *                                         gradients, one decode token
 *   ss_gnorm_fwd, ss_gnorm_bwd            the norms behind and before a layer with its gate, its
 *                                         scale and the residual, and their gradients
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

/* ---------------------------------------------------------------------------
 * Gated delta rule, one state S [dk, dv] per batch row and head h; head h of v uses the keys and
 * queries of head h / (heads / k_heads). Per token t, with g the logarithm of the decay:
 *
 *   k^ = k / sqrt(sum k^2 + eps), q^ likewise       k and q themselves where eps = 0
 *   S' = exp(g_t) S_{t-1}                            0 where reset[b,t] != 0
 *   u  = beta_t (v_t - S'^T k^_t)
 *   S_t = S' + k^_t u^T
 *   y_t = scale S_t^T q^_t
 *
 * A log decay of -200 or less (minus infinity among them) is a decay of 0, as a reset is. A decay
 * of 0 leaves out what it multiplies, so that not even a NaN passes it. A value that is not finite
 * reaches what the formulas say and nothing else, tokens in front of it and documents
 * behind the next reset neither; what it may reach is then made token by token, some microseconds each.
 * g > 0, beta and the lengths of keys that are used as they are (eps = 0) are the caller's: with
 * 0 <= beta |k^|^2 <= 2 no state grows; nothing is checked.
 *
 * q, k and v are views whose last dimension is contiguous and whose rows, tokens and heads lie at any
 * strides (columns of one projection's output, [B, H, L, d] layouts); every other tensor is contiguous
 * row-major. q, k, v, y and the gradients of q, k, v and y have the I/O dtype (fp32 or bf16); gates,
 * states, checkpoints and their gradients are fp32. Sums and states are fp32; products are made on the
 * bf16 matrix instructions, fp32 operands as sums of three bf16 terms (24 bits). */

#define SS_GDR_CHUNK 64   /* tokens between two checkpoints */

typedef struct {
    int64_t batch;      /* B (streams for ss_gdr_step), >= 1                            */
    int64_t seqlen;     /* 0 <= L < 2^31; ignored by ss_gdr_step                         */
    int32_t k_heads;    /* heads of q and k, >= 1                                        */
    int32_t heads;      /* H heads of v, a multiple of k_heads                           */
    int32_t dk, dv;     /* 1 <= dk <= 256, 1 <= dv <= 512                                */
    int32_t io_dtype;   /* ss_dtype of q, k, v, y and their gradients                    */
    float   scale;      /* of y; finite                                                  */
    float   eps;        /* >= 0, finite; 0: q and k are used as they are                 */
    int32_t reserved;   /* 0                                                             */
} ss_gdr_dims;

typedef struct {          /* [B, L, heads, d] view: element (b, t, h, d) at p + b batch_stride + t token_stride + h head_stride + d */
    const void* p;        /* aligned to its element                                          */
    int64_t batch_stride; /* in elements, >= 0; ignored where B = 1                          */
    int64_t token_stride; /* in elements, >= 0; ignored where L = 1 and by ss_gdr_step       */
    int64_t head_stride;  /* in elements, >= 0; ignored where there is one head              */
} ss_head_view;

typedef struct {
    ss_head_view   q, k;     /* [B,L,k_heads,dk]                                             */
    ss_head_view   v;        /* [B,L,H,dv]                                                   */
    const float*   g;        /* [B,L,H] log decays                                           */
    const float*   beta;     /* [B,L,H]                                                      */
    const uint8_t* reset;    /* [B,L] ([B] for ss_gdr_step) or NULL (no resets)              */
    void*          y;        /* [B,L,H,dv] io OUT; must not overlap any input                */
    float*         state;    /* [B,H,dk,dv] IN/OUT, or NULL: zero initial state, final not returned.
                                Required by ss_gdr_step; not used by ss_gdr_bwd              */
    float*         ckpt;     /* ss_gdr_ckpt_floats values for the backward (the states before tokens 0, 64,
                                128, ..., [B,H,ceil(L/64),dk,dv], then u_t / beta_t, [B,L,H,dv]):
                                OUT of ss_gdr_fwd (NULL: not written), IN of ss_gdr_bwd      */
} ss_gdr_args;

/* Values of the checkpoints; 0 for invalid dims. */
size_t ss_gdr_ckpt_floats(const ss_gdr_dims* dims);

/* Bytes of device workspace of ss_gdr_fwd (backward = 0) or ss_gdr_bwd; 0 for invalid dims or L = 0. */
size_t ss_gdr_workspace_bytes(const ss_gdr_dims* dims, int backward);

/* L = 0: y is empty and the state stays as it is. */
ss_status ss_gdr_fwd(const ss_gdr_dims* dims, const ss_gdr_args* args, void* workspace, size_t workspace_bytes,
                     void* stream);

/* One token for every stream: q, k [B,k_heads,dk], v [B,H,dv], g, beta [B,H], y [B,H,dv]; state updated in place. */
ss_status ss_gdr_step(const ss_gdr_dims* dims, const ss_gdr_args* args, void* stream);

typedef struct {
    const void*  dy;           /* [B,L,H,dv] io: gradient of y (required)                        */
    const float* dstate_final; /* [B,H,dk,dv] or NULL (zero): gradient of the returned state     */
    void*  dq;                 /* [B,L,k_heads,dk] io OUT (required), summed over the heads that share it */
    void*  dk;                 /* [B,L,k_heads,dk] io OUT (required), likewise                   */
    void*  dv;                 /* [B,L,H,dv] io OUT (required)                                    */
    float* dg;                 /* [B,L,H] OUT (required); 0 at resets                             */
    float* dbeta;              /* [B,L,H] OUT (required)                                          */
    float* dstate_init;        /* [B,H,dk,dv] OUT or NULL: gradient of the initial state          */
} ss_gdr_grads;

/* Gradients of sum(dy * y) + sum(dstate_final * state_out) for the forward's inputs in `args`, whose
 * ckpt are the checkpoints that forward wrote (y and state are ignored). With W_t the gradient of S_t,
 *   W_t' = W_t + scale q^ dy^T,  dv = beta W_t'^T k^,  dk^ = W_t' u - S' dv,  dq^ = scale S_t dy,
 *   dbeta = (dv / beta) . (u / beta),  dS' = W_t' - k^ dv^T,  dg = <S', dS'>,  W_{t-1} = exp(g) dS'.
 * Outputs are overwritten; none may overlap an input, another output or the workspace. */
ss_status ss_gdr_bwd(const ss_gdr_dims* dims, const ss_gdr_args* args, const ss_gdr_grads* grads, void* workspace,
                     size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * The norms behind and before a layer, with its gate, its scale and the residual. Rows of M, columns of
 * K, in groups of `group` consecutive columns (heads; K: one group):
 *
 *   p = y / sqrt(mean over the group of y^2 + eps) * w      w [group], the same for every group
 *   h = p * gate * sigmoid(gate)                            h = p without a gate
 *   s = residual + scale * h                                scale [K]; without one 1, without a residual 0
 *   n = s / sqrt(mean over the row of s^2 + eps) * w_next   where n is asked for
 *
 * in fp32, with s and n each rounded once (n from s before it is rounded). All matrices are contiguous
 * row-major in the I/O dtype, weights and their gradients fp32. */
typedef struct {
    int64_t rows;       /* M, 1 <= M < 2^31                                              */
    int64_t cols;       /* K, 1 <= K <= 16384                                            */
    int64_t group;      /* a divisor of K                                                */
    int32_t io_dtype;   /* ss_dtype of y, gate, residual, s, n and their gradients       */
    float   eps;        /* > 0, finite                                                   */
} ss_gnorm_dims;

typedef struct {
    const void*  y;        /* [M,K] io                                                     */
    const float* w;        /* [group]                                                      */
    const void*  gate;     /* [M,K] io or NULL                                             */
    const void*  residual; /* [M,K] io or NULL                                             */
    const float* scale;    /* [K] or NULL                                                  */
    const float* w_next;   /* [K]; NULL: n is not made                                     */
    void*        s;        /* [M,K] io OUT; may be y, gate or residual itself. Not used by ss_gnorm_bwd */
    void*        n;        /* [M,K] io OUT; required with w_next, else NULL. Not used by ss_gnorm_bwd   */
} ss_gnorm_args;

ss_status ss_gnorm_fwd(const ss_gnorm_dims* dims, const ss_gnorm_args* args, void* stream);

typedef struct {
    const void* ds;        /* [M,K] io or NULL (zero): gradient of s                        */
    const void* dn;        /* [M,K] io or NULL (zero): gradient of n; only with w_next. One of the two is required */
    void*  dy;             /* [M,K] io OUT (required)                                       */
    void*  dgate;          /* [M,K] io OUT; required with a gate, else NULL                 */
    void*  dresidual;      /* [M,K] io OUT; required with a residual, else NULL             */
    float* dw;             /* [group] OUT (required), summed over rows and groups           */
    float* dscale;         /* [K] OUT; required with a scale, else NULL                     */
    float* dw_next;        /* [K] OUT; required with w_next, else NULL                      */
} ss_gnorm_grads;

size_t ss_gnorm_workspace_bytes(const ss_gnorm_dims* dims);   /* of ss_gnorm_bwd; 0 for invalid dims */

/* Gradients of sum(ds * s) + sum(dn * n) for the forward's inputs, from these alone. Outputs are overwritten;
 * none may overlap an input, another output or the workspace. */
ss_status ss_gnorm_bwd(const ss_gnorm_dims* dims, const ss_gnorm_args* args, const ss_gnorm_grads* grads, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_OPS_H */
