/*
 * libselscan: the operators around the selective scan (same library and conventions as
 * selscan.h, whose ss_dtype and ss_status are used here).
 *
 *   ss_glr_fwd, ss_glr_bwd, ss_glr_step   a gated linear recurrence: forward over whole
 *                                         sequences, its gradients, one decode token
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
 * A[d] <= 0 (not checked; a positive value gives NaN through the square root). A reset
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
 *                                                      term where A s_t = 0 makes w_t = 0).
 * Outputs are overwritten; none may overlap an input, another output or the workspace. */
ss_status ss_glr_bwd(const ss_glr_dims* dims, const ss_glr_args* args, const ss_glr_grads* grads, void* workspace,
                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SELSCAN_OPS_H */
