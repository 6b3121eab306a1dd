// Internal interface between the C-ABI layer of the delta-rule layer's operators (the gated delta rule,
// the norms around a layer; include/selscan_ops.h) and their HIP kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "selscan_ops.h"

namespace selscan {

constexpr int kGdrTri = 6 * 16 * 32;         // values of an upper triangle of 64 x 64 in its blocks of 16 x 32
constexpr int kGdrLow = 10 * 16 * 16;        // of a lower one in its tiles of 16 x 16
// bytes of a value of the inverse: three bf16 terms, or fp32
template <bool BF16> constexpr int kGdrInverseBytes = BF16 ? 6 : 4;

// One launch of the gated delta rule, already validated by the C-ABI layer.
struct LaunchGdr {
    enum Pass { kFwd, kBwd, kStep } pass;
    bool bf16;
    bool vec;                    // rows of q and k start on 16 bytes and hold whole accesses of 16 bytes
    bool vec_v;                  // 64 tokens of v lie within 32-bit offsets
    bool vec_y;                  // four columns of y are one access
    bool vec_dy, vec_ck, vec_dk; // the backward: whole accesses of 16 bytes of the gradient of y, of the checkpoints and of the
                                 // workspace, four columns of the gradients of q and k
    bool vec_state;              // the step: dv a multiple of 4, the state on 16 bytes
    int64_t B, L, nchunks;
    int H, Hk, dk, dv;
    float scale, eps;
    ss_head_view q, k, v;
    const float* g; const float* beta; const uint8_t* reset; void* y; float* state;
    float* ckpt;                 // [B, H, chunks, dk, dv] states in front of the chunks
    float* ckptX;                // [B, L, H, dv] solutions x_t
    ss_gdr_grads gr;
    // workspace
    int64_t seg;                 // chunks of a segment (all of them: one segment)
    int nseg;
    float *wE, *wM, *wF;         // several segments: [nseg, B, H, dk, dv] states in front of the segments (the first: the caller's, if
                                 // there is one), [nseg - 1, B, H, dk, dk] what they make of these, [nseg - 1, B, H] whether
                                 // anything of it is left
                                 // The backward: [nseg - 1, B, H, dk, dv] gradients of the states behind the segments in wE
    float* wX;                   // [nseg - 1, B, H, dk, dv] states behind the segments, written where they are not those in front of
                                 // the next ones (the backward: in front of a segment, and behind the one in front of it)
    uint32_t* wQ;                // [B, H, tiles of 64 columns, nseg, 4 waves] 1 where that is, 2 more where anything is not finite
    float *co, *wT;              // [B, H, chunks]: factors of tokens, inverses in the order of operands
    float *wS, *wV;              // the backward: [B, H, chunks, dk, dv] adjoints behind the chunks, [B, L, H, dv] gradients of v
    uint32_t* wG;                // the backward: [B, H, chunks, 4 waves] whether a chunk's gradients hold anything that is not finite
    float *part_q, *part_k;      // the backward where heads share keys: [B, L, H, dk] each head's share
    void* stream;
};
// Chunks of a segment, forward and backward. One after the other a chunk takes about as long as any work of its 64 columns;
// with segments the states, or their gradients, are made twice.
int64_t gdr_segment(int64_t BH, int64_t dv, int64_t nchunks, bool two);
int64_t gdr_segment_back(int64_t BH, int64_t dv, int64_t nchunks);
hipError_t launch_gdr_bf16(const LaunchGdr& p);
hipError_t launch_gdr_f32(const LaunchGdr& p);
inline hipError_t launch_gdr(const LaunchGdr& p) { return p.bf16 ? launch_gdr_bf16(p) : launch_gdr_f32(p); }

// The norms around a layer (forward or backward).
struct LaunchGnorm {
    bool bf16, vec, back;
    int64_t M, K, group;
    float eps;
    const void *y, *gate, *residual;
    const float *w, *scale, *w_next;
    void *s, *n;
    const void *ds, *dn;
    void *dy, *dgate, *dresidual;
    float *dw, *dscale, *dw_next;
    float* part;                 // workspace of the backward: [gnorm_groups, 3, K] sums of columns
    void* stream;
};
hipError_t launch_gnorm(const LaunchGnorm& p);
// workgroups of the backward, each with its rows' sums of columns
int64_t gnorm_groups(int64_t M, int64_t K);
constexpr int64_t kGnormMaxCols = 16384;

}  // namespace selscan
