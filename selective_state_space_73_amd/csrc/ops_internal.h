// Internal interface between the C-ABI layer of the operators (include/selscan_ops.h) and
// their HIP kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "selscan_internal.h"
#include "selscan_ops.h"

namespace selscan {

constexpr int kGlrCols = 128;       // channels per workgroup of the recurrence kernels (2 per lane)
constexpr int kGlrFwdChunk = 128;   // tokens of a forward chunk
// Tokens of a backward chunk. With many rows of tiles the shorter one, whose four waves a CU has
// twice (B 8, L 2048, D 5120, bf16: 313 us against 351 with 128); with few, half as many chunks
// to wait for (B 1, L 65536, D 1024: 322 against 380).
inline int64_t glr_bwd_chunk(int64_t B, int64_t D) { return B * ((D + kGlrCols - 1) / kGlrCols) >= 32 ? 64 : 128; }

// One launch of the recurrence, already validated by the C-ABI layer.
struct LaunchGlr {
    enum Pass { kFwd, kBwd, kStep } pass;
    bool bf16;
    bool vec;                    // every row starts on two elements and D is even: two channels per access
    int64_t batch, L, D;
    ss_view x, r, i;
    const float* A; const uint8_t* reset; void* y; float* state; float* ckpt;
    ss_glr_grads g;
    int64_t chunk, nchunks;      // tokens of a chunk, chunks per batch row
    unsigned* ticket;            // workspace: next tile to take (several chunks only)
    uint64_t* slots;             // workspace: [nchunks, B, D] published chunk results (several chunks only)
    float* part;                 // workspace of the backward: [nchunks, B, D] parts of dA
    void* stream;
};
hipError_t launch_glr(const LaunchGlr& p);

// Rounding to 8 bits, with (w given) or without the norm in front.
constexpr int64_t kQ8WaveRows = 1024;    // rows from which a row has one wave, not a workgroup of four
struct LaunchQ8 {
    bool bf16, vec, square;
    const void* x; const void* res; const float* w; float eps;
    uint8_t* q; float* scale; void* sum;
    int64_t M, K;
    void* stream;
};
hipError_t launch_q8(const LaunchQ8& p);

// Y[M, N] = (xq xs)(wq ws)^T (+ R). Y may lie in two matrices side by side: columns
// [0, split) in Y[0] and the rest in Y[1] (split = N: one matrix).
struct LaunchGemmQ8 {
    bool y_bf16;
    const uint8_t* xq; const float* xs; const uint8_t* wq; const float* ws;
    const void* R; void* Y[2];
    int64_t split, M, N, K;
    void* stream;
};
hipError_t launch_gemm_q8(const LaunchGemmQ8& p);

}  // namespace selscan
