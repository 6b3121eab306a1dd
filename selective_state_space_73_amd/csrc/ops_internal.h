// Internal interface between the C-ABI layer of the operators (include/selscan_ops.h) and
// their HIP kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "selscan_internal.h"
#include "selscan_ops.h"

namespace selscan {

constexpr int kGlrCols = 128;       // channels per workgroup of the recurrence kernels (2 per lane)
// Few tiles: chunks of 64 tokens, whose runs of 8 by eight waves spread over more CUs (a CU's
// arithmetic is what the time goes to there), as long as the chunks to wait for are not too many.
// Forward, up to one such tile a CU: B 1, L 300, D 512, fp32 10.4 us against 14.2 with chunks of
// 128, bf16 10.2 against 12.9; with 320 tiles (L 600, D 4096) 20.3 against 17.1, with L 4800, D 100
// 20.2 against 18.1. Backward, one workgroup a CU against two of the other kernel's, up to the
// crossover between three and four of its rounds (us in bf16 and fp32, then the other kernel's): 300 tiles
// (B 1, L 300, D 7680) 28 34, 32 37; 512 (B 1, L 2000, D 2048) 37 45, 42 55; 640 (B 8, L 500, D 1280) 43 52, 50 60;
// 768 (B 4, L 1000, D 1536) 48 58, 53 66; 896 (B 1, L 1000, D 7168) 53 65, 55 68 and (B 1, L 2000, D 3584) 55 67, 52 67;
// 960 (B 4, L 1000, D 1920) 56 67, 56 70; 1008 (B 2, L 4000, D 1024) 61 76, 60 77; 1024 (B 8, L 500, D 2048) 59 71, 55 72.
inline bool glr_fine(bool backward, int64_t B, int64_t L, int64_t D) {
    return L <= (backward ? 4096 : 2048) && B * ((D + kGlrCols - 1) / kGlrCols) * ((L + 63) / 64) <= (backward ? 896 : 256);
}

// Tokens of a forward chunk. Few rows of tiles, long sequences: twice as many, half as many
// chunks to wait for (bf16: B 1, L 131072, D 2048 557 us against 620 with 128, B 3, L 16384,
// D 512 64 against 73, B 1, L 262144, D 128 125 against 221); shorter, or with tiles enough, two
// workgroups a CU are better than one of twice the waves (B 1, L 1024, D 2048 14.8 us against
// 20.2 with 256, B 8, L 2048, D 5120 165 against 180). fp32 runs have half the tokens, and a
// workgroup no room for more waves.
inline int64_t glr_fwd_chunk(bool bf16, int64_t B, int64_t L, int64_t D) {
    if (L > 128 && glr_fine(false, B, L, D)) return 64;
    return bf16 && L >= 4096 && B * ((D + kGlrCols - 1) / kGlrCols) < 64 ? 256 : 128;
}
// Tokens of a backward chunk. With many rows of tiles the shorter one, whose four waves a CU has
// twice (a call with B 8, L 2048, D 5120, bf16: 337 us against 378 with 128, fp32 473 against 488); with
// few, half as many chunks to wait for (B 1, L 65536, D 1024, bf16: 348 against 396, fp32 475 against 487).
inline int64_t glr_bwd_chunk(int64_t B, int64_t L, int64_t D) {
    return glr_fine(true, B, L, D) || B * ((D + kGlrCols - 1) / kGlrCols) >= 32 ? 64 : 128;
}

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
constexpr int64_t kQ8LaunchRows = int64_t(1) << 22;
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
