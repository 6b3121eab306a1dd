// Device code of the gated linear recurrence (ss_glr_fwd, ss_glr_bwd, ss_glr_step).
//
//   s = sigmoid(r), a = exp(A s), w = sqrt(1 - a^2), h_t = a_t h_{t-1} + w_t sigmoid(i_t) x_t
//
// Mapping: a lane owns two channels, a wave a run of TT consecutive tokens of 128 channels,
// a workgroup of NW waves a tile of NW * TT tokens (a chunk). Each wave loads its whole run
// at once, so a workgroup has its tile's bytes in flight together, and reduces it in
// registers to the pair (P, S) of the map h -> P h + S over its tokens. The pairs of the
// workgroup's waves meet in LDS, which gives every wave the state in front of its run once
// the state in front of the chunk is known; y_t = S_t + P_t h_in then needs no second read
// of the inputs. One pass: every input is read once and every output written once.
//
// The chunks of one channel depend on each other. A workgroup publishes its chunk's (P, S)
// in a 64-bit word per channel and looks back over the earlier chunks' words for the
// nearest one whose state is known, folds the pairs after it, and replaces its own word by
// the state after its chunk. The fold runs from the known state forward, the same
// operations in the same order wherever it starts, so results do not depend on timing.
//
// Progress: chunks are handed out in order by a ticket counter, so a workgroup waits only
// for chunks that other running workgroups hold, and the lowest unfinished one waits for
// nobody. Each word carries its own state (kEmpty until it is published), is written and
// read with one 64-bit access at device scope, and no other memory is handed over, so no
// fences are needed between the workgroups.
//
// A reset (a = 0, the state before it not read) is kept as a product P of -0.0, which no
// product of non-negative decays gives: folds take S alone there, so a NaN or an infinity
// of one document does not reach the next.
#pragma once
#include "ops_internal.h"
#include "selscan_device.h"

namespace selscan {

// ---------------------------------------------------------------------------
// gates

// expm1(v) for |v| below kEm1Small by its Taylor polynomial (the first dropped term is
// below 2^-26 of the result); elsewhere exp(v) - 1, which loses at most two bits there.
constexpr float kEm1Small = 0.35f;
__device__ __forceinline__ float expm1_small(float v) {
    float p = 1.0f / 5040.0f;
    p = __builtin_fmaf(p, v, 1.0f / 720.0f);
    p = __builtin_fmaf(p, v, 1.0f / 120.0f);
    p = __builtin_fmaf(p, v, 1.0f / 24.0f);
    p = __builtin_fmaf(p, v, 1.0f / 6.0f);
    p = __builtin_fmaf(p, v, 0.5f);
    p = __builtin_fmaf(p, v, 1.0f);
    return p * v;
}

__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.0f + exp2_fast(-kLog2e * v)); }

struct Gate { float s, g, la, a, w2; };   // sigmoid(r), sigmoid(i), A s, exp(A s), 1 - a^2

// The decay near 1 is what a long memory is made of: there a = 1 + expm1(A s), so that its
// error is the rounding of the sum alone, and 1 - a^2 = -e (2 + e) with e = expm1(A s) keeps
// its relative accuracy where 1 - a * a would cancel.
__device__ __forceinline__ Gate glr_gate(float r, float i, float A) {
    Gate q;
    q.s = sigmoid(r);
    q.g = sigmoid(i);
    q.la = A * q.s;
    const float ex = exp2_fast(kLog2e * q.la);
    const float e = __builtin_fabsf(q.la) < kEm1Small ? expm1_small(q.la) : ex - 1.0f;
    q.a = __builtin_fabsf(q.la) < kEm1Small ? 1.0f + e : ex;
    q.w2 = -e * (2.0f + e);
    return q;
}

// ---------------------------------------------------------------------------
// two channels of one row: loads, stores, conversions

template <typename T, bool VEC> struct Pair;
template <> struct Pair<float, true> {
    typedef float v2 __attribute__((ext_vector_type(2)));
    v2 v;
    __device__ __forceinline__ void ld(const float* p, int c0, int) { v = *reinterpret_cast<const v2*>(p + c0); }
    __device__ __forceinline__ float get(int j) const { return v[j]; }
    static __device__ __forceinline__ void st(float* p, int c0, int, bool ok0, bool, float a, float b) {
        if (ok0) *reinterpret_cast<v2*>(p + c0) = v2{a, b};
    }
};
template <> struct Pair<uint16_t, true> {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    uint32_t v;
    __device__ __forceinline__ void ld(const uint16_t* p, int c0, int) { v = *reinterpret_cast<const uint32_t*>(p + c0); }
    __device__ __forceinline__ float get(int j) const {
        return __builtin_bit_cast(float, j ? (v & 0xffff0000u) : (v << 16));
    }
    static __device__ __forceinline__ void st(uint16_t* p, int c0, int, bool ok0, bool, float a, float b) {
        if (ok0) *reinterpret_cast<b2*>(p + c0) = __builtin_convertvector((f2{a, b}), b2);
    }
};
template <typename T> struct Pair<T, false> {
    T v[2];
    __device__ __forceinline__ void ld(const T* p, int c0, int c1) { v[0] = p[c0]; v[1] = p[c1]; }
    __device__ __forceinline__ float get(int j) const { return IO<T>::cvt(v[j]); }
    static __device__ __forceinline__ void st(T* p, int c0, int c1, bool ok0, bool ok1, float a, float b) {
        if (ok0) IO<T>::st(p + c0, a);
        if (ok1) IO<T>::st(p + c1, b);
    }
};

// The two channels of a lane: next to each other where rows allow one access for both,
// else 64 apart, so that a wave's accesses stay contiguous. Lanes past the last channel
// repeat it (their loads stay in range) and store nothing.
struct Chan { int c[2]; bool ok[2]; };
template <bool VEC>
__device__ __forceinline__ Chan lane_chan(int col, int lane, int D) {
    Chan q;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = col * kGlrCols + (VEC ? 2 * lane + j : lane + 64 * j);
        q.ok[j] = c < D;
        q.c[j] = q.ok[j] ? c : (VEC ? D - 2 + j : D - 1);
    }
    return q;
}
// position of a lane's channel j among the workgroup's 128 (LDS arrays)
template <bool VEC> __device__ __forceinline__ int lane_slot(int lane, int j) { return VEC ? 2 * lane + j : lane + 64 * j; }

// ---------------------------------------------------------------------------
// the maps h -> P h + S and their words

constexpr uint32_t kResetBits = 0x80000000u;              // P = -0.0: the state in front is not read
constexpr uint64_t kEmpty = ~uint64_t(0);                 // nothing published yet
constexpr uint32_t kStateTag = 0xfffffffeu;               // the word holds the state after its chunk

__device__ __forceinline__ bool is_reset(float P) { return __builtin_bit_cast(uint32_t, P) == kResetBits; }
__device__ __forceinline__ float fold(float P, float h, float S) { return is_reset(P) ? S : __builtin_fmaf(P, h, S); }
__device__ __forceinline__ float fold_p(float P, float before) { return is_reset(P) ? P : P * before; }

__device__ __forceinline__ uint64_t map_word(float P, float S) {
    const uint32_t p = P != P ? 0x7fc00000u : __builtin_bit_cast(uint32_t, P);   // no NaN looks like a tag
    return (uint64_t)p << 32 | __builtin_bit_cast(uint32_t, S);
}
__device__ __forceinline__ uint64_t state_word(float h) {
    return (uint64_t)kStateTag << 32 | __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ uint32_t word_tag(uint64_t v) { return (uint32_t)(v >> 32); }
__device__ __forceinline__ float word_lo(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)v); }
__device__ __forceinline__ uint64_t word_load(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void word_store(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state in front of a chunk, for one channel: `word` is the word of the chunk just in
// front, the n words of the chunks in front lie `stride` apart towards it, and the first of
// them always ends up as a state. Looks back for the nearest state in groups of kLook words
// loaded together, waiting where a word is still empty, then folds forward from it.
constexpr int kLook = 8;
__device__ __forceinline__ float look_back(const uint64_t* word, int64_t stride, int n) {
    int back = 0;                                  // words between `word` and the one looked at
    for (bool found = false; !found;) {
        uint64_t v[kLook];
#pragma unroll
        for (int q = 0; q < kLook; ++q) {
            const int k = back + q < n ? back + q : n - 1;
            v[q] = word_load(word + (int64_t)k * stride);
        }
        bool stop = false;
#pragma unroll
        for (int q = 0; q < kLook; ++q) {
            if (!stop) {
                if (word_tag(v[q]) == kStateTag) found = stop = true;
                else if (v[q] == kEmpty) { stop = true; __builtin_amdgcn_s_sleep(1); }
                else if (back < n - 1) ++back;
            }
        }
    }
    float h = 0.0f;
    // from the state forward; a word read now may have become a state itself, equal to the fold
    for (int k = back; k >= 0; k -= kLook) {
        uint64_t v[kLook];
#pragma unroll
        for (int q = 0; q < kLook; ++q) v[q] = word_load(word + (int64_t)(k - q > 0 ? k - q : 0) * stride);
#pragma unroll
        for (int q = 0; q < kLook; ++q)
            if (k - q >= 0)
                h = word_tag(v[q]) == kStateTag ? word_lo(v[q])
                                                : fold(__builtin_bit_cast(float, word_tag(v[q])), h, word_lo(v[q]));
    }
    return h;
}

__global__ void __launch_bounds__(256)
k_glr_clear(uint64_t* slots, int64_t n, unsigned* ticket) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i0 == 0) *ticket = 0;
    for (int64_t i = i0; i < n; i += (int64_t)gridDim.x * 256) slots[i] = kEmpty;
}

struct GlrArgs {
    const void* x; const void* r; const void* i;
    int64_t xb, xt, rb, rt, ib, it;              // batch and token strides
    const float* A; const uint8_t* reset; void* y; float* state; float* ckpt;
    const void* dy; const float* dstate_final; void* dx; void* dr; void* di; float* dstate_init;
    float* part;                                  // [nchunks, B, D] parts of dA
    int64_t L; int B, D, ncol, nchunks, nck;
    unsigned tiles;                               // nchunks * B * ncol
    unsigned* ticket; uint64_t* slots;
};

// A tile's place: chunk, batch row and column group. Chunks are the slowest index, so that
// tiles in flight at the same time belong to as few chunks as possible.
struct Tile { int chunk, b, col; };
__device__ __forceinline__ Tile tile_at(const GlrArgs& p, unsigned t) {
    const unsigned per = (unsigned)p.B * (unsigned)p.ncol;
    Tile q;
    q.chunk = (int)(t / per);
    const unsigned in = t % per;
    q.b = (int)(in / (unsigned)p.ncol);
    q.col = (int)(in % (unsigned)p.ncol);
    return q;
}

// Bit k: token t0 + k of batch row b resets. One load for the wave, a lane per token.
template <int TT>
__device__ __forceinline__ uint32_t reset_bits(const GlrArgs& p, int b, int64_t t0, int lane) {
    if (!p.reset) return 0u;
    const int64_t t = t0 + lane;
    const bool on = lane < TT && t < p.L && p.reset[(int64_t)b * p.L + t] != 0;
    return (uint32_t)__ballot(on);
}

// ---------------------------------------------------------------------------
// forward. LOOK: several chunks per batch row, tiles taken by ticket; else one chunk, a
// workgroup per tile.

template <typename T, bool VEC, int TT, int NW, bool LOOK>
__global__ void __launch_bounds__(NW * 64)
k_glr_fwd(const GlrArgs p) {
    using V = Pair<T, VEC>;
    __shared__ float2 s_map[NW][kGlrCols];        // (P, S) of each wave's run
    __shared__ float s_in[NW][kGlrCols];          // state in front of each wave's run
    __shared__ unsigned s_next;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const T* X = static_cast<const T*>(p.x);
    const T* R = static_cast<const T*>(p.r);
    const T* I = static_cast<const T*>(p.i);

    V vx[TT], vr[TT], vi[TT];
    uint32_t resets = 0;
    float A[2];
    auto fetch = [&](unsigned t) {
        const Tile q = tile_at(p, t);
        const Chan c = lane_chan<VEC>(q.col, lane, p.D);
        const int64_t t0 = (int64_t)q.chunk * (NW * TT) + wave * TT;
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            const int64_t tk = t0 + k < p.L ? t0 + k : p.L - 1;
            vx[k].ld(X + q.b * p.xb + tk * p.xt, c.c[0], c.c[1]);
            vr[k].ld(R + q.b * p.rb + tk * p.rt, c.c[0], c.c[1]);
            vi[k].ld(I + q.b * p.ib + tk * p.it, c.c[0], c.c[1]);
        }
        A[0] = p.A[c.c[0]];
        A[1] = p.A[c.c[1]];
        resets = reset_bits<TT>(p, q.b, t0, lane);
    };

    unsigned tile = blockIdx.x;
    if constexpr (LOOK) {
        if (tid == 0) s_next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        tile = __builtin_amdgcn_readfirstlane(s_next);
        __syncthreads();
    }
    if (tile < p.tiles) fetch(tile);
    while (tile < p.tiles) {
        unsigned next = p.tiles;
        if constexpr (LOOK) {
            if (tid == 0) next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        const Tile q = tile_at(p, tile);
        const Chan c = lane_chan<VEC>(q.col, lane, p.D);
        const int64_t t0 = (int64_t)q.chunk * (NW * TT) + wave * TT;
        const int n = (int)(p.L - t0 < TT ? p.L - t0 : TT);      // tokens of this run, 0 or less past the end
        const uint32_t rs = resets;

        // the run from a zero state: h[k] the local state, P[k] what a state in front is multiplied by
        float P[TT][2], h[TT][2];
#pragma unroll
        for (int k = 0; k < TT; ++k) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const Gate g = glr_gate(vr[k].get(j), vi[k].get(j), A[j]);
                const float v = g.g * vx[k].get(j);
                const float Pp = k ? P[k - 1][j] : 1.0f, hp = k ? h[k - 1][j] : 0.0f;
                if (k < n) {                                      // uniform over the wave
                    if (rs >> k & 1u) {
                        P[k][j] = -0.0f;
                        h[k][j] = v;
                    } else {
                        P[k][j] = g.a * Pp;
                        h[k][j] = __builtin_fmaf(g.a, hp, __builtin_amdgcn_sqrtf(g.w2) * v);
                    }
                } else {
                    P[k][j] = Pp;
                    h[k][j] = hp;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) s_map[wave][lane_slot<VEC>(lane, j)] = make_float2(P[TT - 1][j], h[TT - 1][j]);
        if (LOOK && tid == 0) s_next = next;
        __syncthreads();
        if constexpr (LOOK) {
            next = __builtin_amdgcn_readfirstlane(s_next);
            if (next < p.tiles) fetch(next);                      // the next tile's loads run under what follows
        }

        // the states in front of the runs: one lane per channel
        if (tid < kGlrCols && q.col * kGlrCols + tid < p.D) {
            const int64_t bd = (int64_t)q.b * p.D + q.col * kGlrCols + tid;
            const int64_t BD = (int64_t)p.B * p.D;
            float2 m[NW];
#pragma unroll
            for (int w = 0; w < NW; ++w) m[w] = s_map[w][tid];
            float in;
            if (LOOK && q.chunk > 0) {
                float cp = 1.0f, cs = 0.0f;
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    cs = fold(m[w].x, cs, m[w].y);
                    cp = fold_p(m[w].x, cp);
                }
                uint64_t* word = p.slots + (int64_t)q.chunk * BD + bd;
                if (q.chunk + 1 < p.nchunks) word_store(word, map_word(cp, cs));
                in = look_back(word - BD, -BD, q.chunk);
                if (q.chunk + 1 < p.nchunks) word_store(word, state_word(fold(cp, in, cs)));
            } else {
                in = p.state ? p.state[bd] : 0.0f;
            }
            float hh = in;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                s_in[w][tid] = hh;
                hh = fold(m[w].x, hh, m[w].y);
            }
            if (LOOK && q.chunk == 0) word_store(p.slots + bd, state_word(hh));
        }
        __syncthreads();

        float in[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) in[j] = s_in[wave][lane_slot<VEC>(lane, j)];
        if (p.ckpt && n > 0 && t0 % SS_GLR_CKPT == 0)
            Pair<float, VEC>::st(p.ckpt + ((int64_t)q.b * p.nck + t0 / SS_GLR_CKPT) * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1],
                                 in[0], in[1]);
        T* yrow = static_cast<T*>(p.y) + ((int64_t)q.b * p.L + t0) * p.D;
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            if (k < n) {
                float o[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) o[j] = rs ? fold(P[k][j], in[j], h[k][j]) : __builtin_fmaf(P[k][j], in[j], h[k][j]);
                V::st(yrow + (int64_t)k * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], o[0], o[1]);
                if (p.state && t0 + k == p.L - 1)
                    Pair<float, VEC>::st(p.state + (int64_t)q.b * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], o[0], o[1]);
            }
        }
        if constexpr (!LOOK) break;
        tile = next;
    }
}

// ---------------------------------------------------------------------------
// backward: the same tiles, taken from the last chunk to the first. The states in front of
// the runs come from the forward's checkpoints and the runs' maps; what passes from a token
// to the one before it is K_t = a_t g_t, whose map over a run is K -> P K + S with the
// forward's P. Sums of dA over a run stay in registers, over a chunk in LDS; k_glr_da adds
// the chunks.

template <typename T, bool VEC, int TT, int NW, bool LOOK>
__global__ void __launch_bounds__(NW * 64)
k_glr_bwd(const GlrArgs p) {
    static_assert(SS_GLR_CKPT % TT == 0 && (NW * TT) % SS_GLR_CKPT == 0, "checkpoints lie at starts of runs");
    using V = Pair<T, VEC>;
    __shared__ float s_p[NW][kGlrCols], s_f[NW][kGlrCols], s_b[NW][kGlrCols];   // P and both S of each run
    __shared__ float s_h[NW][kGlrCols], s_k[NW][kGlrCols];                      // state in front, K from behind
    __shared__ float s_a[NW][kGlrCols];                                         // parts of dA
    __shared__ unsigned s_next;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const T* X = static_cast<const T*>(p.x);
    const T* R = static_cast<const T*>(p.r);
    const T* I = static_cast<const T*>(p.i);
    const T* DY = static_cast<const T*>(p.dy);

    for (unsigned tile = blockIdx.x;;) {
        if constexpr (LOOK) {
            __syncthreads();                                     // the last tile's s_next and s_a are read
            if (tid == 0) s_next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            tile = __builtin_amdgcn_readfirstlane(s_next);
            if (tile >= p.tiles) break;
        }
        Tile q = tile_at(p, tile);
        q.chunk = p.nchunks - 1 - q.chunk;
        const Chan c = lane_chan<VEC>(q.col, lane, p.D);
        const int64_t t0 = (int64_t)q.chunk * (NW * TT) + wave * TT;
        const int n = (int)(p.L - t0 < TT ? p.L - t0 : TT);

        V vx[TT], vd[TT];
        float s[TT][2], g[TT][2], a[TT][2], w[TT][2];
        float A[2], P[2] = {1.0f, 1.0f}, Sf[2] = {0.0f, 0.0f}, Sb[2] = {0.0f, 0.0f};
        uint32_t rs;
        {
            V vr[TT], vi[TT];
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                const int64_t tk = t0 + k < p.L ? t0 + k : p.L - 1;
                vx[k].ld(X + q.b * p.xb + tk * p.xt, c.c[0], c.c[1]);
                vr[k].ld(R + q.b * p.rb + tk * p.rt, c.c[0], c.c[1]);
                vi[k].ld(I + q.b * p.ib + tk * p.it, c.c[0], c.c[1]);
                vd[k].ld(DY + ((int64_t)q.b * p.L + tk) * p.D, c.c[0], c.c[1]);
            }
            A[0] = p.A[c.c[0]];
            A[1] = p.A[c.c[1]];
            rs = reset_bits<TT>(p, q.b, t0, lane);
#pragma unroll
            for (int k = 0; k < TT; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const Gate e = glr_gate(vr[k].get(j), vi[k].get(j), A[j]);
                    s[k][j] = e.s;
                    g[k][j] = e.g;
                    a[k][j] = e.a;
                    w[k][j] = __builtin_amdgcn_sqrtf(e.w2);
                    if (k < n) {
                        const float v = e.g * vx[k].get(j);
                        if (rs >> k & 1u) {
                            a[k][j] = 0.0f;
                            w[k][j] = 1.0f;
                            P[j] = -0.0f;
                            Sf[j] = v;
                        } else {
                            P[j] *= e.a;
                            Sf[j] = __builtin_fmaf(e.a, Sf[j], w[k][j] * v);
                        }
                    }
                }
        }
#pragma unroll
        for (int k = TT - 1; k >= 0; --k)
            if (k < n)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    Sb[j] = (rs >> k & 1u) ? 0.0f : a[k][j] * (vd[k].get(j) + Sb[j]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = lane_slot<VEC>(lane, j);
            s_p[wave][at] = P[j];
            s_f[wave][at] = Sf[j];
            s_b[wave][at] = Sb[j];
        }
        __syncthreads();

        if (tid < kGlrCols && q.col * kGlrCols + tid < p.D) {
            const int ch = q.col * kGlrCols + tid;
            const int64_t bd = (int64_t)q.b * p.D + ch;
            const int64_t BD = (int64_t)p.B * p.D;
            float mp[NW], mb[NW];
#pragma unroll
            for (int v = 0; v < NW; ++v) { mp[v] = s_p[v][tid]; mb[v] = s_b[v][tid]; }
            float cp = 1.0f, cs = 0.0f;
#pragma unroll
            for (int v = NW - 1; v >= 0; --v) {
                cs = fold(mp[v], cs, mb[v]);
                cp = fold_p(mp[v], cp);
            }
            uint64_t* word = p.slots + (int64_t)q.chunk * BD + bd;
            float in;
            if (LOOK && q.chunk + 1 < p.nchunks) {
                if (q.chunk > 0) word_store(word, map_word(cp, cs));
                in = look_back(word + BD, BD, p.nchunks - 1 - q.chunk);
            } else {
                in = p.dstate_final ? p.dstate_final[bd] : 0.0f;
            }
            if (LOOK && q.chunk > 0) word_store(word, state_word(fold(cp, in, cs)));
#pragma unroll
            for (int v = NW - 1; v >= 0; --v) {
                s_k[v][tid] = in;
                in = fold(mp[v], in, mb[v]);
            }
            float h = 0.0f;
#pragma unroll
            for (int v = 0; v < NW; ++v) {
                const int64_t tv = (int64_t)q.chunk * (NW * TT) + v * TT;
                if (v * TT % SS_GLR_CKPT == 0) h = tv < p.L ? p.ckpt[((int64_t)q.b * p.nck + tv / SS_GLR_CKPT) * p.D + ch] : 0.0f;
                s_h[v][tid] = h;
                h = fold(mp[v], h, s_f[v][tid]);
            }
        }
        __syncthreads();

        // the run again, now with the true states: hb[k] the state before token k
        float hb[TT][2], K[2], dA[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float h = s_h[wave][lane_slot<VEC>(lane, j)];
            K[j] = s_k[wave][lane_slot<VEC>(lane, j)];
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                hb[k][j] = h;
                const float b = w[k][j] * (g[k][j] * vx[k].get(j));
                h = (rs >> k & 1u) ? b : __builtin_fmaf(a[k][j], h, b);
            }
        }
        const int64_t row0 = ((int64_t)q.b * p.L + t0) * p.D;
#pragma unroll
        for (int k = TT - 1; k >= 0; --k) {
            if (k < n) {
                float dx[2], dr[2], di[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float x = vx[k].get(j), G = vd[k].get(j) + K[j];
                    const float gw = G * w[k][j], v = g[k][j] * x;
                    dx[j] = gw * g[k][j];
                    di[j] = gw * (v * (1.0f - g[k][j]));
                    if (rs >> k & 1u) {
                        K[j] = 0.0f;
                        dr[j] = 0.0f;
                    } else {
                        const float rw = w[k][j] > 0.0f ? rcp_fast(w[k][j]) : 0.0f;
                        K[j] = a[k][j] * G;
                        const float dla = K[j] * (hb[k][j] - a[k][j] * rw * v);
                        dr[j] = dla * (A[j] * s[k][j]) * (1.0f - s[k][j]);
                        dA[j] = __builtin_fmaf(dla, s[k][j], dA[j]);
                    }
                }
                const int64_t o = row0 + (int64_t)k * p.D;
                V::st(static_cast<T*>(p.dx) + o, c.c[0], c.c[1], c.ok[0], c.ok[1], dx[0], dx[1]);
                V::st(static_cast<T*>(p.dr) + o, c.c[0], c.c[1], c.ok[0], c.ok[1], dr[0], dr[1]);
                V::st(static_cast<T*>(p.di) + o, c.c[0], c.c[1], c.ok[0], c.ok[1], di[0], di[1]);
            }
        }
        if (p.dstate_init && t0 == 0)
            Pair<float, VEC>::st(p.dstate_init + (int64_t)q.b * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], K[0], K[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) s_a[wave][lane_slot<VEC>(lane, j)] = dA[j];
        __syncthreads();
        if (tid < kGlrCols && q.col * kGlrCols + tid < p.D) {
            float t = s_a[0][tid];
#pragma unroll
            for (int v = 1; v < NW; ++v) t += s_a[v][tid];
            p.part[((int64_t)q.chunk * p.B + q.b) * p.D + q.col * kGlrCols + tid] = t;
        }
        if constexpr (!LOOK) break;
    }
}

// dA[d]: the sum of `rows` parts, 16 waves of a workgroup taking every 16th row of its 64
// channels; in 64 bits, in a fixed order.
__global__ void __launch_bounds__(1024)
k_glr_da(const float* __restrict__ part, float* __restrict__ dA, int64_t rows, int D) {
    __shared__ double sum[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int d = blockIdx.x * 64 + lane;
    double t = 0.0;
    if (d < D)
#pragma unroll 8
        for (int64_t k = wave; k < rows; k += 16) t += (double)part[k * D + d];
    sum[wave][lane] = t;
    __syncthreads();
    if (wave == 0 && d < D) {
#pragma unroll
        for (int v = 1; v < 16; ++v) t += sum[v][lane];
        dA[d] = (float)t;
    }
}

// ---------------------------------------------------------------------------
// one token per stream: a lane per two channels

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_glr_step(const GlrArgs p) {
    using V = Pair<T, VEC>;
    using F = Pair<float, VEC>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t at = (int64_t)blockIdx.x * 4 + wave;
    if (at >= (int64_t)p.B * p.ncol) return;
    const int b = (int)(at / p.ncol), col = (int)(at % p.ncol);
    const Chan c = lane_chan<VEC>(col, lane, p.D);
    V x, r, i;
    F h, A;
    x.ld(static_cast<const T*>(p.x) + b * p.xb, c.c[0], c.c[1]);
    r.ld(static_cast<const T*>(p.r) + b * p.rb, c.c[0], c.c[1]);
    i.ld(static_cast<const T*>(p.i) + b * p.ib, c.c[0], c.c[1]);
    h.ld(p.state + (int64_t)b * p.D, c.c[0], c.c[1]);
    if (VEC) A.ld(p.A, c.c[0], c.c[1]);
    else { A.ld(p.A, c.c[0], c.c[1]); }
    const bool rs = p.reset && p.reset[b] != 0;
    float o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const Gate g = glr_gate(r.get(j), i.get(j), A.get(j));
        const float v = g.g * x.get(j);
        o[j] = rs ? v : __builtin_fmaf(g.a, h.get(j), __builtin_amdgcn_sqrtf(g.w2) * v);
    }
    F::st(p.state + (int64_t)b * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], o[0], o[1]);
    V::st(static_cast<T*>(p.y) + (int64_t)b * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], o[0], o[1]);
}

// ---------------------------------------------------------------------------
// launches

inline GlrArgs glr_args(const LaunchGlr& p) {
    GlrArgs a{};
    a.x = p.x.p; a.xb = p.x.batch_stride; a.xt = p.x.token_stride;
    a.r = p.r.p; a.rb = p.r.batch_stride; a.rt = p.r.token_stride;
    a.i = p.i.p; a.ib = p.i.batch_stride; a.it = p.i.token_stride;
    a.A = p.A; a.reset = p.reset; a.y = p.y; a.state = p.state; a.ckpt = p.ckpt;
    a.dy = p.g.dy; a.dstate_final = p.g.dstate_final; a.dx = p.g.dx; a.dr = p.g.dr; a.di = p.g.di;
    a.dstate_init = p.g.dstate_init;
    a.part = p.part;
    a.L = p.L; a.B = (int)p.batch; a.D = (int)p.D;
    a.ncol = (int)((p.D + kGlrCols - 1) / kGlrCols);
    a.nchunks = (int)p.nchunks;
    a.nck = (int)((p.L + SS_GLR_CKPT - 1) / SS_GLR_CKPT);
    a.tiles = (unsigned)(p.nchunks * p.batch * a.ncol);
    a.ticket = p.ticket; a.slots = p.slots;
    return a;
}

constexpr unsigned kGlrGroups = 1024;    // workgroups of a ticketed launch: more than are resident at once

template <typename T, bool VEC>
hipError_t launch_glr_t(const LaunchGlr& p) {
    const GlrArgs a = glr_args(p);
    hipStream_t st = static_cast<hipStream_t>(p.stream);
    const bool look = p.nchunks > 1;
    if (p.pass == LaunchGlr::kStep) {
        const int64_t waves = p.batch * a.ncol;
        hipLaunchKernelGGL((k_glr_step<T, VEC>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    if (look) {
        const int64_t n = p.nchunks * p.batch * p.D;
        const int64_t groups = (n + 1023) / 1024;
        hipLaunchKernelGGL(k_glr_clear, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, st, p.slots, n, p.ticket);
    }
    const dim3 grid(look && a.tiles > kGlrGroups ? kGlrGroups : a.tiles);
    if (p.pass == LaunchGlr::kFwd) {
        const dim3 block(kGlrFwdWaves * 64);
        if (look) hipLaunchKernelGGL((k_glr_fwd<T, VEC, kGlrFwdTokens, kGlrFwdWaves, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_glr_fwd<T, VEC, kGlrFwdTokens, kGlrFwdWaves, false>), grid, block, 0, st, a);
    } else {
        const dim3 block(kGlrBwdWaves * 64);
        if (look) hipLaunchKernelGGL((k_glr_bwd<T, VEC, kGlrBwdTokens, kGlrBwdWaves, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_glr_bwd<T, VEC, kGlrBwdTokens, kGlrBwdWaves, false>), grid, block, 0, st, a);
        hipLaunchKernelGGL(k_glr_da, dim3((unsigned)((p.D + 63) / 64)), dim3(1024), 0, st, p.part, p.g.dA,
                           p.nchunks * p.batch, (int)p.D);
    }
    return hipGetLastError();
}

}  // namespace selscan
