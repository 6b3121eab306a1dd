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

// expm1(v) near 0: its Taylor polynomial up to v^5 (the first dropped term, v^5 / 720 of the
// result, is below 2^-24 for |v| < kEm1Small, and a decay remembers 1 / |v| tokens of it).
// Further out exp(v) - 1 loses three bits at most.
constexpr float kEm1Small = 0.125f;
__device__ __forceinline__ float expm1_small(float v) {
    float p = __builtin_fmaf(v, 1.0f / 120.0f, 1.0f / 24.0f);
    p = __builtin_fmaf(p, v, 1.0f / 6.0f);
    p = __builtin_fmaf(p, v, 0.5f);
    p = __builtin_fmaf(p, v, 1.0f);
    return p * v;
}

__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.0f + exp2_fast(-kLog2e * v)); }

// A gate for the backward, which needs sigmoid(v) and its slope sigmoid(v) sigmoid(-v), each to its
// last digits: `half` is sigmoid(v) where that is the smaller of the two factors, else -sigmoid(-v)
// (2^-126 more, so that it is never 0), from which the fraction makes the larger one again.
struct Sides { float open, half; };
__device__ __forceinline__ Sides gate_sides(float v) {
    const float E = exp2_fast(-kLog2e * v), open = rcp_fast(1.0f + E), shut = __builtin_fmaf(E, open, 0x1p-126f);
    return Sides{open, v > 0.0f ? -shut : open};
}
__device__ __forceinline__ float gate_open(float half) { return __builtin_amdgcn_fractf(half); }     // half, or 1 + half under 0
__device__ __forceinline__ float gate_slope(float half) {
    return __builtin_fabsf(half) * (1.0f - __builtin_fabsf(half));
}

// The decay near 1 is what a long memory is made of: a = 1 + expm1(A s) has the rounding of the
// sum alone there, and 1 - a^2 = -e (1 + a) with e = expm1(A s) keeps its relative accuracy
// where 1 - a * a would cancel. Further out a is the exponential itself: a sum with 1 would leave a
// small decay, which the gradients have as a factor, whole steps of 2^-24. `bias` is added to A s:
// 0, or minus infinity for a reset, which gives a = 0 and 1 - a^2 = 1.
struct Decay { float a, w2; };            // exp(A s), 1 - a^2
// A of a channel without memory, minus infinity, as the lowest number: times the 0 that stands for
// a shut gate (a token past the end is one) it leaves the state as it is.
__device__ __forceinline__ float glr_rate(float A) { return A < -0x1.fffffep127f ? -0x1.fffffep127f : A; }
__device__ __forceinline__ Decay glr_decay(float s, float A, float bias) {
    const float la = __builtin_fmaf(A, s, bias);
    const float far = exp2_fast(kLog2e * la), near = expm1_small(la);
    const bool small = __builtin_fabsf(la) < kEm1Small;
    const float e = small ? near : far - 1.0f, a = small ? 1.0f + near : far;
    return Decay{a, -__builtin_fmaf(e, a, e)};
}

struct Gate { float g, a, w2; };          // sigmoid(i), and the decay
__device__ __forceinline__ Gate glr_gate(float r, float i, float A, float bias) {
    const Decay d = glr_decay(sigmoid(r), A, bias);
    return Gate{sigmoid(i), d.a, d.w2};
}

// ---------------------------------------------------------------------------
// two channels of one row: loads, stores, conversions

// Rows are addressed by a base that is uniform over the wave and 32-bit byte offsets of the
// lane's channels (D is at most 2^26), which the memory instructions add themselves.
template <typename T> __device__ __forceinline__ const T& at_byte(const void* row, unsigned off) {
    return *reinterpret_cast<const T*>(static_cast<const char*>(row) + off);
}
template <typename T> __device__ __forceinline__ T& at_byte(void* row, unsigned off) {
    return *reinterpret_cast<T*>(static_cast<char*>(row) + off);
}
// renew(): the compiler may not carry over what it has computed from the values before (converted
// copies of a whole run, kept from one pass over it to the next, would take the registers of
// another workgroup).
template <typename T, bool VEC> struct Pair;
template <> struct Pair<float, true> {
    typedef float v2 __attribute__((ext_vector_type(2)));
    v2 v;
    __device__ __forceinline__ void ld(const void* row, unsigned c0, unsigned) { v = at_byte<v2>(row, 4 * c0); }
    __device__ __forceinline__ float get(int j) const { return v[j]; }
    __device__ __forceinline__ void set(float f) { v = v2{f, f}; }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(v)); }
    static __device__ __forceinline__ void st(void* row, unsigned c0, unsigned, bool ok0, bool, float a, float b) {
        if (ok0) at_byte<v2>(row, 4 * c0) = v2{a, b};
    }
};
template <> struct Pair<uint16_t, true> {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    uint32_t v;
    __device__ __forceinline__ void ld(const void* row, unsigned c0, unsigned) { v = at_byte<uint32_t>(row, 2 * c0); }
    __device__ __forceinline__ float get(int j) const {
        return __builtin_bit_cast(float, j ? (v & 0xffff0000u) : (v << 16));
    }
    __device__ __forceinline__ void set(float f) { v = (uint32_t)IO<uint16_t>::bits(f) * 0x10001u; }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(v)); }
    static __device__ __forceinline__ void st(void* row, unsigned c0, unsigned, bool ok0, bool, float a, float b) {
        if (ok0) at_byte<b2>(row, 2 * c0) = __builtin_convertvector((f2{a, b}), b2);
    }
};
template <> struct Pair<float, false> {
    float v[2];
    __device__ __forceinline__ void ld(const void* row, unsigned c0, unsigned c1) {
        v[0] = at_byte<float>(row, 4 * c0);
        v[1] = at_byte<float>(row, 4 * c1);
    }
    __device__ __forceinline__ float get(int j) const { return v[j]; }
    __device__ __forceinline__ void set(float f) { v[0] = v[1] = f; }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(v[0]), "+v"(v[1])); }
    static __device__ __forceinline__ void st(void* row, unsigned c0, unsigned c1, bool ok0, bool ok1, float a, float b) {
        if (ok0) at_byte<float>(row, 4 * c0) = a;
        if (ok1) at_byte<float>(row, 4 * c1) = b;
    }
};
template <> struct Pair<uint16_t, false> {
    typedef uint16_t u2 __attribute__((ext_vector_type(2)));      // one register: the loads fill its halves
    u2 v;
    __device__ __forceinline__ void ld(const void* row, unsigned c0, unsigned c1) {
        v = u2{at_byte<uint16_t>(row, 2 * c0), at_byte<uint16_t>(row, 2 * c1)};
    }
    __device__ __forceinline__ float get(int j) const {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        return __builtin_bit_cast(float, j ? (u & 0xffff0000u) : (u << 16));
    }
    __device__ __forceinline__ void set(float f) { v = u2{IO<uint16_t>::bits(f), IO<uint16_t>::bits(f)}; }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(v)); }
    static __device__ __forceinline__ void st(void* row, unsigned c0, unsigned c1, bool ok0, bool ok1, float a, float b) {
        if (ok0) at_byte<uint16_t>(row, 2 * c0) = IO<uint16_t>::bits(a);
        if (ok1) at_byte<uint16_t>(row, 2 * c1) = IO<uint16_t>::bits(b);
    }
};

// The two channels of a lane: next to each other where rows allow one access for both,
// else 64 apart, so that a wave's accesses stay contiguous. Lanes past the last channel
// repeat it (their loads stay in range) and store nothing.
struct Chan { unsigned c[2]; bool ok[2]; };
template <bool VEC>
__device__ __forceinline__ Chan lane_chan(int col, int lane, int D) {
    Chan q;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = col * kGlrCols + (VEC ? 2 * lane + j : lane + 64 * j);
        q.ok[j] = c < D;
        q.c[j] = (unsigned)(q.ok[j] ? c : (VEC ? D - 2 + j : D - 1));
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

// The state in front of a chunk, for the CH channels of a wave (of whom the first `valid` exist).
// `row` holds the words of the chunk just in front, the n rows of the chunks in front lie
// `stride` apart towards it, and the first of them always ends up as states. The wave's 64 lanes
// read 64 / CH rows at once (lane l channel l % CH, row l / CH, nearest first), go on to the
// rows in front of these until every channel has met a state with no empty word nearer by, and
// start over where one is empty. Then they fold forward over the rows read: a word that is a
// state replaces what was folded so far, so that what lies in front of a channel's nearest
// state, or has become a state since, does not matter. Every lane of a channel gets its state.
template <int CH>
__device__ __forceinline__ float look_back(const uint64_t* row, int64_t stride, int n, int valid, int lane) {
    constexpr int kRows = 64 / CH;
    constexpr uint32_t kAll = (uint32_t)((uint64_t(1) << CH) - 1u);
    const uint32_t want = valid >= CH ? kAll : (1u << valid) - 1u;
    const int ch = lane % CH < valid ? lane % CH : valid - 1, at = lane / CH;
    auto load = [&](int first) { return word_load(row + (int64_t)(first + at < n ? first + at : n - 1) * stride + ch); };
    uint64_t v;
    int first = 0;                                 // rows between `row` and those read
    uint32_t done = 0;                             // channels that have met a state
    while (true) {
        v = load(first);
        const uint64_t st = __ballot(word_tag(v) == kStateTag), em = __ballot(v == kEmpty);
        uint32_t open = want & ~done;              // channels that have met neither a state nor an empty word
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const uint32_t s = (uint32_t)(st >> (i * CH)) & kAll, e = (uint32_t)(em >> (i * CH)) & kAll;
            done |= open & s;
            open &= ~(s | e);
        }
        if (done == want) break;
        if (want & ~done & ~open) {
            first = 0;                             // words nearer by may have become states meanwhile
            done = 0;
            __builtin_amdgcn_s_sleep(1);
        } else {
            first += kRows;
        }
    }
    float h = 0.0f;
    while (true) {
#pragma unroll
        for (int i = kRows - 1; i >= 0; --i) {
            const float t = word_tag(v) == kStateTag ? word_lo(v) : fold(__builtin_bit_cast(float, word_tag(v)), h, word_lo(v));
            h = __shfl(t, i * CH + lane % CH, 64);
        }
        if (first == 0) return h;
        first -= kRows;
        v = load(first);
    }
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

// A lane per token: whether token t0 + lane of batch row b resets. The ballot over it has bit k
// set where token t0 + k does.
template <int TT>
__device__ __forceinline__ bool reset_at(const GlrArgs& p, int b, int64_t t0, int lane) {
    const int64_t t = t0 + lane;
    return p.reset && lane < TT && t < p.L && p.reset[(int64_t)b * p.L + t] != 0;
}

// Tokens of the run that starts at t0: TT of them, fewer at the end, 0 past it.
__device__ __forceinline__ int run_tokens(const GlrArgs& p, int64_t t0, int TT) {
    const int64_t left = p.L - t0;
    return left < TT ? (left > 0 ? (int)left : 0) : TT;
}

// A run's rows: a base and a step that is uniform over the wave, past the last token a step of
// zero, so that every address is one of the sequence's.
template <typename T>
struct Rows {
    const char* at;
    int64_t step;
    __device__ __forceinline__ Rows(const void* p, int64_t sb, int64_t st, int b, int64_t t)
        : at(static_cast<const char*>(p) + (b * sb + t * st) * (int64_t)sizeof(T)), step(st * (int64_t)sizeof(T)) {}
    __device__ __forceinline__ void next(bool more) { at += more ? step : 0; }
};

// ---------------------------------------------------------------------------
// forward

// A wave's run of TT tokens: its rows, then the two factors of y_k = h[k] + P[k] * (state in front).
template <typename T, bool VEC, int TT>
struct FwdRun {
    using V = Pair<T, VEC>;
    V vx[TT], vr[TT], vi[TT];
    float A[2];
    bool reset;
    float P[TT][2], h[TT][2];

    // all rows at once; a run past the end loads the last one
    __device__ __forceinline__ void fetch(const GlrArgs& p, const Tile& q, const Chan& c, int64_t t0, int lane) {
        const int64_t tb = t0 < p.L ? t0 : p.L - 1;
        const int n = run_tokens(p, t0, TT);
        Rows<T> rx(p.x, p.xb, p.xt, q.b, tb), rr(p.r, p.rb, p.rt, q.b, tb), ri(p.i, p.ib, p.it, q.b, tb);
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            vx[k].ld(rx.at, c.c[0], c.c[1]);
            vr[k].ld(rr.at, c.c[0], c.c[1]);
            vi[k].ld(ri.at, c.c[0], c.c[1]);
            const bool more = k + 1 < n;
            rx.next(more); rr.next(more); ri.next(more);
        }
        A[0] = glr_rate(p.A[c.c[0]]);
        A[1] = glr_rate(p.A[c.c[1]]);
        reset = reset_at<TT>(p, q.b, t0, lane);
    }

    // the run from a zero state: h[k] the local state, P[k] what a state in front is multiplied by
    __device__ __forceinline__ void reduce(int n, uint32_t rs) {
        // tokens past the end leave the state as it is: a = exp(A sigmoid(-inf)) = 1, w = 0; a reset
        // token's r is not looked at
        if (n < TT) {
#pragma unroll
            for (int k = 0; k < TT; ++k)
                if (k >= n) { vx[k].set(0.0f); vr[k].set(-__builtin_inff()); vi[k].set(0.0f); }
        }
        if (rs) {
#pragma unroll
            for (int k = 0; k < TT; ++k)
                if (rs >> k & 1u) vr[k].set(0.0f);
        }
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            const bool on = rs >> k & 1u;
            const float bias = on ? -__builtin_inff() : 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const Gate g = glr_gate(vr[k].get(j), vi[k].get(j), A[j], bias);
                P[k][j] = k ? g.a * P[k - 1][j] : g.a;
                h[k][j] = __builtin_amdgcn_sqrtf(g.w2) * (g.g * vx[k].get(j));
                if (k) h[k][j] = __builtin_fmaf(g.a, on ? 0.0f : h[k - 1][j], h[k][j]);
            }
            __builtin_amdgcn_sched_barrier(0);                    // token by token: other waves fill the pipes, and registers are few
        }
    }
    __device__ __forceinline__ float2 map(uint32_t rs, int j) const { return make_float2(rs ? -0.0f : P[TT - 1][j], h[TT - 1][j]); }

    __device__ __forceinline__ void put(const GlrArgs& p, const Tile& q, const Chan& c, int64_t t0, uint32_t rs, const float* in) const {
        const int n = run_tokens(p, t0, TT);
        // The state in front of token 64 m of a batch row is checkpoint m: the one behind token k_ck
        // of this run, if it is one of its tokens and not the sequence's last. The state behind the
        // last token, k_end, is the final one.
        const int k_ck = p.ckpt && n > 0 ? SS_GLR_CKPT - 1 - (int)(t0 % SS_GLR_CKPT) : -1;
        const int k_end = n > 0 && t0 + n == p.L ? n - 1 : -1;
        auto put_ckpt = [&](int64_t t, float a, float b) {
            Pair<float, VEC>::st(p.ckpt + ((int64_t)q.b * p.nck + t / SS_GLR_CKPT) * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], a, b);
        };
        if (p.ckpt && t0 == 0) put_ckpt(0, in[0], in[1]);
        char* yrow = static_cast<char*>(p.y) + ((int64_t)q.b * p.L + t0) * p.D * (int64_t)sizeof(T);
        const int64_t ystep = (int64_t)p.D * (int64_t)sizeof(T);
        auto go = [&](auto plain) {
            constexpr bool kPlain = decltype(plain)::value;       // whole run, no reset
            const int k_rs = rs ? __builtin_ctz(rs) : TT;         // from the first reset on the state in front does not count
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                if (kPlain || k < n) {
                    float o[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        o[j] = kPlain || k < k_rs ? __builtin_fmaf(P[k][j], in[j], h[k][j]) : h[k][j];
                    V::st(yrow, c.c[0], c.c[1], c.ok[0], c.ok[1], o[0], o[1]);
                    yrow += ystep;
                    if (k == k_ck && k != k_end) put_ckpt(t0 + k + 1, o[0], o[1]);
                    if (k == k_end && p.state)
                        Pair<float, VEC>::st(p.state + (int64_t)q.b * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], o[0], o[1]);
                }
            }
        };
        if (n == TT && rs == 0) go(Tag<true>{});
        else go(Tag<false>{});
    }
};

// One chunk per batch row: a workgroup per tile. Latency: a load, a run's gates, the join in LDS
// and the stores (B 1, L 64, D 512, fp32: 5.4 us); with many rows bound by memory (B 256, L 128,
// D 2048, fp32: 204 us, 5.2 TB/s).
template <typename T, bool VEC, int TT, int NW>
__global__ void __launch_bounds__(NW * 64, 4)
k_glr_fwd(const GlrArgs p) {
    static_assert(NW % 4 == 0, "the runs' maps are read four at a time");
    __shared__ float2 s_map[NW][kGlrCols];        // (P, S) of each wave's run
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile q = tile_at(p, blockIdx.x);
    const Chan c = lane_chan<VEC>(q.col, lane, p.D);
    const int64_t t0 = wave * TT;
    FwdRun<T, VEC, TT> run;
    run.fetch(p, q, c, t0, lane);
    float in[2] = {0.0f, 0.0f};
    if (p.state) {
#pragma unroll
        for (int j = 0; j < 2; ++j) in[j] = p.state[(int64_t)q.b * p.D + c.c[j]];
    }
    const uint32_t rs = (uint32_t)__ballot(run.reset);
    run.reduce(run_tokens(p, t0, TT), rs);
#pragma unroll
    for (int j = 0; j < 2; ++j) s_map[wave][lane_slot<VEC>(lane, j)] = run.map(rs, j);
    asm volatile("" : "+v"(in[0]), "+v"(in[1]));  // every wave has the initial state, which one overwrites
    __syncthreads();
    for (int w = 0; w < wave; w += 4) {
        float2 m[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) m[i][j] = s_map[w + i][lane_slot<VEC>(lane, j)];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (w + i < wave) in[j] = fold(m[i][j].x, in[j], m[i][j].y);
    }
    run.put(p, q, c, t0, rs, in);
}

// Several chunks per batch row, tiles taken by ticket. Loading the next tile's rows before the
// wait for the state in front was slower: the look-back's loads return behind them, and every
// chunk after this one waits for it. So was a wave of its own for the look-back with the next
// rows in flight meanwhile (B 1, L 131072, D 2048: 700 us against 620): a word's way between two
// workgroups is through memory, and takes longer the fuller the memory's queues are.
template <typename T, bool VEC, int TT, int NW>
__global__ void __launch_bounds__(NW * 64, 4)
k_glr_scan(const GlrArgs p) {
    __shared__ float2 s_map[NW][kGlrCols];        // (P, S) of each wave's run
    __shared__ float s_in[NW][kGlrCols];          // state in front of each wave's run
    __shared__ unsigned s_next;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid == 0) s_next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    unsigned tile = __builtin_amdgcn_readfirstlane(s_next);
    __syncthreads();
    while (tile < p.tiles) {
        const Tile q = tile_at(p, tile);
        const Chan c = lane_chan<VEC>(q.col, lane, p.D);
        const int64_t t0 = (int64_t)q.chunk * (NW * TT) + wave * TT;
        FwdRun<T, VEC, TT> run;
        run.fetch(p, q, c, t0, lane);
        unsigned next = 0;
        if (tid == 0) next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t rs = (uint32_t)__ballot(run.reset);
        run.reduce(run_tokens(p, t0, TT), rs);
#pragma unroll
        for (int j = 0; j < 2; ++j) s_map[wave][lane_slot<VEC>(lane, j)] = run.map(rs, j);
        if (tid == 0) s_next = next;
        __syncthreads();
        tile = __builtin_amdgcn_readfirstlane(s_next);

        // the states in front of the runs: each wave for 128 / NW channels
        {
            constexpr int CH = kGlrCols / NW;
            const int ch = wave * CH + lane % CH;
            const int valid = p.D - q.col * kGlrCols - wave * CH;    // channels that exist from this wave's first on
            if (valid > 0) {
                const int64_t bd0 = (int64_t)q.b * p.D + q.col * kGlrCols + wave * CH, BD = (int64_t)p.B * p.D;
                const bool mine = lane < CH && lane < valid;         // the lane that writes for its channel
                float in = 0.0f;
                if (q.chunk > 0) {
                    float cp = 1.0f, cs = 0.0f;
#pragma unroll 4
                    for (int w = 0; w < NW; ++w) {
                        const float2 m = s_map[w][ch];
                        cs = fold(m.x, cs, m.y);
                        cp = fold_p(m.x, cp);
                    }
                    uint64_t* row = p.slots + (int64_t)q.chunk * BD + bd0;
                    const bool pass = mine && q.chunk + 1 < p.nchunks;
                    if (pass) word_store(row + lane, map_word(cp, cs));
                    in = look_back<CH>(row - BD, -BD, q.chunk, valid, lane);
                    if (pass) word_store(row + lane, state_word(fold(cp, in, cs)));
                } else if (mine && p.state) {
                    in = p.state[bd0 + lane];
                }
                if (mine) {
                    float hh = in;
#pragma unroll 4
                    for (int w = 0; w < NW; ++w) {
                        const float2 m = s_map[w][ch];
                        s_in[w][ch] = hh;
                        hh = fold(m.x, hh, m.y);
                    }
                    if (q.chunk == 0) word_store(p.slots + bd0 + lane, state_word(hh));
                }
            }
        }
        __syncthreads();
        float in[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) in[j] = s_in[wave][lane_slot<VEC>(lane, j)];
        run.put(p, q, c, t0, rs, in);
    }
}

// ---------------------------------------------------------------------------
// backward: the same tiles, taken from the last chunk to the first. The states in front of the
// runs come from the forward's checkpoints and the runs' maps; what passes from a token to the
// one before it is K_t = a_t g_t, and over a run K -> P K + S with the forward's P and
// S = sum_k P_k dy_k, P_k the product of the decays up to token k. The first pass over a run
// keeps half of each gate and, of the state in front of each token, its part from within the run and
// the factor of what comes from outside; the second, backward in time, has the true states and
// takes the decay and write coefficient from the gates again (half of a gate's cost, for
// four registers a token). Sums of dA over a run stay in registers, over a chunk in LDS;
// k_glr_da adds the chunks. B 8, L 2048, D 5120, bf16: 317 us, 3.7 TB/s over the seven tensors; two
// waves a SIMD (225 registers), whose arithmetic (70 percent of the vector units' time) overlaps with
// the loads of one other workgroup.

template <typename T, bool VEC, int TT, int NW, bool LOOK>
__global__ void __launch_bounds__(NW * 64, NW > 8 ? 4 : 2)
k_glr_bwd(const GlrArgs p) {
    constexpr int CK = NW * TT / SS_GLR_CKPT;                     // checkpoints of a chunk
    static_assert(SS_GLR_CKPT % TT == 0 && CK * SS_GLR_CKPT == NW * TT, "checkpoints lie at starts of runs");
    using V = Pair<T, VEC>;
    __shared__ float s_p[NW][kGlrCols], s_f[NW][kGlrCols], s_b[NW][kGlrCols];   // P and both S of each run
    __shared__ float s_h[NW][kGlrCols], s_k[NW][kGlrCols];                      // state in front, K from behind
    __shared__ float s_a[NW][kGlrCols];                                         // parts of dA
    __shared__ unsigned s_next;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int CH = kGlrCols / NW;                             // channels that a wave joins runs for

    unsigned tile = blockIdx.x;
    if constexpr (LOOK) {
        if (tid == 0) s_next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        tile = __builtin_amdgcn_readfirstlane(s_next);
        __syncthreads();
    }
    while (tile < p.tiles) {
        unsigned next = p.tiles;
        if constexpr (LOOK) {
            if (tid == 0) next = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        Tile q = tile_at(p, tile);
        q.chunk = p.nchunks - 1 - q.chunk;
        const Chan c = lane_chan<VEC>(q.col, lane, p.D);
        const int64_t t0 = (int64_t)q.chunk * (NW * TT) + wave * TT;
        const int n = run_tokens(p, t0, TT);
        const int64_t bd0 = (int64_t)q.b * p.D + q.col * kGlrCols + wave * CH, BD = (int64_t)p.B * p.D;
        const int valid = p.D - q.col * kGlrCols - wave * CH;     // channels that exist from this wave's first on
        const bool mine = lane < CH && lane < valid;              // the lane that writes for its channel

        V vx[TT], vd[TT];
        float s[TT][2], g[TT][2], A[2];                           // the halves of both gates
        float P[TT][2], h[TT][2];                                 // in front of token k: state h + P times the run's
        float ck[CK];
        uint32_t rs;
        int k_rs;
        {
            V vr[TT], vi[TT];
            const int64_t tb = t0 < p.L ? t0 : p.L - 1;
            Rows<T> rx(p.x, p.xb, p.xt, q.b, tb), rr(p.r, p.rb, p.rt, q.b, tb), ri(p.i, p.ib, p.it, q.b, tb),
                rd(p.dy, p.L * p.D, p.D, q.b, tb);
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                vx[k].ld(rx.at, c.c[0], c.c[1]);
                vr[k].ld(rr.at, c.c[0], c.c[1]);
                vi[k].ld(ri.at, c.c[0], c.c[1]);
                vd[k].ld(rd.at, c.c[0], c.c[1]);
                const bool more = k + 1 < n;
                rx.next(more); rr.next(more); ri.next(more); rd.next(more);
            }
            A[0] = glr_rate(p.A[c.c[0]]);
            A[1] = glr_rate(p.A[c.c[1]]);
#pragma unroll
            for (int m = 0; m < CK; ++m) {
                const int64_t ci = (int64_t)q.chunk * CK + m;
                ck[m] = mine && ci < p.nck ? p.ckpt[((int64_t)q.b * p.nck + ci) * p.D + q.col * kGlrCols + wave * CH + lane] : 0.0f;
            }
            rs = (uint32_t)__ballot(reset_at<TT>(p, q.b, t0, lane));
            k_rs = rs ? __builtin_ctz(rs) : TT;
            if (n < TT) {                                         // past the end: a = 1, w = 0, no gradient
#pragma unroll
                for (int k = 0; k < TT; ++k)
                    if (k >= n) { vx[k].set(0.0f); vr[k].set(-__builtin_inff()); vi[k].set(0.0f); vd[k].set(0.0f); }
            }
            if (rs) {
#pragma unroll
                for (int k = 0; k < TT; ++k)
                    if (rs >> k & 1u) vr[k].set(0.0f);
            }
            float Pk[2] = {1.0f, 1.0f}, Sf[2] = {0.0f, 0.0f}, Sb[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                const bool on = rs >> k & 1u;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const Sides sr = gate_sides(vr[k].get(j)), si = gate_sides(vi[k].get(j));
                    s[k][j] = sr.half;
                    g[k][j] = si.half;
                    asm volatile("" : "+v"(s[k][j]), "+v"(g[k][j]));  // now, and not what they are made of kept instead
                    const Decay e = glr_decay(sr.open, A[j], on ? -__builtin_inff() : 0.0f);
                    P[k][j] = Pk[j];
                    h[k][j] = Sf[j];
                    Pk[j] *= e.a;
                    Sf[j] = __builtin_fmaf(e.a, on ? 0.0f : Sf[j],
                                            __builtin_amdgcn_sqrtf(e.w2) * (si.open * vx[k].get(j)));
                    Sb[j] = k < k_rs ? __builtin_fmaf(Pk[j], vd[k].get(j), Sb[j]) : Sb[j];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = lane_slot<VEC>(lane, j);
                s_p[wave][at] = rs ? -0.0f : Pk[j];
                s_f[wave][at] = Sf[j];
                s_b[wave][at] = Sb[j];
            }
        }
        if (LOOK && tid == 0) s_next = next;
        __syncthreads();
        if constexpr (LOOK) next = __builtin_amdgcn_readfirstlane(s_next);

        if (valid > 0) {
            const int ch = wave * CH + lane % CH;
            float in = 0.0f;
            if (LOOK && q.chunk + 1 < p.nchunks) {
                float cp = 1.0f, cs = 0.0f;
#pragma unroll 4
                for (int v = NW - 1; v >= 0; --v) {
                    cs = fold(s_p[v][ch], cs, s_b[v][ch]);
                    cp = fold_p(s_p[v][ch], cp);
                }
                uint64_t* row = p.slots + (int64_t)q.chunk * BD + bd0;
                const bool pass = mine && q.chunk > 0;
                if (pass) word_store(row + lane, map_word(cp, cs));
                in = look_back<CH>(row + BD, BD, p.nchunks - 1 - q.chunk, valid, lane);
                if (pass) word_store(row + lane, state_word(fold(cp, in, cs)));
            } else if (mine && p.dstate_final) {
                in = p.dstate_final[bd0 + lane];
            }
            if (mine) {
#pragma unroll 4
                for (int v = NW - 1; v >= 0; --v) {
                    s_k[v][ch] = in;
                    in = fold(s_p[v][ch], in, s_b[v][ch]);
                }
                if (LOOK && q.chunk + 1 == p.nchunks) word_store(p.slots + (int64_t)q.chunk * BD + bd0 + lane, state_word(in));
#pragma unroll
                for (int m = 0; m < CK; ++m) {
                    float hh = ck[m];
#pragma unroll 4
                    for (int v = m * (NW / CK); v < (m + 1) * (NW / CK); ++v) {
                        s_h[v][ch] = hh;
                        hh = fold(s_p[v][ch], hh, s_f[v][ch]);
                    }
                }
            }
        }
        __syncthreads();

        float K[2], dA[2] = {0.0f, 0.0f}, in[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            in[j] = s_h[wave][lane_slot<VEC>(lane, j)];
            K[j] = s_k[wave][lane_slot<VEC>(lane, j)];
        }
        const int64_t o1 = (((int64_t)q.b * p.L + t0 + n) * p.D) * (int64_t)sizeof(T), step = (int64_t)p.D * (int64_t)sizeof(T);
        char* px = static_cast<char*>(p.dx) + o1;                 // behind the run's last row
        char* pr = static_cast<char*>(p.dr) + o1;
        char* pi = static_cast<char*>(p.di) + o1;
#pragma unroll
        for (int k = TT - 1; k >= 0; --k) {
            const bool on = rs >> k & 1u;
            float dx[2], dr[2], di[2];
            vx[k].renew();
            vd[k].renew();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                asm volatile("" : "+v"(s[k][j]), "+v"(g[k][j]));      // see renew()
                const float sr = gate_open(s[k][j]), gi = gate_open(g[k][j]);
                const Decay e = glr_decay(sr, A[j], on ? -__builtin_inff() : 0.0f);
                // 1 / w, and w from it; both 0 where w^2 is 0 or below the smallest normal number (whose
                // root the instruction takes as that of 0): the slope there is taken as 0
                const float rw = e.w2 >= 0x1p-126f ? __builtin_amdgcn_rsqf(e.w2) : 0.0f, w = e.w2 * rw;
                const float before = k <= k_rs ? __builtin_fmaf(P[k][j], in[j], h[k][j]) : h[k][j];
                const float x = vx[k].get(j), G = vd[k].get(j) + K[j];
                const float gw = G * w, v = gi * x;
                dx[j] = gw * gi;
                di[j] = gw * (x * gate_slope(g[k][j]));
                K[j] = on ? 0.0f : e.a * G;
                const float dla = on ? 0.0f : K[j] * (before - e.a * rw * v);
                dr[j] = dla * (A[j] * gate_slope(s[k][j]));
                dA[j] = __builtin_fmaf(dla, sr, dA[j]);
            }
            if (k < n) {
                px -= step; pr -= step; pi -= step;
                V::st(px, c.c[0], c.c[1], c.ok[0], c.ok[1], dx[0], dx[1]);
                V::st(pr, c.c[0], c.c[1], c.ok[0], c.ok[1], dr[0], dr[1]);
                V::st(pi, c.c[0], c.c[1], c.ok[0], c.ok[1], di[0], di[1]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (p.dstate_init && t0 == 0)
            Pair<float, VEC>::st(p.dstate_init + (int64_t)q.b * p.D, c.c[0], c.c[1], c.ok[0], c.ok[1], K[0], K[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) s_a[wave][lane_slot<VEC>(lane, j)] = dA[j];
        __syncthreads();
        if (mine) {
            float t = s_a[0][wave * CH + lane];
#pragma unroll
            for (int v = 1; v < NW; ++v) t += s_a[v][wave * CH + lane];
            p.part[(int64_t)q.chunk * BD + bd0 + lane] = t;
        }
        if constexpr (!LOOK) break;
        tile = next;
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
// one token per stream: a lane per two channels; memory and a launch's latency (S 64, D 8192, bf16:
// 3.5 us for 8.4 MB)

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
    A.ld(p.A, c.c[0], c.c[1]);
    const bool rs = p.reset && p.reset[b] != 0;
    float o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const Gate g = glr_gate(r.get(j), i.get(j), glr_rate(A.get(j)), 0.0f);
        const float v = g.g * x.get(j);                               // what a reset leaves
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
        const int64_t groups = (n + 255) / 256;
        hipLaunchKernelGGL(k_glr_clear, dim3((unsigned)(groups < 2048 ? groups : 2048)), dim3(256), 0, st, p.slots, n, p.ticket);
    }
    const dim3 grid(look && a.tiles > kGlrGroups ? kGlrGroups : a.tiles);
    auto go = [&](auto kernel, int64_t waves) { hipLaunchKernelGGL(kernel, grid, dim3((unsigned)waves * 64), 0, st, a); };
    if (p.pass == LaunchGlr::kFwd) {
        // One chunk is a matter of latency: 16 waves with runs of 8 tokens, of 4 up to 64 tokens (B 1, L 64,
        // D 512, fp32: 5.5 us against 8.2 with runs of 8). Several: runs of 16 tokens where a row's two
        // channels fit one register (B 8, L 2048, D 5120, bf16: 164 us against 196 with 16 waves of 8
        // tokens), else runs of 8 (fp32, B 8, L 2048, D 2560: 144 against 153)
        if (!look) {
            if (p.L <= 64) go(k_glr_fwd<T, VEC, 4, 16>, 16);
            else go(k_glr_fwd<T, VEC, 8, 16>, 16);
        } else if (p.chunk == 64) {
            go(k_glr_scan<T, VEC, 8, 8>, 8);
        } else if constexpr (sizeof(T) == 2) {
            if (p.chunk == 256) go(k_glr_scan<T, VEC, 16, 16>, 16);
            else go(k_glr_scan<T, VEC, 16, 8>, 8);
        } else {
            go(k_glr_scan<T, VEC, 8, 16>, 16);
        }
    } else {
        // runs of 16 tokens, with few tiles of 8; one chunk (64 tokens then) in runs of 4 (B 1, L 64,
        // D 512: 10.7 us against 13.1 with 16; B 256, L 64, D 4096, bf16: 266 both)
        if (!look) {
            go(k_glr_bwd<T, VEC, 4, 16, false>, 16);
        } else if (glr_fine(true, p.batch, p.L, p.D)) {
            go(k_glr_bwd<T, VEC, 8, 8, true>, 8);
        } else if (p.chunk == 64) {
            go(k_glr_bwd<T, VEC, 16, 4, true>, 4);
        } else {
            go(k_glr_bwd<T, VEC, 16, 8, true>, 8);
        }
        hipLaunchKernelGGL(k_glr_da, dim3((unsigned)((p.D + 63) / 64)), dim3(1024), 0, st, p.part, p.g.dA,
                           p.nchunks * p.batch, (int)p.D);
    }
    return hipGetLastError();
}

}  // namespace selscan
