// Device code of the 8-bit product (ss_gemm_q8): Y[M, N] = X W^T (+ R) with
// X[m, k] = xs[m, k / 128] xq[m, k] and W[n, k] = ws[n / 128, k / 128] wq[n, k], the q e4m3.
//
// The scales are constant over blocks of 128 along k: the matrix cores sum a block's 128
// products from zero, and the vector units add the result to the running fp32 sum with its
// scale, acc += (xs ws) p. W rows are the first operand, so that a lane of a 16 x 16 result
// holds one row m of X (l % 16) and four consecutive rows n of W (4 (l / 16) + v): its block
// scale is one number.
//
// Precision of a block's sum. The 8-bit matrix instructions add the products of eight neighbouring k
// on a common exponent and drop what lies below 2^-13 of the largest (measured: a second product
// survives at 2^-13 and is lost at 2^-14 within eight k, at 2^-23 and 2^-24 further apart): two
// large products that cancel take a small one with them. So both operands are converted to bf16,
// which holds every e4m3 value, for the bf16 instruction, whose products and sums keep fp32 (1e-8
// off), at half the rate: bf16 out, M 16384, N 10240, K 2560 860 us against 470, M 64 with W from memory
// 11.7 against 11.2.
//
// Both operands are k-contiguous and a sum over k has no order of its own here, so a lane's
// 32 bytes of an operand may be any two 16-byte chunks of the block as long as both operands
// take the same two: lane l takes chunks l / 16 and l / 16 + 4 of its row.
#pragma once
#include <type_traits>

#include "ops_internal.h"
#include "selscan_device.h"

namespace selscan {

typedef int gq_i4 __attribute__((ext_vector_type(4)));
typedef float gq_f4 __attribute__((ext_vector_type(4)));
typedef __bf16 gq_b8 __attribute__((ext_vector_type(8)));
typedef __bf16 gq_b2 __attribute__((ext_vector_type(2)));

// A lane's 32 bytes of one operand as four operands of the bf16 instruction.
struct GqFrag {
    gq_b8 v[4];
    __device__ __forceinline__ void set(gq_i4 a, gq_i4 b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int w = j < 4 ? a[j] : b[j - 4];
            const gq_b2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
            const gq_b2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
            v[j / 2][4 * (j % 2)] = lo[0]; v[j / 2][4 * (j % 2) + 1] = lo[1];
            v[j / 2][4 * (j % 2) + 2] = hi[0]; v[j / 2][4 * (j % 2) + 3] = hi[1];
        }
    }
};
// A block's products of one row fragment with N column fragments, the N sums taking turns.
template <int N>
__device__ __forceinline__ void gq_dot(const GqFrag& a, const GqFrag (&x)[N], gq_f4 (&q)[N]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int b = 0; b < N; ++b)
            q[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[j], x[b].v[j], j ? q[b] : gq_f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
}

// 64 lanes' 16-byte chunks from a matrix straight into 1024 consecutive bytes of LDS: byte
// offset voff (per lane) + soff from the base, which may lie anywhere in memory.
struct GqSource {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit GqSource(const uint8_t* p)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, -1, kBufDword3)) {}
    __device__ __forceinline__ void to_lds(gq_i4* lds, unsigned voff, unsigned soff) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, voff, soff, 0, 0);
    }
    __device__ __forceinline__ void to_lds4(gq_i4* lds, unsigned voff, unsigned soff) const {      // four bytes a lane
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 4, voff, soff, 0, 0);
    }
};

struct GemmQ8Args {
    const uint8_t* xq; const float* xs; const uint8_t* wq; const float* ws;
    const void* R; void* Y0; void* Y1;
    int64_t split, M, N, K;
    int KB;                       // blocks along k
};

// W consecutive columns n .. n + W - 1 of row m, n a multiple of W.
template <typename T, bool RES, int W>
__device__ __forceinline__ void gq_store(const GemmQ8Args& p, int64_t m, int64_t n, const float* v) {
    if (m >= p.M || n >= p.N) return;
    const bool one = n >= p.split;
    const int64_t ld = one ? p.N - p.split : p.split, c = one ? n - p.split : n;
    if (c + W <= ld) {                                           // in one matrix: whole accesses, wherever the row starts
        constexpr int A = 16 / sizeof(T) < W ? 16 / sizeof(T) : W;    // elements of one access
        typedef T ta __attribute__((ext_vector_type(A), aligned(sizeof(T))));
        T* y = static_cast<T*>(one ? p.Y1 : p.Y0) + m * ld + c;
        const T* r = RES ? static_cast<const T*>(p.R) + m * ld + c : nullptr;
#pragma unroll
        for (int h = 0; h < W; h += A) {
            ta o, rv;
            if (RES) rv = *reinterpret_cast<const ta*>(r + h);
#pragma unroll
            for (int j = 0; j < A; ++j) o[j] = IO<T>::bits(RES ? v[h + j] + IO<T>::cvt(rv[j]) : v[h + j]);
            *reinterpret_cast<ta*>(y + h) = o;
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (n + j >= p.N) break;
            const bool o2 = n + j >= p.split;
            const int64_t l2 = o2 ? p.N - p.split : p.split, at = m * l2 + (o2 ? n + j - p.split : n + j);
            float f = v[j];
            if (RES) f += IO<T>::ld(static_cast<const T*>(p.R) + at);
            IO<T>::st(static_cast<T*>(o2 ? p.Y1 : p.Y0) + at, f);
        }
    }
}

// Workgroups go to the eight XCDs in turn, each with an L2 of its own: an XCD takes a
// contiguous run of the tiles, in groups of kGqGroup tile rows, so that the tiles it works on
// at one time share rows of X and of W.
constexpr int kGqGroup = 4;
struct GqTile { int m, n; };
__device__ __forceinline__ GqTile gq_tile(unsigned id, int tiles_m, int tiles_n) {
    const unsigned total = (unsigned)tiles_m * (unsigned)tiles_n;
    const unsigned xcd = id & 7u, per = total >> 3, rest = total & 7u;
    const unsigned t = xcd * per + (xcd < rest ? xcd : rest) + (id >> 3);
    const unsigned in_group = kGqGroup * (unsigned)tiles_n;
    const unsigned g = t / in_group, first = g * kGqGroup;
    const unsigned rows = (unsigned)tiles_m - first < kGqGroup ? (unsigned)tiles_m - first : kGqGroup;
    const unsigned at = t - g * in_group;
    return GqTile{(int)(first + at % rows), (int)(at / rows)};
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup of WN x WM waves, each with 16 NF rows of W and 16 MF rows of X. A
// block of both (128 bytes of each row) goes from memory straight into LDS, into one of two
// buffers while the waves multiply the other.
//
// W's rows are dealt to the 16 x 16 products so that a lane ends up with eight consecutive
// columns of Y, four from each of two products: product a takes row
// 32 (a / 2) + 8 (i / 4) + 4 (a % 2) + i % 4 as its row i. A row's eight 16-byte chunks lie in
// LDS at chunk ^ key(row), with a key that spreads the 16 rows a fragment read touches at one
// chunk over the banks; the transfers write LDS in lane order, so the permutation is in what
// they fetch. Rows past the end repeat the last one, chunks past K are zero.
//
// 128 x 128 tiles, four waves of 64 x 64: M 16384, N 10240, K 2560, bf16 out 860 us = 1.0 PFLOP/s (fp32 out
// 910), where a bf16 library product of 8192^3 reaches 1.16. The matrix units are busy 44 percent of
// the time and the other vector instructions, half of them conversions, take another 43 (counters):
// a SIMD's two waves hardly overlap the two. Tiles of 256 x 256 spill; 128 x 256 take 830 here, and
// 17 percent more at M 2048.
__device__ __forceinline__ int gq_key_w(int row) { return (row >> 1 & 1) | (row >> 3 & 3) << 1; }
__device__ __forceinline__ int gq_key_x(int row) { return row >> 1 & 7; }

template <typename T, bool RES, int NF, int MF, int WN, int WM>
__global__ void __launch_bounds__(64 * WN * WM, 2)
k_gemm_q8(const GemmQ8Args p, int tiles_m, int tiles_n) {
    constexpr int TN = 16 * NF * WN, TM = 16 * MF * WM, TH = 64 * WN * WM;
    constexpr int CW = TN * 8 / TH, CX = TM * 8 / TH;             // 16-byte chunks per thread and block
    static_assert(128 % (16 * NF) == 0, "one scale of W per wave");
    using Frag = GqFrag;
    __shared__ gq_i4 sW[2][TN * 8], sX[2][TM * 8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WM, wm = wave % WM;
    const int fr = lane & 15, fc = lane >> 4;
    const int wr = 8 * (fr >> 2) + (fr & 3);                      // row i = fr of product 0; its key is every product's
    const int cw0 = wr * 8 + (fc ^ gq_key_w(wr)), cw1 = wr * 8 + ((fc + 4) ^ gq_key_w(wr));
    const int cx0 = fr * 8 + (fc ^ gq_key_x(fr)), cx1 = fr * 8 + ((fc + 4) ^ gq_key_x(fr));
    auto frag_w = [&](int buf, int a) {
        const int row0 = wn * 16 * NF + 32 * (a / 2) + 4 * (a % 2);
        Frag f;
        f.set(sW[buf][row0 * 8 + cw0], sW[buf][row0 * 8 + cw1]);
        return f;
    };
    auto frag_x = [&](int buf, int b) {
        const int row0 = wm * 16 * MF + 16 * b;
        Frag f;
        f.set(sX[buf][row0 * 8 + cx0], sX[buf][row0 * 8 + cx1]);
        return f;
    };

    // where the next block comes from: a tile's rows, as byte offsets of this thread's chunks in
    // the tile's first block, and their scales
    int64_t m0, n0;
    GqSource from_w(p.wq), from_x(p.xq);
    unsigned ow[CW], ox[CX], xo[MF];
    const float* xsb;
    const float* wsb;
    auto aim = [&](int id) {
        const GqTile tile = gq_tile((unsigned)id, tiles_m, tiles_n);
        m0 = (int64_t)tile.m * TM;
        n0 = (int64_t)tile.n * TN;
        from_w = GqSource(p.wq + n0 * p.K);
        from_x = GqSource(p.xq + m0 * p.K);
        const int rows_w = (int)(p.N - n0 < TN ? p.N - n0 : TN), rows_x = (int)(p.M - m0 < TM ? p.M - m0 : TM);
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            const int idx = tid + TH * i, r = idx >> 3, row = r < rows_w ? r : rows_w - 1;
            ow[i] = (unsigned)row * (unsigned)p.K + 16u * ((idx & 7) ^ gq_key_w(r));
        }
#pragma unroll
        for (int i = 0; i < CX; ++i) {
            const int idx = tid + TH * i, r = idx >> 3, row = r < rows_x ? r : rows_x - 1;
            ox[i] = (unsigned)row * (unsigned)p.K + 16u * ((idx & 7) ^ gq_key_x(r));
        }
        xsb = p.xs + m0 * p.KB;
#pragma unroll
        for (int b = 0; b < MF; ++b) {
            const int r = wm * 16 * MF + 16 * b + fr;
            xo[b] = (unsigned)(r < rows_x ? r : rows_x - 1) * (unsigned)p.KB;
        }
        const int64_t nw = n0 + wn * 16 * NF;
        wsb = p.ws + (nw < p.N ? nw : p.N - 1) / 128 * p.KB;
    };
    auto stage = [&](int kb, int buf) {
        const unsigned k0 = (unsigned)kb * 128u;
#pragma unroll
        for (int i = 0; i < CX; ++i) from_x.to_lds(&sX[buf][64 * wave + TH * i], ox[i], k0);
#pragma unroll
        for (int i = 0; i < CW; ++i) from_w.to_lds(&sW[buf][64 * wave + TH * i], ow[i], k0);
    };
    auto stage_end = [&](int kb, int buf) {                       // the last block of a K that is no multiple of 128
        const unsigned k0 = (unsigned)kb * 128u;
        const int left = (int)(p.K - k0) / 16;                    // its chunks
#pragma unroll
        for (int i = 0; i < CX; ++i) {
            const int idx = tid + TH * i;
            if (((idx & 7) ^ gq_key_x(idx >> 3)) < left) from_x.to_lds(&sX[buf][64 * wave + TH * i], ox[i], k0);
            else sX[buf][idx] = gq_i4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            const int idx = tid + TH * i;
            if (((idx & 7) ^ gq_key_w(idx >> 3)) < left) from_w.to_lds(&sW[buf][64 * wave + TH * i], ow[i], k0);
            else sW[buf][idx] = gq_i4{0, 0, 0, 0};
        }
    };

    gq_f4 acc[NF][MF];
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b) acc[a][b] = gq_f4{0.f, 0.f, 0.f, 0.f};

    const int tiles = tiles_m * tiles_n;
    int id = blockIdx.x, kb = 0, buf = 0;
    aim(id);
    float nx[MF], nws = wsb[0];                                   // the next block's scales
#pragma unroll
    for (int b = 0; b < MF; ++b) nx[b] = xsb[xo[b]];
    if (p.K >= 128) stage(0, 0);
    else stage_end(0, 0);
    while (true) {
        __syncthreads();                                          // this block is in LDS, the last one's readers are done
        float sc[MF];
#pragma unroll
        for (int b = 0; b < MF; ++b) sc[b] = nx[b] * nws;
        const bool last = kb + 1 == p.KB;                         // block of this tile
        const int64_t m_now = m0, n_now = n0;
        const int next = last ? id + (int)gridDim.x : id;
        const int k_next = last ? 0 : kb + 1;
        const bool more = next < tiles;
        const bool whole = more && (unsigned)k_next * 128u + 128u <= (unsigned)p.K;
        if (more) {
            if (last) aim(next);
            nws = wsb[k_next];
#pragma unroll
            for (int b = 0; b < MF; ++b) nx[b] = xsb[xo[b] + k_next];
            if (!whole) stage_end(k_next, buf ^ 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        Frag fx[MF];
#pragma unroll
        for (int b = 0; b < MF; ++b) fx[b] = frag_x(buf, b);
        Frag fw = frag_w(buf, 0);
        // behind the first fragment reads (in front of them, or spread over the products, measured slower)
        if (whole) stage(k_next, buf ^ 1);
        gq_f4 q[MF];                                              // the last product row's results, on their way to acc
#pragma unroll
        for (int a = 0; a <= NF; ++a) {
            gq_f4 t[MF];
            if (a < NF) {
                const Frag cur = fw;
                if (a + 1 < NF) fw = frag_w(buf, a + 1);
                gq_dot(cur, fx, t);
            }
            if (a > 0) {
#pragma unroll
                for (int b = 0; b < MF; ++b) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[a - 1][b][v] = __builtin_fmaf(q[b][v], sc[b], acc[a - 1][b][v]);
                    asm volatile("" : "+v"(acc[a - 1][b]));   // here, and not behind all the products, whose results do not fit
                }
            }
#pragma unroll
            for (int b = 0; b < MF; ++b) q[b] = t[b];
            // one matrix instruction, then two of the additions and conversions that run in its shadow
            if (a + 1 < NF) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
            for (int b = 0; b < 4 * MF; ++b) {
                if (a < NF) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        buf ^= 1;
        if (!last) {
            ++kb;
            continue;
        }
        // the tile is done: its stores run under the next tile's first blocks
#pragma unroll
        for (int a = 0; a < NF; a += 2)
#pragma unroll
            for (int b = 0; b < MF; ++b) {
                const float v[8] = {acc[a][b][0], acc[a][b][1], acc[a][b][2], acc[a][b][3],
                                    acc[a + 1][b][0], acc[a + 1][b][1], acc[a + 1][b][2], acc[a + 1][b][3]};
                gq_store<T, RES, 8>(p, m_now + wm * 16 * MF + 16 * b + fr, n_now + (wn * NF + a) * 16 + 8 * fc, v);
                acc[a][b] = acc[a + 1][b] = gq_f4{0.f, 0.f, 0.f, 0.f};
            }
        if (next >= tiles) break;
        id = next;
        kb = 0;
    }
}

// ---------------------------------------------------------------------------
// Few tiles: KS groups of WN x WM waves share a workgroup's tile and take the blocks of k in
// turn, each with two LDS buffers of its own, so that a CU has enough bytes on their way and
// waves enough to read and multiply them while the grid is short. What bounds it is the waves'
// instructions (three buffers with as many fewer groups were slower by a tenth), so a whole
// block's transfers have no conditions, the scales come by transfers as well (the first wave of a
// group fetches them) and a step knows its buffer. The groups' sums meet in LDS and are added in
// order. Staged as above; row i of product a is row 16 a + i of the wave's rows of W.
template <typename T, bool RES, int NF, int MF, int WN, int WM, int KS>
__global__ void __launch_bounds__(64 * WN * WM * KS)
k_gemm_q8_split(const GemmQ8Args p, int tiles_m, int tiles_n) {
    constexpr int TN = 16 * NF * WN, TM = 16 * MF * WM, TH = 64 * WN * WM;
    constexpr int CW = (TN * 8 + TH - 1) / TH, CX = (TM * 8 + TH - 1) / TH;
    constexpr int LD = TN + 4;                                    // row of the sums: 4 floats on, against bank conflicts
    constexpr int BUF = (TN + TM) * 8 + 32;                       // chunks of a buffer: W, X, 64 scales of X, 64 times that of W
    static_assert(128 % TN == 0 && (TN * 8) % 64 == 0 && (TM * 8) % 64 == 0 && TM <= 64, "one scale of W; whole transfers");
    static_assert(TM * LD * 4 <= 2 * BUF * 16, "the sums fit in the block buffers");
    static_assert(TN * 8 % TH == 0 && (TM * 8 % TH == 0 || CX == 1), "no condition on W's transfers, one on X's");
    using Frag = GqFrag;
    __shared__ gq_i4 lds[KS][2 * BUF];
    const int tid = threadIdx.x % TH, lane = tid & 63;
    const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / TH);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WM, wm = wave % WM;
    const int fr = lane & 15, fc = lane >> 4;
    const GqTile tile = gq_tile(blockIdx.x, tiles_m, tiles_n);
    const int64_t m0 = (int64_t)tile.m * TM, n0 = (int64_t)tile.n * TN;

    const GqSource from_w(p.wq + n0 * p.K), from_x(p.xq + m0 * p.K);
    const GqSource from_ws(reinterpret_cast<const uint8_t*>(p.ws + n0 / 128 * p.KB)), from_xs(reinterpret_cast<const uint8_t*>(p.xs + m0 * p.KB));
    const int rows_w = (int)(p.N - n0 < TN ? p.N - n0 : TN), rows_x = (int)(p.M - m0 < TM ? p.M - m0 : TM);
    unsigned ow[CW], ox[CX];
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        const int idx = tid + TH * i, r = idx >> 3, row = r < rows_w ? r : rows_w - 1;
        ow[i] = (unsigned)row * (unsigned)p.K + 16u * ((idx & 7) ^ gq_key_x(r));
    }
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const int idx = tid + TH * i, r = idx >> 3, row = r < rows_x ? r : rows_x - 1;
        ox[i] = (unsigned)row * (unsigned)p.K + 16u * ((idx & 7) ^ gq_key_x(r));
    }
    const unsigned os = (unsigned)(lane < rows_x ? lane : rows_x - 1) * (unsigned)p.KB * 4u;
    auto stage = [&](int kb, gq_i4* to) {
        if (kb >= p.KB) return;
        const unsigned k0 = (unsigned)kb * 128u;
        const int left = ((int)p.K - (int)k0) / 16;               // chunks from this block on
        if (wave == 0) {
            from_xs.to_lds4(to + (TN + TM) * 8, os, (unsigned)kb * 4u);
            from_ws.to_lds4(to + (TN + TM) * 8 + 16, 0u, (unsigned)kb * 4u);
        }
        auto part = [&](auto whole) {                             // a whole block, or one that K ends in
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                const int idx = tid + TH * i;
                if (decltype(whole)::value || ((idx & 7) ^ gq_key_x(idx >> 3)) < left)
                    from_w.to_lds(to + 64 * wave + TH * i, ow[i], k0);
                else to[idx] = gq_i4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < CX; ++i) {
                const int idx = tid + TH * i;
                if (TM * 8 % TH == 0 || 64 * wave < TM * 8) {       // uniform: whole waves
                    if (decltype(whole)::value || ((idx & 7) ^ gq_key_x(idx >> 3)) < left)
                        from_x.to_lds(to + TN * 8 + 64 * wave + TH * i, ox[i], k0);
                    else to[TN * 8 + idx] = gq_i4{0, 0, 0, 0};
                }
            }
        };
        if (left >= 8) part(std::true_type{});
        else part(std::false_type{});
    };
    const int c0 = fr * 8 + (fc ^ gq_key_x(fr)), c1 = fr * 8 + ((fc + 4) ^ gq_key_x(fr));
    auto frag = [&](const gq_i4* s, int row0) {
        Frag f;
        f.set(s[row0 * 8 + c0], s[row0 * 8 + c1]);
        return f;
    };
    gq_f4 acc[NF][MF];
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b) acc[a][b] = gq_f4{0.f, 0.f, 0.f, 0.f};

    auto step = [&](int kb, auto which) {
        const gq_i4* buf = lds[grp] + decltype(which)::value * BUF;
        __syncthreads();                                          // this block is in LDS, the last one's readers are done
        stage(kb + KS, lds[grp] + (1 - decltype(which)::value) * BUF);
        if (kb >= p.KB) return;
        const float* scales = reinterpret_cast<const float*>(buf + (TN + TM) * 8);
        const float sw = scales[64 + lane];
        float sc[MF];
        Frag fx[MF];
#pragma unroll
        for (int b = 0; b < MF; ++b) {
            sc[b] = scales[wm * 16 * MF + 16 * b + fr] * sw;
            fx[b] = frag(buf + TN * 8, wm * 16 * MF + 16 * b);
        }
#pragma unroll
        for (int a = 0; a < NF; ++a) {
            const Frag fw = frag(buf, wn * 16 * NF + 16 * a);
            gq_f4 q[MF];
            gq_dot(fw, fx, q);
#pragma unroll
            for (int b = 0; b < MF; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[a][b][v] = __builtin_fmaf(q[b][v], sc[b], acc[a][b][v]);
        }
    };
    stage(grp, lds[grp]);
    for (int kb = grp; kb - grp < p.KB; kb += 2 * KS) {
        step(kb, std::integral_constant<int, 0>{});
        if (kb - grp + KS < p.KB) step(kb + KS, std::integral_constant<int, 1>{});
    }
    __syncthreads();                                              // every block is read: the buffers hold the sums now
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b)
            *reinterpret_cast<gq_f4*>(reinterpret_cast<float*>(lds[grp]) + (wm * 16 * MF + 16 * b + fr) * LD + wn * 16 * NF +
                                      16 * a + 4 * fc) = acc[a][b];
    __syncthreads();
    for (int i = threadIdx.x; i < TM * TN / 8; i += TH * KS) {
        const int r = i / (TN / 8), c = i % (TN / 8) * 8;
        float v[8];
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            gq_f4 t = *reinterpret_cast<const gq_f4*>(reinterpret_cast<const float*>(lds[0]) + r * LD + c + h);
#pragma unroll
            for (int g = 1; g < KS; ++g) t += *reinterpret_cast<const gq_f4*>(reinterpret_cast<const float*>(lds[g]) + r * LD + c + h);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[h + j] = t[j];
        }
        gq_store<T, RES, 8>(p, m0 + r, n0 + c, v);
    }
}

// Which kernel (measured, microseconds, bf16 outputs; fp32 ones are up to 5 percent above). The smallest
// of these tiles of which there are no more than CUs, so that each has a CU to itself, whose waves
// split k four or eight ways (at K 128 and 512 they are within 0.6 of each other, 3.8 to 4.8):
//  - 16 x 32: M 16, N 2560, K 2048 4.3 (16 x 64: 5.8), K 8192 10.4 (16.7);
//  - 16 x 64 where X has no more rows: M 16, N 10240, K 2048 6.9 (64 x 64: 7.8, 16 x 32 8.6), K 8192 18.9 (21.1, 22.8);
//  - 32 x 32: M 64, N 2560, K 2048 5.0 (32 x 64: 6.0), K 8192 11.9 (16.7);
//  - 32 x 64: M 32, N 10240, K 2048 7.2 (64 x 64: 8.2), K 8192 19.6 (21.4);
//  - 64 x 64: M 200, N 2560, K 2048 7.8 (32 x 64: 10.7, split two ways 9.1), K 8192 22.0 (31.7, 28.9).
// With more, k split two ways and two workgroups to a CU or more: 32 x 64 for a single row of tiles
// (M 64, N 40960, K 512 8.4, K 2048 20.2; 64 x 64: 9.5, 21.2; 128 x 128: 11.4, 31.9), else the cheaper by
// n = tiles / CUs, rounded up, and KB = blocks of k, in twentieths of a microsecond:
//  - 64 x 64: n (16 + 6 KB) + 2 KB;
//  - 128 x 128: n (28 + 19 KB) + 3 KB.
// 64 x 64 against 128 x 128 at K 128, 512, 2048, 8192: M 192, N 10240 4.7 4.8, 6.1 8.0, 14.2 22.2, 45.6 77.4;
// M 512 9.2 6.9, 12.3 12.4, 32.2 35.3, 110 128; M 1024 15.5 9.7, 21.8 16.9, 60.4 51.6, 215 190; M 2048 27.3 14.4,
// 40.3 26.6, 114 88, 413 319; M 1500, N 3000 9.0 6.5, 12.2 11.9, 30.3 34.0, 104 124.
constexpr int64_t kGqCUs = 256;
template <typename T, bool RES>
hipError_t launch_gemm_q8_t(const LaunchGemmQ8& p) {
    const GemmQ8Args a{p.xq, p.xs, p.wq, p.ws, p.R, p.Y[0], p.Y[1], p.split, p.M, p.N, p.K, (int)((p.K + 127) / 128)};
    hipStream_t st = static_cast<hipStream_t>(p.stream);
    auto count = [&](int64_t m, int64_t n) { return ((p.M + m - 1) / m) * ((p.N + n - 1) / n); };
    auto go = [&](auto kernel, int m, int n, int threads, int64_t most) {
        const int tm = (int)((p.M + m - 1) / m), tn = (int)((p.N + n - 1) / n);
        const int64_t tiles = (int64_t)tm * tn;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < most ? tiles : most)), dim3((unsigned)threads), 0, st, a, tm, tn);
        return hipGetLastError();
    };
    constexpr int64_t kAll = INT32_MAX;
    if (count(16, 32) <= kGqCUs) return go(k_gemm_q8_split<T, RES, 2, 1, 1, 1, 8>, 16, 32, 512, kAll);
    if (p.M <= 16 && count(16, 64) <= kGqCUs) return go(k_gemm_q8_split<T, RES, 1, 1, 4, 1, 4>, 16, 64, 1024, kAll);
    if (count(32, 32) <= kGqCUs) return go(k_gemm_q8_split<T, RES, 2, 2, 1, 1, 8>, 32, 32, 512, kAll);
    if (count(32, 64) <= kGqCUs) return go(k_gemm_q8_split<T, RES, 2, 2, 2, 1, 4>, 32, 64, 512, kAll);
    if (count(64, 64) <= kGqCUs) return go(k_gemm_q8_split<T, RES, 2, 4, 2, 1, 4>, 64, 64, 512, kAll);
    // (a launch holds fewer than 2^32 lanes: more than 2^22 tiles go to the persistent kernels)
    constexpr int64_t kMost = int64_t(1) << 22;
    if (p.M <= 64 && count(32, 64) <= kMost) return go(k_gemm_q8_split<T, RES, 2, 2, 2, 1, 2>, 32, 64, 256, kAll);
    auto turns = [&](int64_t m, int64_t n) { return (count(m, n) + kGqCUs - 1) / kGqCUs; };
    const int64_t kb = a.KB;
    const int64_t t64 = turns(64, 64) * (16 + 6 * kb) + 2 * kb, t128 = turns(128, 128) * (28 + 19 * kb) + 3 * kb;
    // the grid of the persistent kernel is a multiple of the eight XCDs: a workgroup's tiles stay on one
    if (t64 < t128 && count(64, 64) <= kMost) return go(k_gemm_q8_split<T, RES, 2, 4, 2, 1, 2>, 64, 64, 256, kAll);
    return go(k_gemm_q8<T, RES, 4, 4, 2, 2>, 128, 128, 256, 2 * kGqCUs);
}

}  // namespace selscan
