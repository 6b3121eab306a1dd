// Device code of the gated delta rule (ss_gdr_fwd, ss_gdr_bwd, ss_gdr_step).
//
//   S' = e^g_t S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,  y_t = scale S_t^T q_t
//
// Chunks of 64 tokens. With G the running sum of g inside a chunk, D_ij = e^(G_i - G_j) for i >= j and
// S0 the state in front of it, x_t = u_t / beta_t solves a triangular system that needs no state,
//
//   (1 + N) X = V - e^G (K S0),    N_ij = beta_j D_ij (k_i . k_j), i > j
//   Y = scale e^G (Q S0) + (P beta) X,    P_ij = scale D_ij (q_i . k_j), i >= j
//   S = e^G_last S0 + (beta e^(G_last - G) K)^T X
//
// k_gdr_solve makes (1 + N)^-1 and the tokens' factors for every chunk at once; k_gdr_walk goes from
// chunk to chunk with the state in registers. The columns of S are independent, so a head is split over
// workgroups by them. q and k enter the matrix cores as they came; their lengths are factors of tokens.
// The backward makes the transposed inverses, goes through the chunks from the last to the first
// (k_gdr_walk_back) and then makes every chunk's gradients at once from the states on both sides (k_gdr_grads).
//
// Layout of the matrix instructions (16 x 16 tiles, 32 terms of a sum): lane l = 16 g + m holds row m of
// A, or column m of B, at the terms 4 g + r and 16 + 4 g + r, r < 4, of its 32 (any order of the terms
// is right as long as both operands have the same). The result's lane holds column m at rows 4 g + r: two
// tiles of a result below each other are the next product's B without a move between lanes. So
// a wave keeps its columns of the state and everything that is made from them in registers, and
// only A operands, which all waves share, lie in LDS, in the order in which lanes read them.
#pragma once
#include "ops_layer_internal.h"
#include "selscan_device.h"

namespace selscan {

typedef float gf4 __attribute__((ext_vector_type(4)));
typedef float gf8 __attribute__((ext_vector_type(8)));
typedef __bf16 gb8 __attribute__((ext_vector_type(8)));
typedef short gs4 __attribute__((ext_vector_type(4)));
typedef uint32_t gu4 __attribute__((ext_vector_type(4)));

constexpr int kGdrC = SS_GDR_CHUNK;           // 64
static_assert(kGdrC == 64, "a wave is a chunk's tokens");

// Operands by I/O type. bf16: q, k, v and gradients of y are exact operands; what is made in fp32
// (states, inverses, solutions) goes in as a sum of three bf16 terms (24 bits, and the six largest of the nine products of
// two such: 2^-24 of their size is left out, as a rounding to fp32 leaves it out). fp32: every operand as three terms, made where
// it is read: six bf16 products take 2.7 times less of the matrix cores than one fp32 product, and with
// their terms made a chunk still takes less (a prompt of 64 tokens: 20.6 to 17 us).
template <typename T> struct Mx;

template <> struct Mx<uint16_t> {
    static constexpr int NT = 3;                                // terms of what is made in fp32
    static_assert(NT * 2 == kGdrInverseBytes<true>);
    typedef gb8 F;
    template <int N> struct S { gb8 t[N]; };
    static __device__ __forceinline__ F ld(const uint16_t* p) { return *reinterpret_cast<const gb8*>(p); }
    // Two values a conversion; what each leaves, v - its term, by the product of two pairs with (-1, 0) or (0, -1), which is
    // exact and one instruction where taking the term out of its half would be another. (The pair is a register: as
    // an immediate it is taken for a float's, with -1 in the upper half.)
    template <int N>
    static __device__ __forceinline__ S<N> split(gf8 v) {
        typedef __bf16 gb2 __attribute__((ext_vector_type(2)));
        typedef float gf2 __attribute__((ext_vector_type(2)));
        uint32_t lower = 0x0000bf80u, upper = 0xbf800000u;
        asm("" : "+s"(lower), "+s"(upper));
        S<N> s;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            gu4 u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const gb2 t = __builtin_convertvector(gf2{v[2 * j], v[2 * j + 1]}, gb2);
                u[j] = __builtin_bit_cast(uint32_t, t);
                if (k + 1 < N) {
                    v[2 * j] = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(gb2, lower), v[2 * j], false);
                    v[2 * j + 1] = __builtin_amdgcn_fdot2_f32_bf16(t, __builtin_bit_cast(gb2, upper), v[2 * j + 1], false);
                }
            }
            s.t[k] = __builtin_bit_cast(gb8, u);
        }
        return s;
    }
    static __device__ __forceinline__ gf4 mm(const gb8& a, const gb8& b, gf4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // the pairs of terms of a product of two sums, the smallest first
    template <int N, typename Fn>
    static __device__ __forceinline__ void each(Fn&& f) {
        if constexpr (N == 3) { f(1, 1); f(2, 0); f(0, 2); }
        f(1, 0);
        f(0, 1);
        f(0, 0);
    }
    // an exact operand by a sum of terms
    template <int N>
    static __device__ __forceinline__ gf4 mul(const F& a, const S<N>& b, gf4 c) {
#pragma unroll
        for (int k = N - 1; k >= 0; --k) c = mm(a, b.t[k], c);
        return c;
    }
    template <int N>
    static __device__ __forceinline__ gf4 mul(const S<N>& a, const F& b, gf4 c) {
#pragma unroll
        for (int k = N - 1; k >= 0; --k) c = mm(a.t[k], b, c);
        return c;
    }
    template <int N>
    static __device__ __forceinline__ gf4 mul(const S<N>& a, const S<N>& b, gf4 c) {
        if constexpr (N == 3) {
            c = mm(a.t[1], b.t[1], c);
            c = mm(a.t[2], b.t[0], c);
            c = mm(a.t[0], b.t[2], c);
        }
        c = mm(a.t[1], b.t[0], c);
        c = mm(a.t[0], b.t[1], c);
        return mm(a.t[0], b.t[0], c);
    }
};

template <> struct Mx<float> {
    static constexpr int NT = 1;
    static_assert(NT * 4 == kGdrInverseBytes<false>);
    typedef gf8 F;
    template <int N> struct S { gf8 t[1]; };
    template <int N, typename Fn>
    static __device__ __forceinline__ void each(Fn&& f) { f(0, 0); }
    static __device__ __forceinline__ F ld(const float* p) { return *reinterpret_cast<const gf8*>(p); }
    template <int N>
    static __device__ __forceinline__ S<N> split(gf8 v) { return S<N>{{v}}; }
    static __device__ __forceinline__ gf4 mm(const gf8& a, const gf8& b, gf4 c) {
        const auto x = Mx<uint16_t>::split<3>(a), y = Mx<uint16_t>::split<3>(b);
        return Mx<uint16_t>::mul(x, y, c);
    }
    template <int N>
    static __device__ __forceinline__ gf4 mul(const F& a, const S<N>& b, gf4 c) { return mm(a, b.t[0], c); }
    template <int N>
    static __device__ __forceinline__ gf4 mul(const S<N>& a, const F& b, gf4 c) { return mm(a.t[0], b, c); }
    template <int N>
    static __device__ __forceinline__ gf4 mul(const S<N>& a, const S<N>& b, gf4 c) { return mm(a.t[0], b.t[0], c); }
};

__device__ __forceinline__ gf8 gdr_pair(gf4 a, gf4 b) { return gf8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// This wave's number, known to be the same in all its lanes.
__device__ __forceinline__ int gdr_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The blocks of an upper triangle of 64 x 64 that hold anything, 16 rows by 32 columns: (row tile, column
// pair) 00 01 10 11 21 31.
__device__ __forceinline__ constexpr int gdr_up(int mt, int s) { return mt < 2 ? 2 * mt + s : mt + 2; }
// Where a block of a lower triangle lies, in values: 10 20 30 31, then the first halves of 00 and 21, whose others are above the
// diagonal. (Three terms of T and of P then take what three and two would in whole blocks, and two workgroups' LDS fits a CU.)
__device__ __forceinline__ constexpr bool gdr_half(int mt, int s) { return mt == 2 * s; }
__device__ __forceinline__ constexpr int gdr_low(int mt, int s) { return gdr_half(mt, s) ? 4 * 512 + s * 256 : (mt - 1 + s) * 512; }

// Eight values of a row at d, zeros past dk or (none) in a row that is not there.
template <typename T>
__device__ __forceinline__ void gdr_row8(const T* row, int d, int dk, bool vec, bool there, T* out) {
    if (there && vec && d < dk) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<gu4*>(out) = *reinterpret_cast<const gu4*>(row + d);
        } else {
            *reinterpret_cast<gu4*>(out) = *reinterpret_cast<const gu4*>(row + d);
            *reinterpret_cast<gu4*>(out + 4) = *reinterpret_cast<const gu4*>(row + d + 4);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = there && d + j < dk ? row[d + j] : T(0);
    }
}

template <typename T>
__device__ __forceinline__ float gdr_f(T v) { return IO<T>::ld(&v); }

__device__ __forceinline__ void gdr_tile(int tile, int& mt, int& nt) {
    mt = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3;
    nt = tile - mt * (mt + 1) / 2;
}

// ---------------------------------------------------------------------------
// Operands in LDS: 64 rows of DKP columns as fragments (row tile i, columns 32 s to 32 s + 31): lane 16 g + m
// reads row 16 i + m at columns 32 s + 8 g + j, 16 bytes (an fp32 fragment is two such units, j < 4 and the rest).
// A unit goes from memory to LDS without registers, 16 bytes a lane at consecutive places: place
// 4 m + (g ^ (m >> 1 & 3)), so that neither the lanes that read a fragment nor those that read across rows for the
// transposed one meet in a bank. The state's tiles follow: row 4 g + r of tile 2 s + h is d = 32 s + 8 g + 4 h + r.
__device__ __forceinline__ int gdr_place(int g, int m) { return 4 * m + (g ^ (m >> 1 & 3)); }

template <typename T>
__device__ __forceinline__ typename Mx<T>::F gdr_rows_frag(const T* base, int unit, int place) {
    if constexpr (sizeof(T) == 2) return *reinterpret_cast<const gb8*>(base + (unit * 64 + place) * 8);
    else return gdr_pair(*reinterpret_cast<const gf4*>(base + (unit * 128 + place) * 4), *reinterpret_cast<const gf4*>(base + (unit * 128 + 64 + place) * 4));
}
// Operands that are made here lie by lane.
template <typename T>
__device__ __forceinline__ typename Mx<T>::F gdr_frag(const T* base, int unit, int lane) { return gdr_rows_frag<T>(base, unit, lane); }

// The transposed operand: rows are the columns of the state's tile (sd, h), terms the tokens of the row
// tiles 2 s and 2 s + 1.
template <typename T, int KD>
__device__ __forceinline__ typename Mx<T>::F gdr_frag_t(const T* base, int s, int sd, int h, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (sizeof(T) == 2) {
        const int place = gdr_place(i & 3, 4 * g + (i >> 2));
        gs4 a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const T* q = base + (((2 * s + e) * KD + sd) * 64 + place) * 8 + 4 * h;
            a[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((gs4 __attribute__((address_space(3)))*)q);
        }
        typedef short gs8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(gb8, gs8{a[0][0], a[0][1], a[0][2], a[0][3], a[1][0], a[1][1], a[1][2], a[1][3]});
    } else {
        gf8 a;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            a[j] = base[((((2 * s + (j >> 2)) * KD + sd) * 2 + h) * 64 + gdr_place(i >> 2, 4 * g + (j & 3))) * 4 + (i & 3)];
        return a;
    }
}
// A term of an operand over tokens: block of the triangle's six (or any unit), as above.
template <typename T, int N>
__device__ __forceinline__ typename Mx<T>::template S<N> gdr_terms(const T* base, int plane, int unit, int lane) {
    typename Mx<T>::template S<N> f;
#pragma unroll
    for (int k = 0; k < (sizeof(T) == 2 ? N : 1); ++k) f.t[k] = gdr_frag<T>(base + k * plane, unit, lane);
    return f;
}

// The same of a lower triangle.
template <typename T>
__device__ __forceinline__ typename Mx<T>::template S<Mx<T>::NT> gdr_low_terms(const T* base, int mt, int s, int lane) {
    typename Mx<T>::template S<Mx<T>::NT> f;
#pragma unroll
    for (int k = 0; k < Mx<T>::NT; ++k) {
        const T* at = base + k * kGdrLow + gdr_low(mt, s);
        if (!gdr_half(mt, s)) {
            f.t[k] = gdr_frag<T>(at, 0, lane);
        } else if constexpr (sizeof(T) == 2) {
            typedef short gs8 __attribute__((ext_vector_type(8)));
            const gs4 a = *reinterpret_cast<const gs4*>(at + lane * 4);
            f.t[k] = __builtin_bit_cast(gb8, gs8{a[0], a[1], a[2], a[3], 0, 0, 0, 0});
        } else {
            f.t[k] = gdr_pair(*reinterpret_cast<const gf4*>(at + lane * 4), gf4{0, 0, 0, 0});
        }
    }
    return f;
}

// Elements at a lane's offset and the wave's, in bytes, from a chunk's start: no 64-bit address per element. At `bytes` and
// behind it nothing is stored and zeros are read, so that the last rows and columns need no branch: a lane that has none is
// at kGdrOut. (The wave's part is below `bytes` wherever it is used.)
constexpr unsigned kGdrOut = 0x80000000u;
template <typename T>
struct GdrBuf {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit GdrBuf(const T* p, unsigned bytes = ~0u)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), 0, (int)bytes, kBufDword3)) {}
    __device__ __forceinline__ T ld(unsigned lane, unsigned wave) const {
        if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, lane, wave, 0);
        else return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, lane, wave, 0));
    }
    __device__ __forceinline__ gu4 ld16(unsigned lane) const { return __builtin_amdgcn_raw_buffer_load_b128(r, lane, 0, 0); }
    // eight values from column c of n on, `at` bytes from the start, zeros past n. VEC: rows are whole accesses of 16 bytes
    // (known when compiling: where two ways to load meet, the values are copied, and the copy waits for them). An access of
    // 16 bytes may start at any dword, so that fp32 needs no others, only its last columns cut.
    template <bool VEC>
    __device__ __forceinline__ void ld8(unsigned at, int c, int n, T* out) const {
        constexpr int E = 16 / (int)sizeof(T);
        if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < 8 / E; ++e) reinterpret_cast<gu4*>(out)[e] = ld16(c + e * E < n ? at + e * 16 : kGdrOut);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 8 / E; ++e) reinterpret_cast<gu4*>(out)[e] = ld16(c + e * E < n ? at + e * 16 : kGdrOut);
            if (n - c < 8)
#pragma unroll
                for (int j = 0; j < 8; ++j) out[j] = c + j < n ? out[j] : T(0);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = ld(c + j < n ? at + j * (unsigned)sizeof(T) : kGdrOut, 0);
        }
    }
    template <bool VEC>
    __device__ __forceinline__ gf8 ld8(unsigned at, int c, int n) const {
        alignas(16) T x[8];
        ld8<VEC>(at, c, n, x);
        return __builtin_bit_cast(gf8, x);
    }
    __device__ __forceinline__ void st(float v, unsigned lane, unsigned wave) const {
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(IO<T>::bits(v), r, lane, wave, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, lane, wave, 0);
    }
    __device__ __forceinline__ void st4(gf4 v, unsigned lane, unsigned wave) const {
        if constexpr (sizeof(T) == 2) {
            typedef __bf16 gb4 __attribute__((ext_vector_type(4)));
            typedef uint32_t gu2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(gu2, __builtin_convertvector(v, gb4)), r, lane, wave, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(gu4, v), r, lane, wave, 0);
        }
    }
};

// 64 lanes' 16 bytes from memory straight into 1024 consecutive bytes of LDS, a lane's offset and the wave's.
struct GdrSource {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ explicit GdrSource(const void* p) : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, -1, kBufDword3)) {}
    __device__ __forceinline__ void to_lds(gu4* lds, unsigned lane, unsigned wave) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, lds, 16, lane, wave, 0, 0);
    }
};

// Where a head's keys or queries lie. AL: rows start on 16 bytes, hold whole accesses of 16 bytes, and 64 of them
// lie within 32-bit offsets.
template <typename T, int KD, bool AL>
struct GdrRows {
    const T* base;
    int64_t stride;
    int dk;
    __device__ __forceinline__ GdrRows(const ss_head_view& v, int64_t b, int head, int dk_)
        : base(static_cast<const T*>(v.p) + b * v.batch_stride + head * v.head_stride), stride(v.token_stride), dk(dk_) {}
    // 64 rows from token t0 on into `tiles`, rows past the last token as copies of it (what they are multiplied by is
    // 0). Columns past dk are left as they are (AL) or 0. Complete once this wave's loads are.
    __device__ __forceinline__ void load(T* tiles, int64_t t0, int64_t L) const {
        const T* at = base + t0 * stride;
        const int last = L - t0 < 64 ? (int)(L - t0) - 1 : 63;
        if constexpr (AL) {
            constexpr int H = sizeof(T) / 2, U = 4 * KD * H;          // units of 16 bytes a lane
            const int lane = threadIdx.x & 63, w = gdr_wave(), m = lane >> 2, g = (lane & 3) ^ (m >> 1 & 3);
            const GdrSource from(at);
            const unsigned row_bytes = (unsigned)stride * (unsigned)sizeof(T), lo = 8 * g * (unsigned)sizeof(T);
            if (last == 63) {
#pragma unroll
                for (int e = 0; e < U / 4; ++e) {
                    const int u = e * 4 + w, h = u % H, s = u / H % KD;
                    if (32 * s + 8 * g < dk)
                        from.to_lds(reinterpret_cast<gu4*>(tiles + u * (1024 / sizeof(T))), m * row_bytes + lo,
                                    16 * (u / H / KD) * row_bytes + (32 * s + 4 * h) * (unsigned)sizeof(T));
                }
            } else {
#pragma unroll
                for (int e = 0; e < U / 4; ++e) {
                    const int u = e * 4 + w, h = u % H, s = u / H % KD, row = 16 * (u / H / KD) + m;
                    if (32 * s + 8 * g < dk)
                        from.to_lds(reinterpret_cast<gu4*>(tiles + u * (1024 / sizeof(T))), (row < last ? row : last) * row_bytes + lo,
                                    (32 * s + 4 * h) * (unsigned)sizeof(T));
                }
            }
        } else {
            // eights of a row, element by element, two of them in flight
#pragma unroll 1
            for (int e = threadIdx.x; e < 256 * KD; e += 512) {
                alignas(16) T x[2][8];
                int to[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int o = (e + 256 * u) % (4 * KD), row = (e + 256 * u) / (4 * KD);
                    const T* from = at + (row < last ? row : last) * stride;
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[u][j] = from[8 * o + j < dk ? 8 * o + j : dk - 1];
                    to[u] = ((row >> 4) * KD + (o >> 2)) * 512 + gdr_place(o & 3, row & 15) * (16 / (int)sizeof(T));
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int o = (e + 256 * u) % (4 * KD);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (8 * o + j >= dk) x[u][j] = T(0);
#pragma unroll
                    for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                        *reinterpret_cast<gu4*>(tiles + to[u] + 256 * h) = reinterpret_cast<const gu4*>(x[u])[h];
                }
            }
        }
    }
};

// What k_gdr_solve leaves of a chunk's tokens: rows of 64 floats.
//   a1 e^G / |k|, a2 e^G, a3 beta e^(G_last - G) / |k|, bk beta / |k|, misc { e^G_last, whether no factor is 0,
//   G_last in powers of two, whether every beta |k|^2 is in [0, 2], whether a decay is 0,
//   whether a key, a beta or a log decay is not finite },
//   G itself, times log2 e, in 64 bits (two rows)
//   for the gradients as well: e^(G_last - G) / |k|, beta, 1 / |k|
enum GdrTok { tA1, tA2, tA3, tBk, tMisc, tG, kGdrTok = 7, tA3b = 7, tBeta, tRk, kGdrTokAll };

// Waits for this wave's transfers to LDS, then for the workgroup's.
__device__ __forceinline__ void gdr_arrived() {
    __builtin_amdgcn_s_waitcnt(0x0f70);               // vmcnt(0)
    __syncthreads();
}

// ---------------------------------------------------------------------------
// A chunk of one head: its factors and T = (1 + N)^-1, one wave each, so that nothing waits for a barrier.
// Sums of g in 64 bits: a reset, or a decay of any size, is a term of -200 at least (e^-200 is 0 in
// fp32), and the differences of what follows keep their digits. The inverse: blocks of 16 on the
// diagonal row by row, below them block by block, T_ij = -T_ii sum_l N_il T_lj, in fp32 products
// whose operands stay in registers.
// BACK: T transposed, which is how the results lie.
// 32768 chunks of keys of 128 in bf16: 272 us, 4.1 TB/s of keys read and factors written, which is what bounds
// it; 4 chunks: 11 us, one wave's chain of products.
template <typename T, int DKP, bool BACK>
__global__ void __launch_bounds__(256)
k_gdr_solve(const LaunchGdr p) {
    using M = Mx<T>;
    constexpr int KD = DKP / 32, LD = 68;
    __shared__ alignas(16) float mats[4][64 * LD];
    __shared__ alignas(16) double sg[4][64];
    __shared__ alignas(16) float sv[4][2][64];
    const int lane = threadIdx.x & 63, w = gdr_wave(), g = lane >> 4, m = lane & 15;
    const int64_t id = (int64_t)blockIdx.x * 4 + w, nc = p.nchunks;
    if (id >= p.B * p.H * nc) return;                 // whole waves, and no barrier below
    const int64_t n = id % nc, bh = id / nc, b = bh / p.H, t0 = n * kGdrC;
    const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk);
    float* mat = mats[w];

    double G = 0.0;
    float beta = 0.0f;
    bool cut = false;
    if (t0 + lane < p.L) {
        const int64_t at = (b * p.L + t0 + lane) * p.H + h;
        G = (double)p.g[at];
        beta = p.beta[at];
        cut = p.reset && p.reset[b * p.L + t0 + lane];
    }
    // products of keys: the lower triangle's ten tiles
    gf4 kk[10] = {};
    {
        const T* base = static_cast<const T*>(p.k.p) + b * p.k.batch_stride + hk * p.k.head_stride + t0 * p.k.token_stride;
        const int last = p.L - t0 < 64 ? (int)(p.L - t0) - 1 : 63;
#pragma unroll
        for (int s = 0; s < KD; ++s) {
            typename M::F f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * i + m, d = 32 * s + 8 * g;
                const T* at = base + (row < last ? row : last) * p.k.token_stride;
                alignas(16) T x[8];
                if (p.vec) {
                    const T* from = at + (d < p.dk ? d : 0);
#pragma unroll
                    for (int e = 0; e < (int)sizeof(T) / 2; ++e) reinterpret_cast<gu4*>(x)[e] = reinterpret_cast<const gu4*>(from)[e];
                    if (d >= p.dk)
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = T(0);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const T v = at[d + j < p.dk ? d + j : p.dk - 1];
                        x[j] = d + j < p.dk ? v : T(0);
                    }
                }
                f[i] = __builtin_bit_cast(typename M::F, x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) kk[i * (i + 1) / 2 + j] = M::mm(f[i], f[j], kk[i * (i + 1) / 2 + j]);
        }
    }
    cut |= G <= -200.0;
    G = (cut ? -200.0 : G) * 1.4426950408889634;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(G, o, 64);
        if (lane >= o) G += u;
    }
    const double Gl = __shfl(G, 63, 64);
    sg[w][lane] = G;
    // lengths of keys: the diagonal
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (m == 4 * g + r) sv[w][0][16 * i + m] = kk[i * (i + 1) / 2 + i][r];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const float k2 = sv[w][0][lane], rk = p.eps > 0.0f ? 1.0f / sqrtf(k2 + p.eps) : 1.0f, bk = rk * beta;
    sv[w][0][lane] = rk;
    sv[w][1][lane] = bk;
    {
        float* tok = p.co + id * (kGdrTokAll * 64) + lane;
        const float e = __builtin_amdgcn_exp2f((float)G), a3 = __builtin_amdgcn_exp2f((float)(Gl - G)), a1 = e * rk;
        tok[tA1 * 64] = a1;
        tok[tA2 * 64] = e;
        tok[tA3 * 64] = a3 * bk;
        tok[tA3b * 64] = a3 * rk;
        tok[tBeta * 64] = beta;
        tok[tRk * 64] = rk;
        tok[tBk * 64] = bk;
        const bool clean = __all(a1 != 0.0f && e != 0.0f);
        const float grow = p.eps > 0.0f ? beta : beta * k2;
        const bool tame = __all(grow >= 0.0f && grow <= 2.0f), any_cut = __any(cut);
        const bool wrong = !__all(fabsf(k2) < __builtin_inff() && fabsf(beta) < __builtin_inff() && fabsf((float)G) < __builtin_inff());
        tok[tMisc * 64] = lane == 0 ? __builtin_amdgcn_exp2f((float)Gl) : lane == 2 ? (float)Gl : (lane == 1 ? clean : lane == 3 ? tame : lane == 4 ? any_cut : wrong) ? 1.0f : 0.0f;
        *reinterpret_cast<double*>(p.co + id * (kGdrTokAll * 64) + tG * 64 + 2 * lane) = G;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // N, row by row
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        double gi[4];
        const gf4 ri = *reinterpret_cast<const gf4*>(&sv[w][0][16 * i + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) gi[r] = sg[w][16 * i + 4 * g + r];
#pragma unroll
        for (int j = 0; j <= i; ++j) {
            const double gj = sg[w][16 * j + m];
            const float bj = sv[w][1][16 * j + m];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * g + r, col = 16 * j + m;
                const float d = row > col ? __builtin_amdgcn_exp2f((float)(gi[r] - gj)) : 0.0f;
                // a decay to nothing leaves out what it multiplies, whatever it is
                mat[row * LD + col] = d != 0.0f ? kk[i * (i + 1) / 2 + j][r] * d * ri[r] * bj : 0.0f;
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // operands of the blocks below the diagonal, then the diagonal's inverses: lanes of group g have block g
    gf4 nb[6];
#pragma unroll
    for (int i = 1; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < i; ++j) nb[i * (i - 1) / 2 + j] = *reinterpret_cast<const gf4*>(&mat[(16 * i + m) * LD + 16 * j + 4 * g]);
    {
        float x[16];
        float* blk = mat + 16 * g * LD + 16 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == m ? 1.0f : 0.0f;
#pragma unroll
            for (int l = 0; l < i; ++l) s = __builtin_fmaf(-blk[i * LD + l], x[l], s);
            x[i] = s;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < 16; ++i) blk[i * LD + m] = x[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    gf4 ti[4], tb[10];                                // -T_ii's rows; T's tiles as results lie
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ti[i] = -*reinterpret_cast<const gf4*>(&mat[(16 * i + m) * LD + 16 * i + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) tb[i * (i + 1) / 2 + i][r] = mat[(16 * i + 4 * g + r) * LD + 16 * i + m];
    }
#pragma unroll
    for (int lev = 1; lev < 4; ++lev)
#pragma unroll
        for (int j = 0; j + lev < 4; ++j) {
            const int i = j + lev;
            gf4 acc = {0, 0, 0, 0}, out = {0, 0, 0, 0};
#pragma unroll
            for (int l = j; l < i; ++l)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(nb[i * (i - 1) / 2 + l][r], tb[l * (l + 1) / 2 + j][r], acc, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) out = __builtin_amdgcn_mfma_f32_16x16x4f32(ti[i][r], acc[r], out, 0, 0, 0);
            tb[i * (i + 1) / 2 + j] = out;
        }
    constexpr int TP = BACK ? kGdrTri : kGdrLow;
    T* out = reinterpret_cast<T*>(p.wT) + id * (M::NT * TP);
    auto put = [&](int at, gf4 a, gf4 c) {
        if constexpr (sizeof(T) == 2) {
            const auto sp = M::template split<M::NT>(gdr_pair(a, c));
#pragma unroll
            for (int k = 0; k < M::NT; ++k) *reinterpret_cast<gb8*>(out + k * TP + at + lane * 8) = sp.t[k];
        } else {
            *reinterpret_cast<gf4*>(out + at + lane * 4) = a;
            *reinterpret_cast<gf4*>(out + at + (64 + lane) * 4) = c;
        }
    };
    if constexpr (BACK) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = j >> 1; s < 2; ++s) {
                const int i = 2 * s;                  // row tiles i and i + 1 are the terms
                put(gdr_up(j, s) * 512, i >= j ? tb[i * (i + 1) / 2 + j] : gf4{0, 0, 0, 0}, tb[(i + 1) * (i + 2) / 2 + j]);
            }
    } else {
        // through LDS, rows by lane
#pragma unroll
        for (int i = 1; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < i; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) mat[(16 * i + 4 * g + r) * LD + 16 * j + m] = tb[i * (i + 1) / 2 + j][r];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s <= i >> 1; ++s) {
                const gf4 a = *reinterpret_cast<const gf4*>(&mat[(16 * i + m) * LD + 32 * s + 4 * g]);
                if (!gdr_half(i, s)) {
                    put(gdr_low(i, s), a, *reinterpret_cast<const gf4*>(&mat[(16 * i + m) * LD + 32 * s + 16 + 4 * g]));
                } else if constexpr (sizeof(T) == 2) {
                    const auto sp = M::template split<M::NT>(gdr_pair(a, gf4{0, 0, 0, 0}));
#pragma unroll
                    for (int k = 0; k < M::NT; ++k) {
                        typedef uint32_t gu2 __attribute__((ext_vector_type(2)));
                        const gu4 u = __builtin_bit_cast(gu4, sp.t[k]);
                        *reinterpret_cast<gu2*>(out + k * TP + gdr_low(i, s) + lane * 4) = gu2{u[0], u[1]};
                    }
                } else {
                    *reinterpret_cast<gf4*>(out + gdr_low(i, s) + lane * 4) = a;
                }
            }
    }
}

// ---------------------------------------------------------------------------
// A wave's 16 columns of a state, or of its gradient, in registers.
template <int ROWS>
struct GdrState {
    static constexpr int ND = ROWS / 16;
    const LaunchGdr& p;
    int lane, w, g, m, col;
    bool in;
    gf4 S[ND];
    __device__ __forceinline__ GdrState(const LaunchGdr& a, int col_)
        : p(a), lane(threadIdx.x & 63), w(gdr_wave()), g(lane >> 4), m(lane & 15), col(col_), in(col_ < a.dv) {}

    // this wave's columns of a state [dk, n]; zeros where there is none
    __device__ __forceinline__ void load_state(const float* from, int n) {
        const GdrBuf<float> buf(from, from ? (unsigned)(p.dk * n) * 4 : 0);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + r;
                S[d][r] = buf.ld(in ? (unsigned)(row * n + col) * 4 : kGdrOut, 0);
            }
    }
    __device__ __forceinline__ void store_state(float* to, int n) const {
        int g = this->g, col = this->col;
        asm volatile("" : "+v"(g), "+v"(col));
        if (in)
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + r;
                    if (row < p.dk) to[row * n + col] = S[d][r];
                }
    }
    // Whether this wave's columns are those of the state at `with`: within 2^-16 of the largest of a column, or the smallest
    // normal number. Not for NaN and infinities. (Two ways through a segment without decay differ by up to 2^-20, by the
    // roundings of both; with that as the bound 65536 tokens of 4 heads took 3.3 ms, with this 0.82.)
    __device__ __forceinline__ bool agrees(const float* with) const {
        const GdrBuf<float> buf(with, (unsigned)(p.dk * p.dv) * 4);
        int g = this->g, col = this->col;             // places are made here, not kept from where the state was loaded
        asm volatile("" : "+v"(g), "+v"(col));
        float most = 0.0f, off = 0.0f;
        bool same = true;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 32 * (d >> 1) + 8 * g + 4 * (d & 1) + r;
                const float by = fabsf(S[d][r] - buf.ld(in ? (unsigned)(row * p.dv + col) * 4 : kGdrOut, 0));
                most = fmaxf(most, fabsf(S[d][r]));
                off = fmaxf(off, by);
                same &= by < __builtin_inff();
            }
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) {
            most = fmaxf(most, __shfl_xor(most, o, 64));
            off = fmaxf(off, __shfl_xor(off, o, 64));
        }
        return __all(!in || (same && off <= fmaxf(most * 0x1p-16f, 0x1p-126f)));
    }
};

// ---------------------------------------------------------------------------
// From chunk to chunk: a workgroup holds 64 columns of one head's state, a wave 16 of them, in
// registers. What all waves need lies in LDS: keys twice (the next chunk's come while this one's are in
// use), queries, T and the tokens' factors once, loaded again as soon as the last wave has used them; P is
// made here, two or three tiles a wave, since reading it back would cost as much as T. Two workgroups a CU
// in bf16 (registers and LDS hold no third). 131072 tokens of 16 heads of 128 x 128 in bf16: 1.1 ms, a chunk 16,100 cycles
// for two workgroups and 13,700 for one alone on its CU: what bounds it is a chunk's chain (read, multiply, solve,
// multiply; 236 matrix instructions a wave). With checkpoints it writes more
// than it reads: 8 x 2048 tokens of 40 heads 600 us, 3.1 TB/s (640 workgroups for 512 places: about a quarter of it).
template <typename T, int DKP, bool TWO, bool AL>
struct GdrWalk : GdrState<DKP> {
    using M = Mx<T>;
    using B = GdrState<DKP>;
    using B::p; using B::lane; using B::w; using B::g; using B::m; using B::col; using B::in; using B::S;
    static constexpr int KD = DKP / 32, ND = DKP / 16, TP = kGdrLow;
    static constexpr bool kTwo = TWO;
    GdrRows<T, KD, AL> rk, rq;
    T *tq, *tt, *tp;
    float *tok, *srq;
    int64_t b, bh, nc;
    int h, place;
    bool from_v = true, wrong = false;                // wrong: something that was not finite came by
    const T* vb;
    T* yb;
    T v[16];                                          // the next values as they came, no use of them before they are needed

    __device__ __forceinline__ GdrWalk(const LaunchGdr& a, T* q_, T* t_, T* p_, float* tok_, float* srq_, int64_t b_, int64_t bh_, int h_,
                                       int hk, int col_)
        : B(a, col_), rk(a.k, b_, hk, a.dk), rq(a.q, b_, hk, a.dk), tq(q_), tt(t_), tp(p_), tok(tok_), srq(srq_), b(b_), bh(bh_),
          nc(a.nchunks), h(h_), place(gdr_place(g, m)), vb(static_cast<const T*>(a.v.p) + b_ * a.v.batch_stride + h_ * a.v.head_stride),
          yb(static_cast<T*>(a.y) + (b_ * a.L * a.H + h_) * a.dv) {}

    template <bool OUT>
    __device__ __forceinline__ void rest(int64_t n) const {       // queries, T, factors of chunk n
        if (OUT) rq.load(tq, n * kGdrC, p.L);
        const int64_t id = bh * nc + n;
        const GdrSource from(reinterpret_cast<T*>(p.wT) + id * (M::NT * TP)), tokens(p.co + id * (kGdrTokAll * 64));
        constexpr int U = M::NT * TP * (int)sizeof(T) / 1024;
#pragma unroll
        for (int e = 0; e < (U + 3) / 4; ++e) {
            const int u = e * 4 + w;
            if (u < U) from.to_lds(reinterpret_cast<gu4*>(tt + u * (1024 / sizeof(T))), lane * 16, u * 1024);
        }
        if (w * 64 + lane < kGdrTok * 16) tokens.to_lds(reinterpret_cast<gu4*>(tok + w * 256), lane * 16, w * 1024);
    }
    // (rows past the last token: zeros, or copies of it as the keys'; their beta is 0)
    __device__ __forceinline__ void values(int64_t n) {
        const int64_t t0 = n * kGdrC;
        const T* at = vb + t0 * p.v.token_stride;
        const int c = in ? col : p.dv - 1, last = p.L - t0 < kGdrC ? (int)(p.L - t0) - 1 : kGdrC - 1;
        if constexpr (AL) {
            unsigned row = (unsigned)p.v.token_stride * (unsigned)sizeof(T);
            asm volatile("" : "+s"(row));
            const GdrBuf<T> buf(at, last * row + p.dv * (unsigned)sizeof(T));
            const unsigned lo = 4 * g * row + c * (unsigned)sizeof(T);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = buf.ld(lo + (i & 3) * row, 16 * (i >> 2) <= last ? 16 * (i >> 2) * row : 0);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = 16 * (i >> 2) + 4 * g + (i & 3), u = t < last ? t : last;
                v[i] = at[u * p.v.token_stride + c];
            }
        }
    }

    // one chunk; keys in `tk`, the next chunk's on their way to `tn`. OUT: with outputs, else the state alone
    template <bool OUT>
    __device__ __forceinline__ void chunk(int64_t n, int64_t end_n, T* tk, T* tn) {
        // places in LDS are made again for every chunk: kept over the loop they would spill
        int lane = this->lane;
        asm volatile("" : "+v"(lane));
        const int g = lane >> 4, m = lane & 15, place = gdr_place(g, m);
        const int64_t t0 = n * kGdrC;
        gdr_arrived();
        if (TWO && n + 1 < end_n) rk.load(tn, t0 + kGdrC, p.L);
        if (OUT && p.ckpt) {
            unsigned dvb = p.dv * 4;
            asm volatile("" : "+s"(dvb));             // offsets made where they are used, not kept over the loop
            const GdrBuf<float> ck(p.ckpt + (bh * nc + n) * p.dk * p.dv, p.dk * dvb);
            const unsigned lo = in ? 8 * g * dvb + col * 4 : kGdrOut;
#pragma unroll
            for (int s = 0; s < KD; ++s) {
                if (32 * s >= p.dk) break;            // (aligned rows: dk is a multiple of 8, whole eights are there or not)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (AL) ck.st(S[2 * s + (e >> 2)][e & 3], lo, (32 * s + e) * dvb);
                    else ck.st(S[2 * s + (e >> 2)][e & 3], lo + (32 * s + e) * dvb, 0);
                }
            }
        }
        // K S0; Q S0 transposed (a lane has a token's row), which is how it is stored; P's row tile of this wave, transposed
        // too, without the queries' lengths; and these lengths, a diagonal. The next fragments are read ahead of
        // the products of these.
        gf4 ks[4] = {}, qs[4] = {}, pt[4] = {}, len = {0, 0, 0, 0};
        {
            typename M::F f[2][8];
            auto read = [&](int s, typename M::F (&x)[8]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = gdr_rows_frag<T>(tk, i * KD + s, place);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (OUT) x[4 + i] = gdr_rows_frag<T>(tq, i * KD + s, place);
            };
            read(0, f[0]);
#pragma unroll
            for (int s = 0; s < KD; ++s) {
                typename M::F own;
                if (OUT) own = gdr_rows_frag<T>(tq, w * KD + s, place);
                if (s + 1 < KD) read(s + 1, f[(s + 1) & 1]);
                __builtin_amdgcn_sched_barrier(0);
                auto& x = f[s & 1];
                const auto sb = M::template split<3>(gdr_pair(S[2 * s], S[2 * s + 1]));
                if (OUT) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) pt[i] = M::mm(x[i], own, pt[i]);
                    len = M::mm(own, own, len);
                }
#pragma unroll
                for (int k = sizeof(T) == 2 ? 2 : 0; k >= 0; --k) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) ks[i] = M::mm(x[i], sb.t[k], ks[i]);
                    if (OUT)
#pragma unroll
                        for (int i = 0; i < 4; ++i) qs[i] = M::mm(sb.t[k], x[4 + i], qs[i]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (OUT) {
            const double* G = reinterpret_cast<const double*>(tok + tG * 64);
            const double gi = G[16 * w + m];
            int tile = w;
            asm volatile("" : "+s"(tile));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i > w) break;
                const gf4 bk = *reinterpret_cast<const gf4*>(&tok[tBk * 64 + 16 * i + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = __builtin_amdgcn_exp2f((float)(gi - G[16 * i + 4 * g + r]));
                    pt[i][r] = d != 0.0f && (i < w || m >= 4 * g + r) ? pt[i][r] * d * bk[r] : 0.0f;
                }
                const bool half = gdr_half(tile, i >> 1);
                T* at = tp + gdr_low(tile, i >> 1);
                if constexpr (sizeof(T) == 2) {
                    const auto both = M::template split<M::NT>(gdr_pair(pt[i], gf4{0, 0, 0, 0}));
                    at += half ? lane * 4 : lane * 8 + 4 * (i & 1);
#pragma unroll
                    for (int k = 0; k < M::NT; ++k) {
                        typedef uint32_t gu2 __attribute__((ext_vector_type(2)));
                        const gu4 u = __builtin_bit_cast(gu4, both.t[k]);
                        *reinterpret_cast<gu2*>(at + k * TP) = gu2{u[0], u[1]};
                    }
                } else {
                    *reinterpret_cast<gf4*>(at + ((i & 1) * 64 + lane) * 4) = pt[i];
                }
            }
            const float q2 = (m & 3) == 0 ? len[0] : (m & 3) == 1 ? len[1] : (m & 3) == 2 ? len[2] : len[3];
            if (m >> 2 == g) srq[16 * w + m] = p.eps > 0.0f ? p.scale * __builtin_amdgcn_rsqf(q2 + p.eps) : p.scale;
        }
        // V - e^G K S0; where a decay is nothing it leaves out what it multiplies
        const float end = tok[tMisc * 64];
        const bool clean = tok[tMisc * 64 + 1] != 0.0f;
        gf4 a3[4], V[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const gf4 a1 = *reinterpret_cast<const gf4*>(&tok[tA1 * 64 + 16 * i + 4 * g]);
            const float a2 = tok[tA2 * 64 + 16 * i + m];
            a3[i] = *reinterpret_cast<const gf4*>(&tok[tA3 * 64 + 16 * i + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) V[i][r] = IO<T>::cvt(v[4 * i + r]);
            if (clean) {
                V[i] -= a1 * ks[i];
                if (OUT) qs[i] *= a2;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    V[i][r] -= a1[r] != 0.0f ? a1[r] * ks[i][r] : 0.0f;
                    if (OUT) qs[i][r] = a2 != 0.0f ? a2 * qs[i][r] : 0.0f;
                }
            }
        }
        gf4 X[4] = {};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            typename M::template S<M::NT> tf[4];
#pragma unroll
            for (int i = 2 * s; i < 4; ++i) tf[i] = gdr_low_terms(tt, i, s, lane);
            const auto rb = M::template split<M::NT>(gdr_pair(V[2 * s], V[2 * s + 1]));
            M::template each<M::NT>([&](int a, int c) {
#pragma unroll
                for (int i = 2 * s; i < 4; ++i) X[i] = M::mm(tf[i].t[a], rb.t[c], X[i]);
            });
        }
        if (OUT) {
            // zeros above the diagonals do not keep what is not finite from other tokens, in front of it and behind a reset
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += (X[i][0] + X[i][1]) + (X[i][2] + X[i][3]);
            wrong |= tok[tMisc * 64 + 5] != 0.0f || !__all(fabsf(sum) < __builtin_inff());
        }
        __syncthreads();                              // P is there; queries, T and factors are used up
        if (n + 1 < end_n) {
            rest<OUT>(n + 1);
            if (from_v) values(n + 1);
        }
        if constexpr (OUT) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);        // the second half's operands are not read over the first's
            const auto xb = M::template split<M::NT>(gdr_pair(X[2 * s], X[2 * s + 1]));
            typename M::template S<M::NT> pf[4];
#pragma unroll
            for (int i = 2 * s; i < 4; ++i) pf[i] = gdr_low_terms(tp, i, s, lane);
            M::template each<M::NT>([&](int a, int c) {
#pragma unroll
                for (int i = 2 * s; i < 4; ++i) qs[i] = M::mm(xb.t[a], pf[i].t[c], qs[i]);
            });
        }
        {
            const int left = p.L - t0 < kGdrC ? (int)(p.L - t0) : kGdrC;
            unsigned row = (unsigned)(p.H * p.dv);
            asm volatile("" : "+s"(row));
            const unsigned size = (left - 1) * row + p.dv;
            const GdrBuf<T> yt(yb + t0 * row, size * (unsigned)sizeof(T));
            const int c0 = col - m + 4 * g;
            const unsigned lo = (m * row + c0) * (unsigned)sizeof(T);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (16 * i >= left) break;
                qs[i] *= srq[16 * i + m];
                if (p.vec_y) {
                    yt.st4(qs[i], c0 < p.dv ? lo : kGdrOut, 16 * i * row * (unsigned)sizeof(T));
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) yt.st(qs[i][r], c0 + r < p.dv ? lo + r * (unsigned)sizeof(T) : kGdrOut, 16 * i * row * (unsigned)sizeof(T));
                }
            }
            if (p.ckpt) {
                const GdrBuf<float> xt(p.ckptX + ((b * p.L + t0) * p.H + h) * p.dv, size * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (16 * i >= left) break;
#pragma unroll
                    for (int r = 0; r < 4; ++r) xt.st(X[i][r], in ? ((4 * g + r) * row + col) * 4 : kGdrOut, 16 * i * row * 4);
                }
            }
        }
        }
        // the next state
        {
            constexpr int NB = 2 * ND / 4;            // batches of four tiles, tokens' first half, then the second
            typename M::F f[2][4];
            auto read = [&](int q, typename M::F (&x)[4]) {
#pragma unroll
                for (int d = 0; d < 4; ++d) x[d] = gdr_frag_t<T, KD>(tk, q / (ND / 4), q % (ND / 4) * 2 + (d >> 1), d & 1, lane);
            };
            read(0, f[0]);
#pragma unroll
            for (int d = 0; d < ND; ++d) S[d] = end != 0.0f ? S[d] * end : gf4{0, 0, 0, 0};
            typename M::template S<3> xb;
#pragma unroll
            for (int q = 0; q < NB; ++q) {
                const int s = q / (ND / 4), d0 = q % (ND / 4) * 4;
                if (q + 1 < NB) read(q + 1, f[(q + 1) & 1]);
                if (d0 == 0) xb = M::template split<3>(gdr_pair(X[2 * s] * a3[2 * s], X[2 * s + 1] * a3[2 * s + 1]));
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = sizeof(T) == 2 ? 2 : 0; k >= 0; --k)
#pragma unroll
                    for (int d = 0; d < 4; ++d) S[d0 + d] = M::mm(f[q & 1][d], xb.t[k], S[d0 + d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (!TWO && n + 1 < end_n) {
            __syncthreads();
            rk.load(tk, t0 + kGdrC, p.L);
        }
    }
};

// This wave's columns token after token, from the state at `init` to k.S: where a value is not finite, so that it reaches what
// the formulas say and nothing else. 128 x 128: 2.5 to 3.5 us a token.
template <typename T, typename W>
__device__ __forceinline__ void gdr_tokens(W& k, const float* init) {
    const LaunchGdr& p = k.p;
    const int64_t kv = (int64_t)p.dk * p.dv;
    const int c = k.in ? k.col : p.dv - 1;
    k.load_state(init, p.dv);
    auto sum = [](float v) {
        v += __shfl_xor(v, 16, 64);
        return v + __shfl_xor(v, 32, 64);
    };
#pragma unroll 1
    for (int64_t t = 0; t < p.L; ++t) {
        if (p.ckpt && t % kGdrC == 0) k.store_state(p.ckpt + (k.bh * k.nc + t / kGdrC) * kv, p.dv);
        const int64_t at = (k.b * p.L + t) * p.H + k.h;
        const float beta = p.beta[at], decay = p.reset && p.reset[k.b * p.L + t] ? 0.0f : expf(p.g[at]);
        const T *kr = k.rk.base + t * k.rk.stride, *qr = k.rq.base + t * k.rq.stride;
        gf4 kt[W::ND], qt[W::ND];
        float k2 = 0.0f, q2 = 0.0f, sk = 0.0f, sq = 0.0f;
#pragma unroll
        for (int d = 0; d < W::ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 32 * (d >> 1) + 8 * k.g + 4 * (d & 1) + r, some = row < p.dk ? row : 0;
                const float kx = gdr_f<T>(kr[some]), qx = gdr_f<T>(qr[some]);
                kt[d][r] = row < p.dk ? kx : 0.0f;
                qt[d][r] = row < p.dk ? qx : 0.0f;
                k.S[d][r] = decay != 0.0f && row < p.dk ? k.S[d][r] * decay : 0.0f;
                k2 = __builtin_fmaf(kt[d][r], kt[d][r], k2);
                q2 = __builtin_fmaf(qt[d][r], qt[d][r], q2);
                sk = __builtin_fmaf(k.S[d][r], kt[d][r], sk);
            }
        const float rk = p.eps > 0.0f ? 1.0f / sqrtf(sum(k2) + p.eps) : 1.0f, rq = p.eps > 0.0f ? 1.0f / sqrtf(sum(q2) + p.eps) : 1.0f;
        const float x = gdr_f<T>(k.vb[t * p.v.token_stride + c]) - rk * sum(sk), u = beta * x;
#pragma unroll
        for (int d = 0; d < W::ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (32 * (d >> 1) + 8 * k.g + 4 * (d & 1) + r < p.dk) {
                    k.S[d][r] = __builtin_fmaf(kt[d][r] * rk, u, k.S[d][r]);
                    sq = __builtin_fmaf(k.S[d][r], qt[d][r], sq);
                }
        const float y = p.scale * rq * sum(sq);
        if (k.g == 0 && k.in) {
            IO<T>::st(k.yb + t * p.H * p.dv + k.col, y);
            if (p.ckpt) p.ckptX[at * p.dv + k.col] = x;
        }
    }
}

// The chunks [n0, n1) of one head and 64 columns, from the state in k.S on.
template <bool OUT, typename W, typename T>
__device__ __forceinline__ void gdr_walk(W& k, int64_t n0, int64_t n1, T* k0, T* k1) {
    k.rk.load(k0, n0 * kGdrC, k.p.L);
    k.template rest<OUT>(n0);
    if (k.from_v) k.values(n0);
    if constexpr (W::kTwo) {
        for (int64_t n = n0; n < n1; n += 2) {
            k.template chunk<OUT>(n, n1, k0, k1);
            if (n + 1 < n1) k.template chunk<OUT>(n + 1, n1, k1, k0);
        }
    } else {
        for (int64_t n = n0; n < n1; ++n) k.template chunk<OUT>(n, n1, k0, k0);
    }
}

// Zeros where no load writes: LDS columns past dk, blocks above the diagonal of the backward's P.
template <int N, typename T>
__device__ __forceinline__ void gdr_clear(T* lds) {
    for (int e = threadIdx.x; e < N * (int)sizeof(T) / 16; e += 256) reinterpret_cast<gu4*>(lds)[e] = gu4{0, 0, 0, 0};
}

template <typename T, int DKP, bool TWO, bool AL, int GROUPS>
__global__ void __launch_bounds__(256, GROUPS)
k_gdr_walk(const LaunchGdr p) {
    using W = GdrWalk<T, DKP, TWO, AL>;
    __shared__ alignas(16) T k0[64 * DKP], k1[TWO ? 64 * DKP : 8], tq[64 * DKP], tt[Mx<T>::NT * kGdrLow], tp[Mx<T>::NT * kGdrLow];
    __shared__ alignas(16) float tok[kGdrTok * 64], srq[64];
    const int64_t BH = p.B * p.H, rest = blockIdx.x / BH, bh = blockIdx.x % BH, b = bh / p.H, nc = p.nchunks;
    const int tiles = (p.dv + 63) / 64, seg = (int)(rest / tiles);
    const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk), col = (int)(rest % tiles) * 64 + gdr_wave() * 16 + (threadIdx.x & 15);
    W k(p, tq, tt, tp, tok, srq, b, bh, h, hk, col);
    const int64_t kv = (int64_t)p.dk * p.dv, n0 = seg * p.seg, n1 = n0 + p.seg < nc ? n0 + p.seg : nc;
    // several segments: never the caller's state, which the last of them overwrites whenever it gets there
    const float* from = p.state ? p.state + bh * kv : nullptr;
    if (p.nseg > 1) from = seg || p.state ? p.wE + (seg * BH + bh) * kv : nullptr;
    k.load_state(from, p.dv);
    if (p.dk < DKP) {
        gdr_clear<64 * DKP>(k0);
        gdr_clear<64 * DKP>(tq);
        if (TWO) gdr_clear<64 * DKP>(k1);
    }
    __syncthreads();
    gdr_walk<true>(k, n0, n1, k0, k1);
    if (p.nseg == 1 && k.wrong) gdr_tokens<T>(k, from);
    if (p.state && n1 == nc) k.store_state(p.state + bh * kv, p.dv);
    if (p.nseg > 1) {
        const int64_t next = (seg + 1) * BH + bh;
        const bool same = n1 == nc || k.agrees(p.wE + next * kv);
        if (!same) k.store_state(p.wX + (next - BH) * kv, p.dv);
        if ((threadIdx.x & 63) == 0) p.wQ[((bh * tiles + rest % tiles) * p.nseg + seg) * 4 + k.w] = (same ? 0 : 1) + (k.wrong ? 2 : 0);
    }
}

// How many of the chunks [n0, n1), from its end backwards or (AHEAD) from its start on, it takes until they leave less than
// 2^-48 of a state that passes them; all if they never do, `gone` says whether they do. Where no beta |k|^2 is outside
// [0, 2] no state, and no gradient of one, grows on the way but by what is added to it, so that behind those chunks nothing in
// front of them is left but 2^-48 of its own size. That is nothing beside a state of that size; whether it is nothing beside
// what the segment makes is seen when the walk gets to its end (k_gdr_again). A chunk with a decay of 0 leaves
// nothing, whatever its beta and theirs, of a state of NaN neither (which a map of zeros would not stop).
template <bool AHEAD>
__device__ __forceinline__ int64_t gdr_reach(const LaunchGdr& p, int64_t bh, int64_t n0, int64_t n1, bool& gone) {
    const int lane = threadIdx.x & 63;
    gone = false;
    float sum = 0.0f;
    bool shrinks = true;
    for (int64_t done = 0; done < n1 - n0; done += 64) {
        const int64_t at = done + lane;
        float g = 0.0f;
        bool tame = true, cut = false;
        if (at < n1 - n0) {
            const float* misc = p.co + (bh * p.nchunks + (AHEAD ? n0 + at : n1 - 1 - at)) * (kGdrTokAll * 64) + tMisc * 64;
            g = misc[2];
            tame = misc[3] != 0.0f;
            cut = misc[4] != 0.0f;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float u = __shfl_up(g, o, 64);
            if (lane >= o) g += u;
        }
        const uint64_t low = __ballot(at < n1 - n0 && sum + g < -48.0f), wild = __ballot(!tame), zero = __ballot(cut);
        const int bad = wild ? __builtin_ctzll(wild) : 64;
        int to = low && shrinks ? __builtin_ctzll(low) : 64;
        if (bad <= to) to = 64;
        if (zero && (int)__builtin_ctzll(zero) < to) to = __builtin_ctzll(zero);
        shrinks &= bad == 64;
        if (to < 64) {
            gone = true;
            return done + to + 1;
        }
        sum += __shfl(g, 63, 64);
    }
    return n1 - n0;
}

// A long sequence in few heads, cut into segments that run at the same time. First the state behind each segment, from
// nothing in front of it (or, the first, from the caller's) and from where it still matters on; and, as dk columns more that
// start as the identity and get no values, what the segment makes of the state in front of it, where anything is
// left of that. The caller's state is copied for the walk's first segment, as its last one overwrites it. k_gdr_join puts the
// ends together. (2048 tokens of 40 heads: 49 and 13 us, 75 for the walk of three segments. 131072 tokens of 16 heads: 266, 5 and
// 1166 us, or 1000 and 120 for ends and join where some heads decay so slowly that their segments let a state through; the
// whole call 1.5 to 2.5 ms, 10.6 in one segment.)
template <typename T, int DKP, bool TWO, bool AL, int GROUPS>
__global__ void __launch_bounds__(256, GROUPS)
k_gdr_ends(const LaunchGdr p) {
    using W = GdrWalk<T, DKP, TWO, AL>;
    __shared__ alignas(16) T k0[64 * DKP], k1[TWO ? 64 * DKP : 8], tt[Mx<T>::NT * kGdrLow];
    __shared__ alignas(16) float tok[kGdrTok * 64];
    const int64_t BH = p.B * p.H, rest = blockIdx.x / BH, bh = blockIdx.x % BH, b = bh / p.H, kv = (int64_t)p.dk * p.dv;
    const int tv = (p.dv + 63) / 64, tiles = tv + (p.dk + 63) / 64, seg = (int)(rest / tiles), tile = (int)(rest % tiles);
    const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk), wave = gdr_wave(), lane = threadIdx.x & 63;
    const bool map = tile >= tv;
    const int col = (map ? tile - tv : tile) * 64 + wave * 16 + (lane & 15);
    const int64_t n1 = (seg + 1) * p.seg;
    bool gone;
    const int64_t reach = gdr_reach<false>(p, bh, seg * p.seg, n1, gone);
    const int64_t n0 = n1 - __builtin_amdgcn_readfirstlane((int)reach);
    if (map) {
        if (seg == 0) return;
        if (tile == tv && threadIdx.x == 0) p.wF[seg * BH + bh] = gone ? 0.0f : 1.0f;
        if (gone) return;
    }
    W k(p, nullptr, tt, nullptr, tok, nullptr, b, bh, h, hk, col);
    if (map) {
        k.from_v = false;
        k.in = col < p.dk;
#pragma unroll
        for (int d = 0; d < W::ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) k.S[d][r] = 32 * (d >> 1) + 8 * k.g + 4 * (d & 1) + r == col ? 1.0f : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) k.v[i] = T(0);
    } else {
        const float* init = seg == 0 && p.state ? p.state + bh * kv : nullptr;
        k.load_state(init, p.dv);
        if (init) k.store_state(p.wE + bh * kv, p.dv);
        if (n0 > 0)
#pragma unroll
            for (int d = 0; d < W::ND; ++d) k.S[d] = gf4{0, 0, 0, 0};
    }
    if (p.dk < DKP) {
        gdr_clear<64 * DKP>(k0);
        if (TWO) gdr_clear<64 * DKP>(k1);
    }
    __syncthreads();
    gdr_walk<false>(k, n0, n1, k0, k1);
    if (map) k.store_state(p.wM + (seg * BH + bh) * (int64_t)p.dk * p.dk, p.dk);
    else k.store_state(p.wE + ((seg + 1) * BH + bh) * kv, p.dv);
}

// The states between segments, one after the other: E_s <- M_s E_(s-1) + E_s, where M_s is there. Waves as in the walk.
template <typename T, int DKP>
__global__ void __launch_bounds__(256)
k_gdr_join(const LaunchGdr p) {
    using M = Mx<T>;
    using W = GdrWalk<T, DKP, false, false>;
    const int64_t BH = p.B * p.H, bh = blockIdx.x % BH, kv = (int64_t)p.dk * p.dv;
    const int lane = threadIdx.x & 63, col = (int)(blockIdx.x / BH) * 64 + gdr_wave() * 16 + (lane & 15), g = lane >> 4, m = lane & 15;
    // nothing in front of any segment counts: its end is as it should be
    const int last = p.nseg - 2;
    bool any = false;
    for (int seg = 1 + lane; seg <= last; seg += 64) any |= p.wF[seg * BH + bh] != 0.0f;
    if (!__any(any)) return;
    W k(p, nullptr, nullptr, nullptr, nullptr, nullptr, 0, bh, 0, 0, col);
    const int64_t kk = (int64_t)p.dk * p.dk;
    // The map's rows of this lane, 32 columns of eight tiles ahead, the next segment's behind the last (256 rows in two halves: all
    // at once, twice, would be the registers there are).
    constexpr int HALVES = W::ND > 8 ? 2 : 1, NH = W::ND / HALVES, STEPS = W::KD * HALVES;
    gf8 x[2][NH];
    auto read = [&](int seg, int step, gf8 (&to)[NH]) {
        const int s = step / HALVES;
        const GdrBuf<float> map(p.wM + (seg * BH + bh) * kk, (unsigned)kk * 4);
#pragma unroll
        for (int e = 0; e < NH; ++e) {
            const int d = step % HALVES * NH + e, row = 32 * (d >> 1) + 8 * (m >> 2) + 4 * (d & 1) + (m & 3);
            to[e] = map.template ld8<false>((unsigned)(row * p.dk + 32 * s + 8 * g) * 4, 32 * s + 8 * g, p.dk);
        }
    };
    k.load_state(p.wE + (BH + bh) * kv, p.dv);
    read(1, 0, x[0]);
#pragma unroll 1
    for (int seg = 1; seg <= last; ++seg) {
        float* end = p.wE + ((seg + 1) * BH + bh) * kv;
        const bool on = p.wF[seg * BH + bh] != 0.0f;  // (without it the map is not written: what is made of it is dropped)
        const int next = seg < last ? seg + 1 : last;
        typename M::template S<M::NT> sb[W::KD];
#pragma unroll
        for (int s = 0; s < W::KD; ++s) sb[s] = M::template split<M::NT>(gdr_pair(k.S[2 * s], k.S[2 * s + 1]));
        k.load_state(end, p.dv);
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            read(q + 1 < STEPS ? seg : next, (q + 1) % STEPS, x[(q + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < NH; ++e) {
                gf4& S = k.S[q % HALVES * NH + e];
                S = M::mul(M::template split<M::NT>(x[q & 1][e]), sb[q / HALVES], S);
            }
        }
        if (on) k.store_state(end, p.dv);
        else k.load_state(end, p.dv);
    }
}

// Segments that did not start from what the one in front came to, once more from there, one after the other: where a segment's
// decays leave little of the state in front, but the segment makes less (values that end, states of very different sizes). And
// columns with anything that is not finite, token after token. Where there is none of them it takes 5 us.
template <typename T, int DKP, bool TWO, bool AL>
__global__ void __launch_bounds__(256, 1)
k_gdr_again(const LaunchGdr p) {
    using W = GdrWalk<T, DKP, TWO, AL>;
    __shared__ alignas(16) T k0[64 * DKP], k1[TWO ? 64 * DKP : 8], tq[64 * DKP], tt[Mx<T>::NT * kGdrLow], tp[Mx<T>::NT * kGdrLow];
    __shared__ alignas(16) float tok[kGdrTok * 64], srq[64];
    const int64_t BH = p.B * p.H, bh = blockIdx.x % BH, tile = blockIdx.x / BH, b = bh / p.H, nc = p.nchunks, kv = (int64_t)p.dk * p.dv;
    const int tiles = (p.dv + 63) / 64, h = (int)(bh % p.H), hk = h / (p.H / p.Hk), lane = threadIdx.x & 63;
    const uint32_t* off = p.wQ + (bh * tiles + tile) * p.nseg * 4;
    bool any = false, wrong = false;
    for (int i = lane; i < p.nseg * 4; i += 64) {
        any |= off[i] != 0;
        wrong |= i % 4 == gdr_wave() && off[i] >= 2;
    }
    if (!__any(any)) return;
    W k(p, tq, tt, tp, tok, srq, b, bh, h, hk, (int)tile * 64 + gdr_wave() * 16 + (lane & 15));
    k.wrong = __any(wrong);
    if (p.dk < DKP) {
        gdr_clear<64 * DKP>(k0);
        gdr_clear<64 * DKP>(tq);
        if (TWO) gdr_clear<64 * DKP>(k1);
    }
    bool here = false;                                // the state in front of the segment is in registers
    for (int seg = 1; seg < p.nseg; ++seg) {
        const float* from = p.wE + (seg * BH + bh) * kv;
        const bool own = !k.wrong && (here ? !k.agrees(from) : off[(seg - 1) * 4 + k.w] != 0);
        // (a barrier, too: the last segment's LDS is used up, the zeros are there)
        if (!__syncthreads_or(own)) {
            here = false;
            continue;
        }
        if (!here) k.load_state(own ? p.wX + ((seg - 1) * BH + bh) * kv : from, p.dv);
        const int64_t n0 = seg * p.seg, n1 = n0 + p.seg < nc ? n0 + p.seg : nc;
        gdr_walk<true>(k, n0, n1, k0, k1);
        here = true;
        if (p.state && n1 == nc) k.store_state(p.state + bh * kv, p.dv);
    }
    if (k.wrong) {
        gdr_tokens<T>(k, p.state ? p.wE + bh * kv : nullptr);
        if (p.state) k.store_state(p.state + bh * kv, p.dv);
    }
}

// ---------------------------------------------------------------------------
// The backward from chunk to chunk, the last first, with W the gradient of the state behind a chunk in
// registers as the forward has the state:
//   dX = (P beta)^T dY + beta e^(G_last - G) K W,  dV = T^T dX,
//   W' = e^G_last W + (scale e^G Q)^T dY - (e^G K)^T dV
// Keys and queries are needed to the end of a chunk and lie in LDS once, so that a CU holds two workgroups, of which
// one waits for its next chunk while the other works. A long sequence in few heads is cut into segments that run at the
// same time. k_gdr_ends_back first makes the gradient behind each of them from the chunks behind it, as far back as they
// count: all of them in the worst case, when the first segment takes as long as one workgroup did, on a card that
// is not full; what the walk comes to says whether that was far enough, and k_gdr_again_back repeats where it was not.
// 8 x 2048 tokens of 40 heads of 128 x 128 in bf16: 634 us, 2.9 TB/s, bound as the forward's; 3 x 1001 tokens of 6 heads of 96 x 129
// in fp32, with resets: 56 and 67 us (239 in one segment).
template <typename T, int DKP, bool AL>
struct GdrWalkBack : GdrState<DKP> {
    using M = Mx<T>;
    using B = GdrState<DKP>;
    using B::p; using B::lane; using B::w; using B::g; using B::m; using B::col; using B::in; using B::S;
    static constexpr int KD = DKP / 32, ND = DKP / 16, TP = kGdrTri;
    GdrRows<T, KD, AL> rk, rq;
    T *tk, *tq, *tt, *tp;
    float *tok, *srq;
    int64_t b, bh, nc;
    int h, place;
    bool wrong = false;                               // something that was not finite came by
    T v[16];                                          // the next gradients of y, as they came

    __device__ __forceinline__ GdrWalkBack(const LaunchGdr& a, T* k_, T* q_, T* t_, T* p_, float* tok_, float* srq_, int64_t b_, int64_t bh_,
                                           int h_, int hk, int col_)
        : B(a, col_), rk(a.k, b_, hk, a.dk), rq(a.q, b_, hk, a.dk), tk(k_), tq(q_), tt(t_), tp(p_), tok(tok_), srq(srq_), b(b_), bh(bh_),
          nc(a.nchunks), h(h_), place(gdr_place(g, m)) {}

    __device__ __forceinline__ void factors(int64_t n) const {    // T^T and the tokens' factors of chunk n
        const int64_t id = bh * nc + n;
        const GdrSource from(reinterpret_cast<T*>(p.wT) + id * (M::NT * TP)), tokens(p.co + id * (kGdrTokAll * 64));
        constexpr int U = M::NT * TP * (int)sizeof(T) / 1024;
#pragma unroll
        for (int e = 0; e < (U + 3) / 4; ++e) {
            const int u = e * 4 + w;
            if (u < U) from.to_lds(reinterpret_cast<gu4*>(tt + u * (1024 / sizeof(T))), lane * 16, u * 1024);
        }
        if (w * 64 + lane < kGdrTok * 16) tokens.to_lds(reinterpret_cast<gu4*>(tok + w * 256), lane * 16, w * 1024);
    }
    __device__ __forceinline__ void values(int64_t n) {
        const int64_t t0 = n * kGdrC;
        unsigned row = (unsigned)(p.H * p.dv) * (unsigned)sizeof(T);
        const int last = p.L - t0 < kGdrC ? (int)(p.L - t0) - 1 : kGdrC - 1;
        asm volatile("" : "+s"(row));
        const GdrBuf<T> buf(static_cast<const T*>(p.gr.dy) + ((b * p.L + t0) * p.H + h) * p.dv, last * row + p.dv * (unsigned)sizeof(T));
        const unsigned lo = in ? 4 * g * row + col * (unsigned)sizeof(T) : kGdrOut;
#pragma unroll
        for (int i = 0; i < 16; ++i) {                // none behind the last token
            const unsigned at = lo + (i & 3) * row;
            v[i] = buf.ld(16 * (i >> 2) <= last ? at : kGdrOut, 16 * (i >> 2) <= last ? 16 * (i >> 2) * row : 0);
        }
    }

    // one chunk. OUT: with gradients, else the state's alone
    template <bool OUT>
    __device__ __forceinline__ void chunk(int64_t n, int64_t first) {
        const int64_t t0 = n * kGdrC, id = bh * nc + n;
        gdr_arrived();
        if constexpr (OUT) {
            unsigned dvb = p.dv * 4;
            asm volatile("" : "+s"(dvb));
            const GdrBuf<float> ws(p.wS + id * p.dk * p.dv, p.dk * dvb);
            const unsigned lo = in ? 8 * g * dvb + col * 4 : kGdrOut;
#pragma unroll
            for (int s = 0; s < KD; ++s) {
                if (32 * s >= p.dk) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (AL) ws.st(S[2 * s + (e >> 2)][e & 3], lo, (32 * s + e) * dvb);
                    else ws.st(S[2 * s + (e >> 2)][e & 3], lo + (32 * s + e) * dvb, 0);
                }
            }
        }
        // K W, and P's row tile of this wave (a lane has a key's column) with its queries' lengths, a diagonal
        gf4 dX[4] = {}, pt[4] = {}, len = {0, 0, 0, 0};
        {
            typename M::F f[2][4];
            auto read = [&](int s, typename M::F (&x)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = gdr_rows_frag<T>(tk, i * KD + s, place);
            };
            read(0, f[0]);
#pragma unroll
            for (int s = 0; s < KD; ++s) {
                const auto own = gdr_rows_frag<T>(tq, w * KD + s, place);
                if (s + 1 < KD) read(s + 1, f[(s + 1) & 1]);
                __builtin_amdgcn_sched_barrier(0);
                auto& x = f[s & 1];
                const auto sb = M::template split<3>(gdr_pair(S[2 * s], S[2 * s + 1]));
#pragma unroll
                for (int i = 0; i < 4; ++i) pt[i] = M::mm(own, x[i], pt[i]);
                len = M::mm(own, own, len);
#pragma unroll
                for (int k = sizeof(T) == 2 ? 2 : 0; k >= 0; --k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dX[i] = M::mm(x[i], sb.t[k], dX[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        {
            const double* G = reinterpret_cast<const double*>(tok + tG * 64);
            gf4 q;
            double gi[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float q2 = __shfl(len[r], g * 16 + 4 * g + r, 64);
                q[r] = p.eps > 0.0f ? p.scale * __builtin_amdgcn_rsqf(q2 + p.eps) : p.scale;
                gi[r] = G[16 * w + 4 * g + r];
            }
            if (m == 0) *reinterpret_cast<gf4*>(&srq[16 * w + 4 * g]) = q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i > w) break;                     // this wave's tiles above the diagonal stay 0 in LDS
                const float bk = tok[tBk * 64 + 16 * i + m];
                const double gj = G[16 * i + m];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float d = __builtin_amdgcn_exp2f((float)(gi[r] - gj));
                    pt[i][r] = d != 0.0f && (i < w || 4 * g + r >= m) ? pt[i][r] * d * bk * q[r] : 0.0f;
                }
                const int unit = i < 2 ? 2 * i + (w >> 1) : i + 2;
                if constexpr (sizeof(T) == 2) {
                    const auto both = M::template split<M::NT>(gdr_pair(pt[i], gf4{0, 0, 0, 0}));
                    T* at = tp + (unit * 64 + lane) * 8 + 4 * (w & 1);
#pragma unroll
                    for (int k = 0; k < M::NT; ++k) {
                        typedef uint32_t gu2 __attribute__((ext_vector_type(2)));
                        const gu4 u = __builtin_bit_cast(gu4, both.t[k]);
                        *reinterpret_cast<gu2*>(at + k * TP) = gu2{u[0], u[1]};
                    }
                } else {
                    *reinterpret_cast<gf4*>(tp + ((unit * 2 + (w & 1)) * 64 + lane) * 4) = pt[i];
                }
            }
        }
        const float end = tok[tMisc * 64];
        const bool clean = tok[tMisc * 64 + 1] != 0.0f;
        gf4 a1[4], a2[4], dY[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const gf4 a3 = *reinterpret_cast<const gf4*>(&tok[tA3 * 64 + 16 * i + 4 * g]);
            a1[i] = *reinterpret_cast<const gf4*>(&tok[tA1 * 64 + 16 * i + 4 * g]);
            a2[i] = *reinterpret_cast<const gf4*>(&tok[tA2 * 64 + 16 * i + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dY[i][r] = IO<T>::cvt(v[4 * i + r]);
                dX[i][r] = a3[r] != 0.0f ? a3[r] * dX[i][r] : 0.0f;
            }
        }
        __syncthreads();                              // P and the queries' lengths are there
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const auto ob = M::template split<1>(gdr_pair(dY[2 * s], dY[2 * s + 1]));     // exact
            typename M::template S<M::NT> pf[4];
#pragma unroll
            for (int i = 0; i < 2 * s + 2; ++i) pf[i] = gdr_terms<T, M::NT>(tp, TP, gdr_up(i, s), lane);
#pragma unroll
            for (int k = M::NT - 1; k >= 0; --k)
#pragma unroll
                for (int i = 0; i < 2 * s + 2; ++i) dX[i] = M::mm(pf[i].t[k], ob.t[0], dX[i]);
        }
        gf4 dV[4] = {};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            typename M::template S<M::NT> tf[4];
#pragma unroll
            for (int i = 0; i < 2 * s + 2; ++i) tf[i] = gdr_terms<T, M::NT>(tt, TP, gdr_up(i, s), lane);
            const auto xb = M::template split<M::NT>(gdr_pair(dX[2 * s], dX[2 * s + 1]));
            M::template each<M::NT>([&](int a, int c) {
#pragma unroll
                for (int i = 0; i < 2 * s + 2; ++i) dV[i] = M::mm(tf[i].t[a], xb.t[c], dV[i]);
            });
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) a2[i] *= *reinterpret_cast<const gf4*>(&srq[16 * i + 4 * g]);
        if (OUT) {
            // as in the forward; and the state's gradient, which a beta of 0 would hide
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += (dV[i][0] + dV[i][1]) + (dV[i][2] + dV[i][3]);
#pragma unroll
            for (int d = 0; d < ND; ++d) sum += (S[d][0] + S[d][1]) + (S[d][2] + S[d][3]);
            wrong |= tok[tMisc * 64 + 5] != 0.0f || !__all(fabsf(sum) < __builtin_inff());
        }
        __syncthreads();                              // T, P and factors are used up
        if (n > first) {
            factors(n - 1);
            values(n - 1);
        }
        if constexpr (OUT) {
            unsigned row = (unsigned)(p.H * p.dv);
            asm volatile("" : "+s"(row));
            const int64_t at = ((b * p.L + t0) * p.H + h) * p.dv;
            const int left = p.L - t0 < kGdrC ? (int)(p.L - t0) : kGdrC;
            const unsigned size = (left - 1) * row + p.dv;
            const GdrBuf<T> dvt(static_cast<T*>(p.gr.dv) + at, size * (unsigned)sizeof(T));
            const GdrBuf<float> wvt(p.wV + at, size * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (16 * i >= left) break;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const unsigned lo = (4 * g + r) * row + col;
                    dvt.st(dV[i][r], in ? lo * (unsigned)sizeof(T) : kGdrOut, 16 * i * row * (unsigned)sizeof(T));
                    wvt.st(dV[i][r], in ? lo * 4 : kGdrOut, 16 * i * row * 4);
                }
            }
        }
        // the gradient of the state in front
        {
            constexpr int NB = 2 * ND / 2;            // batches of two tiles, tokens' first half, then the second
            typename M::F f[2][4];
            auto read = [&](int q, typename M::F (&x)[4]) {
                const int s = q / (ND / 2), sd = q % (ND / 2);
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    x[d] = gdr_frag_t<T, KD>(tk, s, sd, d, lane);
                    x[2 + d] = gdr_frag_t<T, KD>(tq, s, sd, d, lane);
                }
            };
            read(0, f[0]);
#pragma unroll
            for (int d = 0; d < ND; ++d) S[d] = end != 0.0f ? S[d] * end : gf4{0, 0, 0, 0};
            typename M::template S<3> ob, vb;
#pragma unroll
            for (int q = 0; q < NB; ++q) {
                const int s = q / (ND / 2), d0 = q % (ND / 2) * 2;
                if (q + 1 < NB) read(q + 1, f[(q + 1) & 1]);
                if (d0 == 0) {
                    gf4 o[2], x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        o[e] = dY[2 * s + e] * a2[2 * s + e];
                        x[e] = dV[2 * s + e] * -a1[2 * s + e];
                        if (!clean)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                o[e][r] = a2[2 * s + e][r] != 0.0f ? o[e][r] : 0.0f;
                                x[e][r] = a1[2 * s + e][r] != 0.0f ? x[e][r] : 0.0f;
                            }
                    }
                    ob = M::template split<3>(gdr_pair(o[0], o[1]));
                    vb = M::template split<3>(gdr_pair(x[0], x[1]));
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = sizeof(T) == 2 ? 2 : 0; k >= 0; --k) {
#pragma unroll
                    for (int d = 0; d < 2; ++d) S[d0 + d] = M::mm(f[q & 1][d], vb.t[k], S[d0 + d]);
#pragma unroll
                    for (int d = 0; d < 2; ++d) S[d0 + d] = M::mm(f[q & 1][2 + d], ob.t[k], S[d0 + d]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (n > first) {
            __syncthreads();
            rk.load(tk, t0 - kGdrC, p.L);
            rq.load(tq, t0 - kGdrC, p.L);
        }
    }
};

// The chunks [n0, n1), the last first, from the gradient in k.S on; LDS as gdr_clear_back leaves it.
template <bool OUT, typename W>
__device__ __forceinline__ void gdr_walk_back(W& k, int64_t n0, int64_t n1) {
    k.rk.load(k.tk, (n1 - 1) * kGdrC, k.p.L);
    k.rq.load(k.tq, (n1 - 1) * kGdrC, k.p.L);
    k.factors(n1 - 1);
    k.values(n1 - 1);
#pragma unroll 1
    for (int64_t n = n1 - 1; n >= n0; --n) k.template chunk<OUT>(n, n0);
}
template <typename T, int DKP>
__device__ __forceinline__ void gdr_clear_back(const LaunchGdr& p, T* tk, T* tq, T* tp) {
    if (p.dk < DKP) {
        gdr_clear<64 * DKP>(tk);
        gdr_clear<64 * DKP>(tq);
    }
    gdr_clear<Mx<T>::NT * kGdrTri>(tp);
    __syncthreads();
}

// As gdr_tokens, from the last token to the first.
template <typename T, typename W>
__device__ __forceinline__ void gdr_tokens_back(W& k) {
    const LaunchGdr& p = k.p;
    const int64_t kv = (int64_t)p.dk * p.dv;
    const int c = k.in ? k.col : p.dv - 1;
    k.load_state(p.gr.dstate_final ? p.gr.dstate_final + k.bh * kv : nullptr, p.dv);
    auto sum = [](float v) {
        v += __shfl_xor(v, 16, 64);
        return v + __shfl_xor(v, 32, 64);
    };
#pragma unroll 1
    for (int64_t t = p.L - 1; t >= 0; --t) {
        if (t == p.L - 1 || t % kGdrC == kGdrC - 1) k.store_state(p.wS + (k.bh * k.nc + t / kGdrC) * kv, p.dv);
        const int64_t at = (k.b * p.L + t) * p.H + k.h;
        const float beta = p.beta[at], decay = p.reset && p.reset[k.b * p.L + t] ? 0.0f : expf(p.g[at]);
        const T *kr = k.rk.base + t * k.rk.stride, *qr = k.rq.base + t * k.rq.stride;
        gf4 kt[W::ND], qt[W::ND];
        float k2 = 0.0f, q2 = 0.0f, wk = 0.0f;
#pragma unroll
        for (int d = 0; d < W::ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 32 * (d >> 1) + 8 * k.g + 4 * (d & 1) + r, some = row < p.dk ? row : 0;
                const float kx = gdr_f<T>(kr[some]), qx = gdr_f<T>(qr[some]);
                kt[d][r] = row < p.dk ? kx : 0.0f;
                qt[d][r] = row < p.dk ? qx : 0.0f;
                k2 = __builtin_fmaf(kt[d][r], kt[d][r], k2);
                q2 = __builtin_fmaf(qt[d][r], qt[d][r], q2);
            }
        const float rk = p.eps > 0.0f ? 1.0f / sqrtf(sum(k2) + p.eps) : 1.0f, rq = p.scale * (p.eps > 0.0f ? 1.0f / sqrtf(sum(q2) + p.eps) : 1.0f);
        const float dy = gdr_f<T>(static_cast<const T*>(p.gr.dy)[at * p.dv + c]);
#pragma unroll
        for (int d = 0; d < W::ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (32 * (d >> 1) + 8 * k.g + 4 * (d & 1) + r < p.dk) {
                    k.S[d][r] = __builtin_fmaf(qt[d][r] * rq, dy, k.S[d][r]);
                    wk = __builtin_fmaf(k.S[d][r], kt[d][r], wk);
                }
        const float dv = beta * rk * sum(wk);
#pragma unroll
        for (int d = 0; d < W::ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool row = 32 * (d >> 1) + 8 * k.g + 4 * (d & 1) + r < p.dk;
                k.S[d][r] = decay != 0.0f && row ? __builtin_fmaf(kt[d][r] * -rk, dv, k.S[d][r]) * decay : 0.0f;
            }
        if (k.g == 0 && k.in) {
            IO<T>::st(static_cast<T*>(p.gr.dv) + at * p.dv + k.col, dv);
            p.wV[at * p.dv + k.col] = dv;
        }
    }
}

// Several segments: the gradient of the state behind each but the last.
template <typename T, int DKP, bool AL, int GROUPS>
__global__ void __launch_bounds__(256, GROUPS)
k_gdr_ends_back(const LaunchGdr p) {
    using W = GdrWalkBack<T, DKP, AL>;
    __shared__ alignas(16) T tk[64 * DKP], tq[64 * DKP], tt[Mx<T>::NT * kGdrTri], tp[Mx<T>::NT * kGdrTri];
    __shared__ alignas(16) float tok[kGdrTok * 64], srq[64];
    const int64_t BH = p.B * p.H, rest = blockIdx.x / BH, bh = blockIdx.x % BH, b = bh / p.H, kv = (int64_t)p.dk * p.dv;
    const int tiles = (p.dv + 63) / 64, seg = (int)(rest / tiles);
    const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk), col = (int)(rest % tiles) * 64 + gdr_wave() * 16 + (threadIdx.x & 15);
    const int64_t n1 = (seg + 1) * p.seg;
    bool gone;
    const int64_t reach = gdr_reach<true>(p, bh, n1, p.nchunks, gone);
    const int64_t from_n = n1 + __builtin_amdgcn_readfirstlane((int)reach);
    W k(p, tk, tq, tt, tp, tok, srq, b, bh, h, hk, col);
    k.load_state(p.gr.dstate_final && !gone ? p.gr.dstate_final + bh * kv : nullptr, p.dv);
    gdr_clear_back<T, DKP>(p, tk, tq, tp);
    gdr_walk_back<false>(k, n1, from_n);
    k.store_state(p.wE + (seg * BH + bh) * kv, p.dv);
}

template <typename T, int DKP, bool AL, int GROUPS>
__global__ void __launch_bounds__(256, GROUPS)
k_gdr_walk_back(const LaunchGdr p) {
    using W = GdrWalkBack<T, DKP, AL>;
    __shared__ alignas(16) T tk[64 * DKP], tq[64 * DKP], tt[Mx<T>::NT * kGdrTri], tp[Mx<T>::NT * kGdrTri];
    __shared__ alignas(16) float tok[kGdrTok * 64], srq[64];
    const int64_t BH = p.B * p.H, rest = blockIdx.x / BH, bh = blockIdx.x % BH, b = bh / p.H, kv = (int64_t)p.dk * p.dv;
    const int tiles = (p.dv + 63) / 64, seg = (int)(rest / tiles);
    const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk), col = (int)(rest % tiles) * 64 + gdr_wave() * 16 + (threadIdx.x & 15);
    const int64_t n0 = seg * p.seg, n1 = n0 + p.seg < p.nchunks ? n0 + p.seg : p.nchunks;
    W k(p, tk, tq, tt, tp, tok, srq, b, bh, h, hk, col);
    k.load_state(seg < p.nseg - 1 ? p.wE + (seg * BH + bh) * kv : p.gr.dstate_final ? p.gr.dstate_final + bh * kv : nullptr, p.dv);
    gdr_clear_back<T, DKP>(p, tk, tq, tp);
    gdr_walk_back<true>(k, n0, n1);
    if (p.nseg == 1 && k.wrong) gdr_tokens_back<T>(k);
    if (seg == 0 && p.gr.dstate_init) k.store_state(p.gr.dstate_init + bh * kv, p.dv);
    if (p.nseg > 1) {
        const int64_t in_front = (seg - 1) * BH + bh;
        const bool same = seg == 0 || k.agrees(p.wE + in_front * kv);
        if (!same) k.store_state(p.wX + in_front * kv, p.dv);
        if ((threadIdx.x & 63) == 0) p.wQ[((bh * tiles + rest % tiles) * p.nseg + seg) * 4 + k.w] = (same ? 0 : 1) + (k.wrong ? 2 : 0);
    }
}

// As k_gdr_again, from the last segment to the first.
template <typename T, int DKP, bool AL>
__global__ void __launch_bounds__(256, 1)
k_gdr_again_back(const LaunchGdr p) {
    using W = GdrWalkBack<T, DKP, AL>;
    __shared__ alignas(16) T tk[64 * DKP], tq[64 * DKP], tt[Mx<T>::NT * kGdrTri], tp[Mx<T>::NT * kGdrTri];
    __shared__ alignas(16) float tok[kGdrTok * 64], srq[64];
    const int64_t BH = p.B * p.H, bh = blockIdx.x % BH, tile = blockIdx.x / BH, b = bh / p.H, kv = (int64_t)p.dk * p.dv;
    const int tiles = (p.dv + 63) / 64, h = (int)(bh % p.H), hk = h / (p.H / p.Hk), lane = threadIdx.x & 63;
    const uint32_t* off = p.wQ + (bh * tiles + tile) * p.nseg * 4;
    bool any = false, wrong = false;
    for (int i = lane; i < p.nseg * 4; i += 64) {
        any |= off[i] != 0;
        wrong |= i % 4 == gdr_wave() && off[i] >= 2;
    }
    if (!__any(any)) return;
    W k(p, tk, tq, tt, tp, tok, srq, b, bh, h, hk, (int)tile * 64 + gdr_wave() * 16 + (lane & 15));
    k.wrong = __any(wrong);
    gdr_clear_back<T, DKP>(p, tk, tq, tp);
    bool here = false;                                // the gradient behind the segment is in registers
    for (int seg = p.nseg - 2; seg >= 0; --seg) {
        const int64_t at = (seg * BH + bh) * kv;
        const bool own = !k.wrong && (here ? !k.agrees(p.wE + at) : off[(seg + 1) * 4 + k.w] != 0);
        if (!__syncthreads_or(own)) {                 // (a barrier, too: the last segment's LDS is used up)
            here = false;
            continue;
        }
        if (!here) k.load_state(own ? p.wX + at : p.wE + at, p.dv);
        gdr_walk_back<true>(k, seg * p.seg, (seg + 1) * p.seg);
        here = true;
        if (seg == 0 && p.gr.dstate_init) k.store_state(p.gr.dstate_init + bh * kv, p.dv);
    }
    if (k.wrong) {
        gdr_tokens_back<T>(k);
        if (p.gr.dstate_init) k.store_state(p.gr.dstate_init + bh * kv, p.dv);
    }
}

// ---------------------------------------------------------------------------
// The gradients of a chunk's keys, queries and gates, all chunks at once, from the states in front (S0) and
// their gradients behind (W), X and dV:
//   dq = a2 dY S0^T + E' K,     dk = a3 X W^T - a1 dV S0^T + E'^T Q + (F + F^T) K
//   E = dY X^T (i >= j), F = -dV X^T (i > j), each times beta_j and what P and N have beside the product of their rows
//   dbeta_j = k_j . (a3b X W^T)_j + sum_i E_ij P_ij + F_ij N_ij / beta_j     (E, F without beta)
//   dg_t: every term that a token from t on has from one in front of t, summed as such (no difference of
//   two sums, so that the gradient of a small decay, which has it as a factor, keeps its digits):
//   sum_{i >= t > j} beta_j (E P + F N/beta)_ij + sum_{i >= t} (q . a2 dY S0^T - k . a1 dV S0^T)_i
//     + sum_{j < t} beta_j (k . a3b X W^T)_j + e^G_last <S0, W>
// A wave has a quarter of dk, transposed (a lane has a token): sums over dk are sums over registers and two moves, factors
// of tokens one register, and four neighbouring columns one store. Terms over dv go through LDS 32 at a time, the next
// ones on their way to registers meanwhile. 10240 chunks of 128 x 128 in bf16: 745 us, 3.8 TB/s of what it reads and
// writes; a workgroup waits for its first and its last rows while the other of its CU works (with one way to load
// a kernel: where aligned and unaligned loads met, the copies between them waited for memory, 1005 us).
template <typename T, int DKP, bool AL, bool VEC, int GROUPS>
__global__ void __launch_bounds__(256, GROUPS)
k_gdr_grads(const LaunchGdr p) {
    using M = Mx<T>;
    constexpr int KD = DKP / 32, NS = DKP / 64, LD = 68, SL = 4 * 512;      // SL: 64 rows of 32 terms
    constexpr bool BOTH = 2 * 64 * DKP * (int)sizeof(T) <= 32768;          // keys and queries lie in LDS side by side
    constexpr int kPhase1 = (2 * M::NT + 1) * SL * (int)sizeof(T), kPhase2 = 2 * 64 * LD * 4;
    __shared__ alignas(16) T tk[64 * DKP], tq_[BOTH ? 64 * DKP : 8];
    __shared__ alignas(16) char lds[kPhase1 > kPhase2 ? kPhase1 : kPhase2];
    __shared__ alignas(16) float tok[kGdrTokAll * 64];
    __shared__ alignas(16) float srq[64], rows[2][4][64], colsum[4][64], wsum[4];
    T (*lx)[SL] = reinterpret_cast<T (*)[SL]>(lds), (*lv)[SL] = lx + M::NT, *lo = lx[2 * M::NT], *tq = BOTH ? tq_ : tk;
    float (*me)[LD] = reinterpret_cast<float (*)[LD]>(lds), (*mf)[LD] = me + 64;
    const int tid = threadIdx.x, w = gdr_wave();
    int lane = tid & 63, g = lane >> 4, m = lane & 15, place = gdr_place(g, m);
    const int64_t id = blockIdx.x, nc = p.nchunks, n = id % nc, bh = id / nc, b = bh / p.H, t0 = n * kGdrC;
    const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk), left = p.L - t0 < kGdrC ? (int)(p.L - t0) : kGdrC;
    const GdrRows<T, KD, AL> rk(p.k, b, hk, p.dk), rq(p.q, b, hk, p.dk);
    const T* qg = rq.base + t0 * rq.stride;
    if (p.dk < DKP) {
        gdr_clear<64 * DKP>(tk);
        if (BOTH) gdr_clear<64 * DKP>(tq_);
        __syncthreads();
    }
    // what a lane brings of 32 columns: an eight of X, dV and dY for LDS, and its rows of S0 and W
    const int64_t kv = (int64_t)p.dk * p.dv, row0 = (b * p.L + t0) * p.H + h;
    const int ts = tid >> 2, octet = tid & 3;
    const unsigned row_v = (unsigned)(p.H * p.dv), size_v = (left - 1) * row_v + p.dv, size_s = (unsigned)kv * 4;
    const GdrBuf<float> bx(p.ckptX + row0 * p.dv, size_v * 4), bv(p.wV + row0 * p.dv, size_v * 4);
    const GdrBuf<T> bo(static_cast<const T*>(p.gr.dy) + row0 * p.dv, size_v * (unsigned)sizeof(T));
    const GdrBuf<float> bs(p.ckpt + id * kv, size_s), bw(p.wS + id * kv, size_s);
    const int d0 = 8 * (m >> 2) + (m & 3);
    gf8 nx, nv, ns[NS], nw[NS];
    alignas(16) T ny[8];
    // (zeros behind the last token, as it has no gradient, and past dk and dv)
    auto fetch_rows = [&](int c0) {
        const int c = c0 + octet * 8;
        const unsigned at = ts * row_v + c;
        nx = bx.template ld8<VEC>(at * 4, c, p.dv);
        nv = bv.template ld8<VEC>(at * 4, c, p.dv);
        bo.template ld8<VEC>(at * (unsigned)sizeof(T), c, p.dv, ny);
    };
    auto fetch_state = [&](const GdrBuf<float>& from, int c0, gf8 (&to)[NS]) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int q = w * NS + u, e = c0 + 8 * g;
            to[u] = from.template ld8<VEC>((unsigned)((32 * (q >> 1) + 4 * (q & 1) + d0) * p.dv + e) * 4, e, p.dv);
        }
    };
    gf4 aq[NS][4] = {}, av[NS][4] = {}, ax[NS][4] = {}, ae[3] = {}, af[3] = {};
    float ww = 0.0f;
    fetch_rows(0);
    fetch_state(bs, 0, ns);
    fetch_state(bw, 0, nw);
    rk.load(tk, t0, p.L);                             // behind what is needed first
    if (BOTH) rq.load(tq, t0, p.L);
    if (w * 64 + lane < kGdrTokAll * 16)
        GdrSource(p.co + id * (kGdrTokAll * 64)).to_lds(reinterpret_cast<gu4*>(tok + w * 256), lane * 16, w * 1024);
    colsum[tid >> 6][tid & 63] = 0.0f;
    // a lane's places are made again in every turn and behind the last: kept over the loop they would spill
    auto places = [&] {
        asm volatile("" : "+v"(lane));
        g = lane >> 4;
        m = lane & 15;
        place = gdr_place(g, m);
    };
    for (int c0 = 0; c0 < p.dv; c0 += 32) {
        places();
        __syncthreads();
        {
            const auto x = M::template split<M::NT>(nx), v = M::template split<M::NT>(nv);
            const int unit = ts >> 4, pl = gdr_place(octet, ts & 15);
            auto put = [&](T* to, const typename M::F& f) {
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<gb8*>(to + (unit * 64 + pl) * 8) = f;
                } else {
                    *reinterpret_cast<gf4*>(to + (unit * 128 + pl) * 4) = gf4{f[0], f[1], f[2], f[3]};
                    *reinterpret_cast<gf4*>(to + (unit * 128 + 64 + pl) * 4) = gf4{f[4], f[5], f[6], f[7]};
                }
            };
#pragma unroll
            for (int k = 0; k < M::NT; ++k) { put(lx[k], x.t[k]); put(lv[k], v.t[k]); }
            put(lo, __builtin_bit_cast(typename M::F, ny));
        }
        __syncthreads();
        // one of S0 and W as terms at a time, the next of its kind on the way into its registers meanwhile: both at once
        // would not fit
        const bool more = c0 + 32 < p.dv;
        if (more) fetch_rows(c0 + 32);
        {
            typename M::template S<M::NT> sb[NS];
#pragma unroll
            for (int u = 0; u < NS; ++u) {
#pragma unroll
                for (int j = 0; j < 8; ++j) ww = __builtin_fmaf(ns[u][j], nw[u][j], ww);
                sb[u] = M::template split<M::NT>(ns[u]);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (more) fetch_state(bs, c0 + 32, ns);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                typename M::template S<M::NT> vf;
#pragma unroll
                for (int k = 0; k < M::NT; ++k) vf.t[k] = gdr_rows_frag<T>(lv[k], i, place);
                const auto of = gdr_rows_frag<T>(lo, i, place);
                M::template each<M::NT>([&](int a, int c) {
#pragma unroll
                    for (int u = 0; u < NS; ++u) av[u][i] = M::mm(sb[u].t[a], vf.t[c], av[u][i]);
                });
#pragma unroll
                for (int k = M::NT - 1; k >= 0; --k)
#pragma unroll
                    for (int u = 0; u < NS; ++u) aq[u][i] = M::mm(sb[u].t[k], of, aq[u][i]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        {
            typename M::template S<M::NT> wb[NS];
#pragma unroll
            for (int u = 0; u < NS; ++u) wb[u] = M::template split<M::NT>(nw[u]);
            __builtin_amdgcn_sched_barrier(0);
            if (more) fetch_state(bw, c0 + 32, nw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                typename M::template S<M::NT> xf;
#pragma unroll
                for (int k = 0; k < M::NT; ++k) xf.t[k] = gdr_rows_frag<T>(lx[k], i, place);
                M::template each<M::NT>([&](int a, int c) {
#pragma unroll
                    for (int u = 0; u < NS; ++u) ax[u][i] = M::mm(wb[u].t[a], xf.t[c], ax[u][i]);
                });
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            const int tile = w + 4 * u;
            if (tile < 10) {
                int mt, nt;
                gdr_tile(tile, mt, nt);
                typename M::template S<M::NT> xf, vf;
#pragma unroll
                for (int k = 0; k < M::NT; ++k) { xf.t[k] = gdr_rows_frag<T>(lx[k], nt, place); vf.t[k] = gdr_rows_frag<T>(lv[k], mt, place); }
                const auto of = gdr_rows_frag<T>(lo, mt, place);
#pragma unroll
                for (int k = M::NT - 1; k >= 0; --k) ae[u] = M::mm(of, xf.t[k], ae[u]);
                M::template each<M::NT>([&](int a, int c) { af[u] = M::mm(vf.t[a], xf.t[c], af[u]); });
            }
        }
    }
    gdr_arrived();                                    // keys, queries and factors are there
    places();
    // a query's fragment, from LDS or memory
    auto query = [&](int i, int s) {
        if constexpr (BOTH) {
            return gdr_rows_frag<T>(tq, i * KD + s, place);
        } else {
            alignas(16) T x[8];
            const int t = 16 * i + m;
            gdr_row8<T>(qg + (t < left ? t : left - 1) * rq.stride, 32 * s + 8 * g, p.dk, AL, true, x);
            return __builtin_bit_cast(typename M::F, x);
        }
    };
    {
        gf4 len = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KD; ++s) {
            const auto f = query(w, s);
            len = M::mm(f, f, len);
        }
        const float q2 = (m & 3) == 0 ? len[0] : (m & 3) == 1 ? len[1] : (m & 3) == 2 ? len[2] : len[3];
        if (m >> 2 == g) srq[16 * w + m] = p.eps > 0.0f ? __builtin_amdgcn_rsqf(q2 + p.eps) : 1.0f;
    }
    gf4 kk[3] = {}, qk[3] = {};
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int tile = w + 4 * u;
        if (tile < 10) {
            int mt, nt;
            gdr_tile(tile, mt, nt);
#pragma unroll
            for (int s = 0; s < KD; ++s) {
                const auto kn = gdr_rows_frag<T>(tk, nt * KD + s, place);
                kk[u] = M::mm(gdr_rows_frag<T>(tk, mt * KD + s, place), kn, kk[u]);
                qk[u] = M::mm(query(mt, s), kn, qk[u]);
            }
        }
    }
    __syncthreads();                                  // the terms' LDS becomes the pairs', and the queries' lengths are there
    // pairs of tokens: E' on and below me's diagonal, the terms of dg transposed above it; F + F^T in mf
    const double* G = reinterpret_cast<const double*>(tok + tG * 64);
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int tile = w + 4 * u;
        if (tile < 10) {
            int mt, nt;
            gdr_tile(tile, mt, nt);
            const int j = nt * 16 + m, i0 = mt * 16 + 4 * g;
            const float beta = tok[tBeta * 64 + j], rkj = tok[tRk * 64 + j];
            const gf4 ri = *reinterpret_cast<const gf4*>(&tok[tRk * 64 + i0]), qi = *reinterpret_cast<const gf4*>(&srq[i0]);
            const double gj = G[j];
            double gi[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) gi[r] = G[i0 + r];
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + r;
                // where the decay is nothing no gradient passes
                const float d = i < j ? 0.0f : __builtin_amdgcn_exp2f((float)(gi[r] - gj)) * rkj;
                const float fq = d * qi[r] * p.scale, fk = d * ri[r];
                const float e = d != 0.0f ? ae[u][r] : 0.0f, f = i > j && d != 0.0f ? -af[u][r] : 0.0f;
                const float term = d != 0.0f ? e * fq * qk[u][r] + f * fk * kk[u][r] : 0.0f;
                s += term;
                if (i >= j) me[i][j] = e * beta * fq;
                if (i > j) {
                    me[j][i] = term * beta;
                    mf[i][j] = mf[j][i] = f * beta * fk;
                } else if (i == j) {
                    mf[i][i] = 0.0f;
                }
            }
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            if (g == 0) colsum[mt][j] = s;
        }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) ww += __shfl_xor(ww, o, 64);
    if (lane == 0) wsum[w] = ww;
    // sums over dk of a token's row
    auto key4 = [&](const T* tiles, int i, int q) {   // four neighbouring columns of this lane's token
        const int d = 8 * g + 4 * (q & 1), unit = i * KD + (q >> 1), pl = gdr_place(g, m);
        gf4 x;
        if constexpr (sizeof(T) == 2) {
            typedef uint32_t gu2 __attribute__((ext_vector_type(2)));
            const gu2 u = *reinterpret_cast<const gu2*>(tiles + (unit * 64 + pl) * 8 + (d & 7));
            x = gf4{__builtin_bit_cast(float, u[0] << 16), __builtin_bit_cast(float, u[0] & 0xffff0000u),
                    __builtin_bit_cast(float, u[1] << 16), __builtin_bit_cast(float, u[1] & 0xffff0000u)};
        } else {
            x = *reinterpret_cast<const gf4*>(tiles + (unit * 128 + (q & 1) * 64 + pl) * 4);
        }
        return x;
    };
    auto query4 = [&](int i, int q) {
        if constexpr (BOTH) return key4(tq, i, q);
        else {
            gf4 x;
            const int t = 16 * i + m, d = 32 * (q >> 1) + 8 * g + 4 * (q & 1);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = d + r < p.dk ? gdr_f<T>(qg[(t < left ? t : left - 1) * rq.stride + d + r]) : 0.0f;
            return x;
        }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 16 * i + m;
        const float a1 = tok[tA1 * 64 + t], a2 = tok[tA2 * 64 + t] * srq[t] * p.scale, a3 = tok[tA3b * 64 + t], beta = tok[tBeta * 64 + t];
        float y = 0.0f, z = 0.0f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const gf4 k4 = key4(tk, i, w * NS + u), q4 = query4(i, w * NS + u);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                aq[u][i][r] = a2 != 0.0f ? a2 * aq[u][i][r] : 0.0f;
                av[u][i][r] = a1 != 0.0f ? a1 * av[u][i][r] : 0.0f;
                ax[u][i][r] = a3 != 0.0f ? a3 * ax[u][i][r] : 0.0f;
                y = __builtin_fmaf(q4[r], aq[u][i][r], y);
                y = __builtin_fmaf(-k4[r], av[u][i][r], y);
                z = __builtin_fmaf(k4[r], ax[u][i][r], z);
                av[u][i][r] = beta * ax[u][i][r] - av[u][i][r];                    // from here on the key's gradient
            }
        }
        y += __shfl_xor(y, 16, 64);
        z += __shfl_xor(z, 16, 64);
        y += __shfl_xor(y, 32, 64);
        z += __shfl_xor(z, 32, 64);
        if (g == 0) {
            rows[0][w][t] = y;
            rows[1][w][t] = z;
        }
    }
    __syncthreads();
    // dq += E' K, dk += (F + F^T) K, transposed: keys' rows as the first operand
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        typename M::F kf[NS];
#pragma unroll
        for (int u = 0; u < NS; ++u) kf[u] = gdr_frag_t<T, KD>(tk, s, (w * NS + u) >> 1, (w * NS + u) & 1, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * i + m, c = 32 * s + 4 * g;
            gf8 e = gdr_pair(*reinterpret_cast<const gf4*>(&me[r][c]), *reinterpret_cast<const gf4*>(&me[r][c + 16]));
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = c + 16 * (j >> 2) + (j & 3) <= r ? e[j] : 0.0f;
            const auto ef = M::template split<M::NT>(e);
            const auto ff = M::template split<M::NT>(gdr_pair(*reinterpret_cast<const gf4*>(&mf[r][c]), *reinterpret_cast<const gf4*>(&mf[r][c + 16])));
#pragma unroll
            for (int u = 0; u < NS; ++u) {
                if (i >= 2 * s) aq[u][i] = M::template mul<M::NT>(kf[u], ef, aq[u][i]);
                av[u][i] = M::template mul<M::NT>(kf[u], ff, av[u][i]);
            }
        }
    }
    if (!BOTH) {
        __syncthreads();
        rq.load(tk, t0, p.L);
        gdr_arrived();
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        typename M::F qf[NS];
#pragma unroll
        for (int u = 0; u < NS; ++u) qf[u] = gdr_frag_t<T, KD>(tq, s, (w * NS + u) >> 1, (w * NS + u) & 1, lane);
#pragma unroll
        for (int i = 0; i < 2 * s + 2; ++i) {
            gf8 e;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 32 * s + 16 * (j >> 2) + 4 * g + (j & 3);
                e[j] = r >= 16 * i + m ? me[r][16 * i + m] : 0.0f;
            }
            const auto ef = M::template split<M::NT>(e);
#pragma unroll
            for (int u = 0; u < NS; ++u) av[u][i] = M::template mul<M::NT>(qf[u], ef, av[u][i]);
        }
    }
    // gates: a wave has 16 tokens t. Sums over j < t of the terms (i, j) are products with a triangle of ones, and a lane adds
    // its rows i >= t of them.
    {
        gf4 sum = {0, 0, 0, 0};
        float mine = 0.0f;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            if (it < w) continue;
            sum = gf4{0, 0, 0, 0};
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                if (jt > w) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = 16 * it + m, j = 16 * jt + 4 * k + g;
                    const float x = me[j][i];
                    sum = __builtin_amdgcn_mfma_f32_16x16x4f32(i > j ? x : 0.0f, j < 16 * w + m ? 1.0f : 0.0f, sum, 0, 0, 0);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) mine += 16 * it + 4 * g + r >= 16 * w + m ? sum[r] : 0.0f;
        }
        mine += __shfl_xor(mine, 16, 64);
        mine += __shfl_xor(mine, 32, 64);
        float y = rows[0][0][lane] + rows[0][1][lane] + rows[0][2][lane] + rows[0][3][lane];
        const float z = rows[1][0][lane] + rows[1][1][lane] + rows[1][2][lane] + rows[1][3][lane];
        float before = z * tok[tBeta * 64 + lane];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float u = __shfl_up(before, o, 64), v = __shfl_down(y, o, 64);
            if (lane >= o) before += u;
            if (lane + o < 64) y += v;
        }
        before = __shfl_up(before, 1, 64);
        if (lane == 0) before = 0.0f;
        const float end = tok[tMisc * 64];
        mine += __shfl(y + before, 16 * w + m, 64) + (end != 0.0f ? end * (wsum[0] + wsum[1] + wsum[2] + wsum[3]) : 0.0f);
        const int t = 16 * w + m;
        const float db = __shfl(z, t, 64) + colsum[0][t] + colsum[1][t] + colsum[2][t] + colsum[3][t];
        if (g == 0 && t < left) {
            const int64_t at = row0 + (int64_t)t * p.H;
            p.gr.dg[at] = p.reset && p.reset[b * p.L + t0 + t] ? 0.0f : mine;
            p.gr.dbeta[at] = db;
        }
        // zeros of pairs do not keep what is not finite from other tokens
        float of_all = mine + db;
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) of_all += aq[u][i][r] + av[u][i][r];
        const bool wrong = tok[tMisc * 64 + 5] != 0.0f || !__all(fabsf(of_all) < __builtin_inff());
        if (lane == 0) p.wG[id * 4 + w] = wrong;
    }
    if (p.part_q) {
        // heads that share keys: each head's share
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * i + m;
            if (t >= left) continue;
            const int64_t at = (row0 + (int64_t)t * p.H) * p.dk;
#pragma unroll
            for (int u = 0; u < NS; ++u) {
                const int q = w * NS + u, d = 32 * (q >> 1) + 8 * g + 4 * (q & 1);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (d + r < p.dk) {
                        p.part_q[at + d + r] = aq[u][i][r];
                        p.part_k[at + d + r] = av[u][i][r];
                    }
            }
        }
        return;
    }
    // through the division by the length: d - x (x . d) / |x|^2
    __syncthreads();                                  // (where both do not fit, LDS holds the queries by now)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y = 0.0f, z = 0.0f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const gf4 q4 = query4(i, w * NS + u);
            gf4 k4;
            if constexpr (BOTH) {
                k4 = key4(tk, i, w * NS + u);
            } else {
                const int t = 16 * i + m, d = 32 * ((w * NS + u) >> 1) + 8 * g + 4 * ((w * NS + u) & 1);
#pragma unroll
                for (int r = 0; r < 4; ++r) k4[r] = d + r < p.dk ? gdr_f<T>(rk.base[(t0 + (t < left ? t : left - 1)) * rk.stride + d + r]) : 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y = __builtin_fmaf(q4[r], aq[u][i][r], y);
                z = __builtin_fmaf(k4[r], av[u][i][r], z);
            }
        }
        y += __shfl_xor(y, 16, 64);
        z += __shfl_xor(z, 16, 64);
        y += __shfl_xor(y, 32, 64);
        z += __shfl_xor(z, 32, 64);
        if (g == 0) {
            rows[0][w][16 * i + m] = y;
            rows[1][w][16 * i + m] = z;
        }
    }
    __syncthreads();
    const unsigned row = (unsigned)(p.Hk * p.dk);
    const GdrBuf<T> dqt(static_cast<T*>(p.gr.dq) + ((b * p.L + t0) * p.Hk + hk) * p.dk);
    const GdrBuf<T> dkt(static_cast<T*>(p.gr.dk) + ((b * p.L + t0) * p.Hk + hk) * p.dk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 16 * i + m;
        float cq = 0.0f, ck = 0.0f;
        if (p.eps > 0.0f) {
            const float rk2 = tok[tRk * 64 + t], rq2 = srq[t];
            cq = (rows[0][0][t] + rows[0][1][t] + rows[0][2][t] + rows[0][3][t]) * rq2 * rq2;
            ck = (rows[1][0][t] + rows[1][1][t] + rows[1][2][t] + rows[1][3][t]) * rk2 * rk2;
        }
        if (t >= left) continue;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int q = w * NS + u, d = 32 * (q >> 1) + 8 * g + 4 * (q & 1);
            const gf4 q4 = query4(i, q);
            gf4 k4;
            if constexpr (BOTH) {
                k4 = key4(tk, i, q);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) k4[r] = d + r < p.dk ? gdr_f<T>(rk.base[(t0 + t) * rk.stride + d + r]) : 0.0f;
            }
            const gf4 oq = aq[u][i] - q4 * cq, ok = av[u][i] - k4 * ck;
            const unsigned at = (t * row + d) * (unsigned)sizeof(T);
            if (AL && p.vec_dk) {
                if (d < p.dk) {
                    dqt.st4(oq, at, 0);
                    dkt.st4(ok, at, 0);
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (d + r < p.dk) {
                        dqt.st(oq[r], at + r * (unsigned)sizeof(T), 0);
                        dkt.st(ok[r], at + r * (unsigned)sizeof(T), 0);
                    }
            }
        }
    }
}

// The gradients of chunks with anything that is not finite, token by token: the state in front of a token from the chunk's
// first one on, the gradient behind it from the last one back, so that it reaches what the formulas say and nothing else. A lane
// has a row of 16 columns of both, a workgroup eight of a chunk's tokens (blockIdx.y) and some chunks one after the other: 16, or
// 64 where there are thousands and looking at them takes longest. 5 to 10 us where every chunk is finite; where none is,
// 10240 chunks of 128 x 128 take 130 ms.
template <typename T>
__global__ void __launch_bounds__(256)
k_gdr_grads_again(const LaunchGdr p, int per) {
    constexpr int CW = 16, TW = kGdrC / 8;
    __shared__ float lx[kGdrC][CW], lv[kGdrC][CW], lo[kGdrC][CW], decay[kGdrC], beta[kGdrC], rk[kGdrC], rq[kGdrC], sums[4][4];
    const int tid = threadIdx.x, lane = tid & 63, w = gdr_wave();
    const int64_t chunks = p.B * p.H * p.nchunks, kv = (int64_t)p.dk * p.dv;
    for (int64_t first = (int64_t)blockIdx.x * per; first < chunks; first += (int64_t)gridDim.x * per) {
        bool off = false;
        if (lane < per && first + lane < chunks) {
            const gu4 u = *reinterpret_cast<const gu4*>(p.wG + (first + lane) * 4);
            off = (u[0] | u[1] | u[2] | u[3]) != 0;
        }
        uint64_t todo = __ballot(off);                // the same in all waves
        for (; todo; todo &= todo - 1) {
            const int64_t id = first + __builtin_ctzll(todo), n = id % p.nchunks, bh = id / p.nchunks, b = bh / p.H, t0 = n * kGdrC;
            const int h = (int)(bh % p.H), hk = h / (p.H / p.Hk), left = p.L - t0 < kGdrC ? (int)(p.L - t0) : kGdrC, d = tid;
            const int64_t row0 = (b * p.L + t0) * p.H + h;
            const bool row = d < p.dk;
            const T* kr = static_cast<const T*>(p.k.p) + b * p.k.batch_stride + hk * p.k.head_stride + t0 * p.k.token_stride;
            const T* qr = static_cast<const T*>(p.q.p) + b * p.q.batch_stride + hk * p.q.head_stride + t0 * p.q.token_stride;
            __syncthreads();                          // the last chunk's values are used up
            for (int t = w; t < left; t += 4) {
                float k2 = 0.0f, q2 = 0.0f;
                for (int e = lane; e < p.dk; e += 64) {
                    const float kx = gdr_f<T>(kr[t * p.k.token_stride + e]), qx = gdr_f<T>(qr[t * p.q.token_stride + e]);
                    k2 = __builtin_fmaf(kx, kx, k2);
                    q2 = __builtin_fmaf(qx, qx, q2);
                }
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    k2 += __shfl_xor(k2, o, 64);
                    q2 += __shfl_xor(q2, o, 64);
                }
                if (lane == 0) {
                    const int64_t at = row0 + (int64_t)t * p.H;
                    rk[t] = p.eps > 0.0f ? 1.0f / sqrtf(k2 + p.eps) : 1.0f;
                    rq[t] = p.eps > 0.0f ? 1.0f / sqrtf(q2 + p.eps) : 1.0f;
                    decay[t] = p.reset && p.reset[b * p.L + t0 + t] ? 0.0f : expf(p.g[at]);
                    beta[t] = p.beta[at];
                }
            }
            float gq[TW] = {}, gk[TW] = {}, gb[TW] = {}, gg[TW] = {};
            for (int c0 = 0; c0 < p.dv; c0 += CW) {
                const int cols = p.dv - c0 < CW ? p.dv - c0 : CW;
                __syncthreads();
                for (int e = tid; e < kGdrC * CW; e += 256) {
                    const int t = e / CW, c = e % CW;
                    const bool there = t < left && c < cols;
                    const int64_t at = (row0 + (int64_t)(there ? t : 0) * p.H) * p.dv + c0 + (there ? c : 0);
                    lx[t][c] = there ? p.ckptX[at] : 0.0f;
                    lv[t][c] = there ? p.wV[at] : 0.0f;
                    lo[t][c] = there ? gdr_f<T>(static_cast<const T*>(p.gr.dy)[at]) : 0.0f;
                }
                __syncthreads();
                if (!row) continue;                   // (every lane meets every barrier)
                float S0[CW], W0[CW];
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    S0[c] = c < cols ? p.ckpt[id * kv + (int64_t)d * p.dv + c0 + c] : 0.0f;
                    W0[c] = c < cols ? p.wS[id * kv + (int64_t)d * p.dv + c0 + c] : 0.0f;
                }
                // to the first of the eight tokens, and the states in front of them; then back to the last
                const int t1 = blockIdx.y * TW;
                float S[TW][CW];                      // decayed
#pragma unroll 4
                for (int t = 0; t < t1 && t < left; ++t) {
                    const float a = decay[t], kt = gdr_f<T>(kr[t * p.k.token_stride + d]) * rk[t], be = beta[t];
#pragma unroll
                    for (int c = 0; c < CW; ++c) S0[c] = __builtin_fmaf(kt, be * lx[t][c], a != 0.0f ? a * S0[c] : 0.0f);
                }
#pragma unroll
                for (int e = 0; e < TW; ++e) {
                    const int t = t1 + e;
                    if (t >= left) break;
                    const float a = decay[t], kt = gdr_f<T>(kr[t * p.k.token_stride + d]) * rk[t], be = beta[t];
#pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        S[e][c] = a != 0.0f ? a * S0[c] : 0.0f;
                        S0[c] = __builtin_fmaf(kt, be * lx[t][c], S[e][c]);
                    }
                }
#pragma unroll 4
                for (int t = left - 1; t >= t1 + TW; --t) {
                    const float a = decay[t], kt = gdr_f<T>(kr[t * p.k.token_stride + d]) * -rk[t];
                    const float qt = gdr_f<T>(qr[t * p.q.token_stride + d]) * (rq[t] * p.scale);
#pragma unroll
                    for (int c = 0; c < CW; ++c)
                        W0[c] = a != 0.0f ? a * __builtin_fmaf(kt, lv[t][c], __builtin_fmaf(qt, lo[t][c], W0[c])) : 0.0f;
                }
#pragma unroll
                for (int e = TW - 1; e >= 0; --e) {
                    const int t = t1 + e;
                    if (t >= left) continue;
                    const float a = decay[t], kt = gdr_f<T>(kr[t * p.k.token_stride + d]) * rk[t], be = beta[t];
                    const float qt = gdr_f<T>(qr[t * p.q.token_stride + d]) * (rq[t] * p.scale);
#pragma unroll
                    for (int c = 0; c < CW; ++c)
                        if (c < cols) {               // (a NaN times the zeros past dv would count)
                            const float s = S[e][c], u = be * lx[t][c], wt = __builtin_fmaf(qt, lo[t][c], W0[c]), dw = __builtin_fmaf(-kt, lv[t][c], wt);
                            gq[e] = __builtin_fmaf(__builtin_fmaf(kt, u, s), lo[t][c], gq[e]);
                            gk[e] = __builtin_fmaf(wt, u, gk[e]);
                            gk[e] = __builtin_fmaf(-s, lv[t][c], gk[e]);
                            gb[e] = __builtin_fmaf(kt * wt, lx[t][c], gb[e]);
                            gg[e] = __builtin_fmaf(s, dw, gg[e]);
                            W0[c] = a != 0.0f ? a * dw : 0.0f;
                        }
                }
            }
#pragma unroll
            for (int e = 0; e < TW; ++e) {
                const int t = blockIdx.y * TW + e;
                if (t >= left) break;
                const int64_t at = row0 + (int64_t)t * p.H;
                const float kx = row ? gdr_f<T>(kr[t * p.k.token_stride + d]) : 0.0f, qx = row ? gdr_f<T>(qr[t * p.q.token_stride + d]) : 0.0f;
                const float oq = gq[e] * (p.scale * rq[t]), ok = gk[e] * rk[t];
                float v[4] = {gb[e], gg[e], row ? qx * oq : 0.0f, row ? kx * ok : 0.0f};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int o = 1; o < 64; o <<= 1) v[k] += __shfl_xor(v[k], o, 64);
                }
                __syncthreads();
                if (lane == 0)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sums[k][w] = v[k];
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = sums[k][0] + sums[k][1] + sums[k][2] + sums[k][3];
                if (tid == 0) {
                    p.gr.dbeta[at] = v[0];
                    p.gr.dg[at] = p.reset && p.reset[b * p.L + t0 + t] ? 0.0f : v[1];
                }
                if (!row) continue;
                if (p.part_q) {
                    p.part_q[at * p.dk + d] = oq;
                    p.part_k[at * p.dk + d] = ok;
                } else {
                    const int64_t to = ((b * p.L + t0 + t) * p.Hk + hk) * p.dk + d;
                    IO<T>::st(static_cast<T*>(p.gr.dq) + to, p.eps > 0.0f ? oq - qx * (v[2] * rq[t] * rq[t]) : oq);
                    IO<T>::st(static_cast<T*>(p.gr.dk) + to, p.eps > 0.0f ? ok - kx * (v[3] * rk[t] * rk[t]) : ok);
                }
            }
        }
    }
}

// The heads' shares of a key's and a query's gradient, and through the division by the length:
// d = s - x (x . s) / |x|^2. One wave a row, up to 256 columns.
template <typename T>
__global__ void __launch_bounds__(256)
k_gdr_keys(const LaunchGdr p) {
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < p.B * p.L * p.Hk; row += (int64_t)gridDim.x * 4) {
    const int hk = (int)(row % p.Hk), rep = p.H / p.Hk;
    const int64_t bt = row / p.Hk, b = bt / p.L, t = bt % p.L;
    const ss_head_view& v = blockIdx.y ? p.k : p.q;
    const float* part = (blockIdx.y ? p.part_k : p.part_q) + (bt * p.H + (int64_t)hk * rep) * p.dk;
    const T* x = static_cast<const T*>(v.p) + b * v.batch_stride + t * v.token_stride + hk * v.head_stride;
    T* out = static_cast<T*>(blockIdx.y ? p.gr.dk : p.gr.dq) + row * p.dk;
    float s[4], xv[4], dot = 0.0f, len = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = j * 64 + lane;
        s[j] = 0.0f;
        xv[j] = d < p.dk ? IO<T>::ld(x + d) : 0.0f;
        if (d < p.dk)
            for (int i = 0; i < rep; ++i) s[j] += part[(int64_t)i * p.dk + d];
        dot = __builtin_fmaf(xv[j], s[j], dot);
        len = __builtin_fmaf(xv[j], xv[j], len);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        dot += __shfl_xor(dot, o, 64);
        len += __shfl_xor(len, o, 64);
    }
    const float c = p.eps > 0.0f ? dot / (len + p.eps) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = j * 64 + lane;
        if (d < p.dk) IO<T>::st(out + d, p.eps > 0.0f ? s[j] - xv[j] * c : s[j]);
    }
    }
}

// ---------------------------------------------------------------------------
// One token: bound by reading and writing the state. A workgroup has 128 columns of one head, four a lane, or
// 64 where rows do not hold whole accesses of 16 bytes; its rows of lanes share the head's rows, all of
// which are in flight at once, and meet in LDS once:
//   y = scale (e^g S^T q + (q . k) u),  u = beta (v - e^g S^T k)
// Workgroups of one head are eight apart, on the same XCD: rows that share a line meet in its L2, for which
// whole lines only go past it. 64 streams of 64 heads of 128 x 128: 99 us, 5.4 TB/s; 224 streams of 20 heads of
// 128 x 99: 77 us, 5.9 TB/s (300 us with tiles of 32 columns, far apart and past the L2).
template <typename T, int DKP, int CV>
__global__ void __launch_bounds__(256)
k_gdr_step(const LaunchGdr p) {
    typedef float fv __attribute__((ext_vector_type(CV)));
    constexpr int LANES = CV == 4 ? 32 : 64, RG = 256 / LANES, RPT = DKP / RG;
    __shared__ float sq[DKP], sk[DKP], dots[3][4];
    __shared__ alignas(16) float part[2][RG][LANES * CV];
    const int tid = threadIdx.x, lane = tid % LANES, rg = tid / LANES;
    const unsigned tiles = (unsigned)(p.dv + LANES * CV - 1) / (LANES * CV), eight = blockIdx.x / 8, H = (unsigned)p.H;
    const unsigned head = eight / tiles * 8 + blockIdx.x % 8, tile = eight % tiles, h = head % H, hk = h / (H / (unsigned)p.Hk);
    if (head >= (unsigned)p.B * H) return;
    const int64_t bh = head, b = head / H;
    const int col = (int)(tile * LANES + lane) * CV;
    const bool in = col < p.dv;
    float* st = p.state + bh * p.dk * p.dv + col;
    const float* some = in ? st : st - col;                // what is not there is read from somewhere that is, with no branch between the loads
    fv S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = i * RG + rg;
        const fv* from = reinterpret_cast<const fv*>(some + (row < p.dk ? row : 0) * p.dv);
        S[i] = CV == 4 ? __builtin_nontemporal_load(from) : *from;
    }
    float qv = 0.0f, kv = 0.0f;
    if (tid < p.dk) {
        qv = IO<T>::ld(static_cast<const T*>(p.q.p) + b * p.q.batch_stride + hk * p.q.head_stride + tid);
        kv = IO<T>::ld(static_cast<const T*>(p.k.p) + b * p.k.batch_stride + hk * p.k.head_stride + tid);
    }
    if (tid < DKP) { sq[tid] = qv; sk[tid] = kv; }
    float d[3] = {qv * qv, kv * kv, qv * kv};
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
#pragma unroll
        for (int j = 0; j < 3; ++j) d[j] += __shfl_xor(d[j], o, 64);
    if ((tid & 63) == 0) { dots[0][tid >> 6] = d[0]; dots[1][tid >> 6] = d[1]; dots[2][tid >> 6] = d[2]; }
    const float a = p.reset && p.reset[b] ? 0.0f : expf(p.g[bh]), beta = p.beta[bh];
    __syncthreads();
    float rq = 1.0f, rk = 1.0f;
    if (p.eps > 0.0f) {
        rq = 1.0f / sqrtf(dots[0][0] + dots[0][1] + dots[0][2] + dots[0][3] + p.eps);
        rk = 1.0f / sqrtf(dots[1][0] + dots[1][1] + dots[1][2] + dots[1][3] + p.eps);
    }
    const float qk = (dots[2][0] + dots[2][1] + dots[2][2] + dots[2][3]) * rq * rk;
    fv aq = fv(0.0f), ak = fv(0.0f);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        S[i] = a != 0.0f && i * RG + rg < p.dk ? S[i] * a : fv(0.0f);      // a decay of 0: nothing passes, whatever it is
        aq += S[i] * sq[i * RG + rg];
        ak += S[i] * sk[i * RG + rg];
    }
    *reinterpret_cast<fv*>(&part[0][rg][lane * CV]) = aq;
    *reinterpret_cast<fv*>(&part[1][rg][lane * CV]) = ak;
    __syncthreads();
    if (!in) return;
    aq = ak = fv(0.0f);
#pragma unroll
    for (int i = 0; i < RG; ++i) {
        aq += *reinterpret_cast<const fv*>(&part[0][i][lane * CV]);
        ak += *reinterpret_cast<const fv*>(&part[1][i][lane * CV]);
    }
    const T* vp = static_cast<const T*>(p.v.p) + b * p.v.batch_stride + h * p.v.head_stride + col;
    fv u;
#pragma unroll
    for (int j = 0; j < CV; ++j) u[j] = beta * (IO<T>::ld(vp + j) - rk * ak[j]);
    if (rg == 0) {
        T* yp = static_cast<T*>(p.y) + bh * p.dv + col;
#pragma unroll
        for (int j = 0; j < CV; ++j) IO<T>::st(yp + j, p.scale * (rq * aq[j] + qk * u[j]));
    }
    u *= rk;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = i * RG + rg;
        if (row >= p.dk) continue;
        fv* to = reinterpret_cast<fv*>(st + row * p.dv);
        if (CV == 4) __builtin_nontemporal_store(S[i] + u * sk[row], to);
        else *to = S[i] + u * sk[row];
    }
}

template <typename T, int DKP>
hipError_t launch_gdr_d(const LaunchGdr& p) {
    hipStream_t st = static_cast<hipStream_t>(p.stream);
    const int64_t BH = p.B * p.H;
    if (p.pass == LaunchGdr::kStep) {
        const int64_t heads = (BH + 7) / 8 * 8;
        if (p.vec_state) hipLaunchKernelGGL((k_gdr_step<T, DKP, 4>), dim3((unsigned)(heads * ((p.dv + 127) / 128))), dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_gdr_step<T, DKP, 1>), dim3((unsigned)(heads * ((p.dv + 63) / 64))), dim3(256), 0, st, p);
        return hipGetLastError();
    }
    const unsigned chunks = (unsigned)(BH * p.nchunks);
    const unsigned tiles = (unsigned)(BH * ((p.dv + 63) / 64));
    constexpr bool kTwo = DKP * sizeof(T) <= 512;       // keys twice in LDS
    constexpr int kGroups = DKP <= 128 && sizeof(T) == 2 ? 2 : 1;
    constexpr int kGrads = DKP <= 128 ? 2 : 1;
    const bool al = p.vec && p.vec_v;
    if (p.pass == LaunchGdr::kFwd) {
        hipLaunchKernelGGL((k_gdr_solve<T, DKP, false>), dim3((chunks + 3) / 4), dim3(256), 0, st, p);
        if (p.nseg > 1) {
            const dim3 ends((unsigned)(BH * ((p.dv + 63) / 64 + (p.dk + 63) / 64) * (p.nseg - 1)));
            if (al) hipLaunchKernelGGL((k_gdr_ends<T, DKP, kTwo, true, kGroups>), ends, dim3(256), 0, st, p);
            else hipLaunchKernelGGL((k_gdr_ends<T, DKP, kTwo, false, kGroups>), ends, dim3(256), 0, st, p);
            if (p.nseg > 2) hipLaunchKernelGGL((k_gdr_join<T, DKP>), dim3(tiles), dim3(256), 0, st, p);
        }
        const dim3 walk((unsigned)(tiles * p.nseg));
        if (al) hipLaunchKernelGGL((k_gdr_walk<T, DKP, kTwo, true, kGroups>), walk, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_gdr_walk<T, DKP, kTwo, false, kGroups>), walk, dim3(256), 0, st, p);
        if (p.nseg > 1) {
            if (al) hipLaunchKernelGGL((k_gdr_again<T, DKP, kTwo, true>), dim3(tiles), dim3(256), 0, st, p);
            else hipLaunchKernelGGL((k_gdr_again<T, DKP, kTwo, false>), dim3(tiles), dim3(256), 0, st, p);
        }
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_gdr_solve<T, DKP, true>), dim3((chunks + 3) / 4), dim3(256), 0, st, p);
    const dim3 ends(tiles * (p.nseg - 1)), walk(tiles * p.nseg);
    if (p.vec) {
        if (p.nseg > 1) hipLaunchKernelGGL((k_gdr_ends_back<T, DKP, true, kGroups>), ends, dim3(256), 0, st, p);
        hipLaunchKernelGGL((k_gdr_walk_back<T, DKP, true, kGroups>), walk, dim3(256), 0, st, p);
        if (p.nseg > 1) hipLaunchKernelGGL((k_gdr_again_back<T, DKP, true>), dim3(tiles), dim3(256), 0, st, p);
        if (p.vec_ck && p.vec_dy) hipLaunchKernelGGL((k_gdr_grads<T, DKP, true, true, kGrads>), dim3(chunks), dim3(256), 0, st, p);
        else hipLaunchKernelGGL((k_gdr_grads<T, DKP, true, false, kGrads>), dim3(chunks), dim3(256), 0, st, p);
    } else {
        if (p.nseg > 1) hipLaunchKernelGGL((k_gdr_ends_back<T, DKP, false, kGroups>), ends, dim3(256), 0, st, p);
        hipLaunchKernelGGL((k_gdr_walk_back<T, DKP, false, kGroups>), walk, dim3(256), 0, st, p);
        if (p.nseg > 1) hipLaunchKernelGGL((k_gdr_again_back<T, DKP, false>), dim3(tiles), dim3(256), 0, st, p);
        hipLaunchKernelGGL((k_gdr_grads<T, DKP, false, false, kGrads>), dim3(chunks), dim3(256), 0, st, p);
    }
    const int per = chunks < 2048 ? 16 : 64;
    const unsigned look = (chunks + per - 1) / per;
    hipLaunchKernelGGL((k_gdr_grads_again<T>), dim3(look < 512 ? look : 512, 8), dim3(256), 0, st, p, per);
    if (p.part_q) {
        const int64_t rows = (p.B * p.L * p.Hk + 3) / 4;
        hipLaunchKernelGGL((k_gdr_keys<T>), dim3((unsigned)(rows < 1 << 20 ? rows : 1 << 20), 2), dim3(256), 0, st, p);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_gdr_t(const LaunchGdr& p) {
    if (p.dk <= 64) return launch_gdr_d<T, 64>(p);
    if (p.dk <= 128) return launch_gdr_d<T, 128>(p);
    return launch_gdr_d<T, 256>(p);
}

}  // namespace selscan
