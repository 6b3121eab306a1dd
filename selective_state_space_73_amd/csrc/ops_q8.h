// Device code of the 8-bit rounding, alone (ss_quant_q8) and behind the residual's addition
// and the RMS norm (ss_norm_q8).
//
//   s = x + residual;  n = s / sqrt(mean(s^2) + eps) * w
//   per block: scale = max(max |n| / 448, 2^-126),  q = e4m3(448 n / max |n|)
//
// Both are bound by memory: a value is read once, kept in registers through the sums and
// maxima it takes part in, and its byte is written once.
#pragma once
#include "ops_internal.h"
#include "ops_rows.h"
#include "selscan_device.h"

namespace selscan {

constexpr float kQ8Max = 448.0f;             // largest finite e4m3 value
constexpr float kQ8TinyScale = 0x1p-126f;    // smallest scale: its reciprocal is finite

// A block's scale, its largest magnitude (448 2^-126 under the smallest scale) and 448 over that.
struct Q8Scale { float scale, hi, top; };
__device__ __forceinline__ Q8Scale q8_scale(float top) {
    if (top < kQ8Max * kQ8TinyScale) return Q8Scale{kQ8TinyScale, 0x1p126f, kQ8Max * kQ8TinyScale};
    return Q8Scale{top / kQ8Max, kQ8Max / top, top};
}
// t = v hi is within 1.5 fp32 steps of the quotient 448 v / top (a rounded reciprocal, a rounded
// product), so that it goes to the right e4m3 value unless it lies that near to the middle between
// two. How middles are decided depends on where v comes from.
//
// A bf16 v over a bf16 top (8 bits each): if 448 v and middle * top (5 bits) differ, both whole
// multiples of one power of two, they do by 2^-13 of themselves at least. So t rounded to 16 bits is
// a middle where the quotient is one, and on the quotient's side of it everywhere else.
__device__ __forceinline__ float q8_to16(float t) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, t) + 0x80u) & ~0xffu);
}
// Any v: from 2^-6 on the middles are the fp32 numbers whose last 20 bits are a one and zeros. A
// t within two steps of one (a few in a million) is decided by 448 v against middle * top, each
// exactly as the sum of two floats, at top's exponent. (Below, where e4m3 has steps of 2^-9, it is
// left at t.)
__device__ __forceinline__ uint32_t q8_past_middle(float t) {         // two steps below a middle on: 0x1000 a step
    return (__builtin_bit_cast(uint32_t, t) << 12) + 0x80002000u;
}
__device__ __forceinline__ bool q8_near_middle(const float* v, const Q8Scale& s) {
    uint32_t least = ~0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t from = q8_past_middle(v[j] * s.hi);
        least = from < least ? from : least;
    }
    return least <= 0x4000u;
}
__device__ __forceinline__ float q8_decided(float v, const Q8Scale& s) {
    const float t = v * s.hi;
    const uint32_t b = __builtin_bit_cast(uint32_t, t), m = ((b & 0x7fffffffu) + 4u) & ~7u;
    const float a = __builtin_ldexpf(__builtin_fabsf(v), -__builtin_amdgcn_frexp_expf(s.top)), c = __builtin_amdgcn_frexp_mantf(s.top);
    const float mid = __builtin_bit_cast(float, m);
    const float p = kQ8Max * a, q = mid * c;
    const float d = p != q ? p - q : __builtin_fmaf(kQ8Max, a, -p) - __builtin_fmaf(mid, c, -q);
    const uint32_t side = m + (d > 0.0f ? 1u : 0u) - (d < 0.0f ? 1u : 0u);
    return q8_past_middle(t) <= 0x4000u ? __builtin_bit_cast(float, side | (b & 0x80000000u)) : t;
}
__device__ __forceinline__ uint64_t q8_bytes(const float* t) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false), b = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], b, true);
    return (uint64_t)(uint32_t)b << 32 | (uint32_t)a;
}
// Eight values as eight e4m3 bytes, each quotient rounded to the nearest, ties to even. SHORT: bf16
// values of bf16 blocks.
template <bool SHORT>
__device__ __forceinline__ uint64_t q8_eight(const float* v, const Q8Scale& s) {
    float t[8];
    if constexpr (SHORT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = q8_to16(v[j] * s.hi);
    } else if (__any(q8_near_middle(v, s))) {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = q8_decided(v[j], s);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = v[j] * s.hi;
    }
    return q8_bytes(t);
}

template <bool VEC>
__device__ __forceinline__ void st8_q(uint8_t* row, int64_t c, int64_t K, uint64_t u) {
    if (c + 8 <= K) {
        *reinterpret_cast<typename Q8Wide<VEC>::u8*>(row + c) = u;
    } else if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < K) row[c + j] = (uint8_t)(u >> (8 * j));
    }
}

// largest |v| among the 16 lanes that hold one block of 128
__device__ __forceinline__ float top16(const float* v) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = __builtin_fmaxf(t, __builtin_fabsf(v[j]));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) t = __builtin_fmaxf(t, __shfl_xor(t, o, 64));
    return t;
}

struct Q8Args {
    const void* x; const void* res; const float* w; uint8_t* q; float* scale; void* sum;
    int64_t M, K, KB;
    float eps;
};

// A row per G lanes (64 or 256), eight consecutive columns per lane and step, so that 16
// neighbouring lanes hold one block. NV > 0: the row fits in NV steps and stays in registers.
// NV = 0: longer rows are read again for each pass over them. Bound by memory with many rows
// (norm with residual, bf16, M 16384, K 2560, from memory: 56 us, 5.3 TB/s), by the latency of a load, the row's
// sum and a store with few (M 64: 3.9 us).
template <typename T, bool VEC, bool NORM, bool RES, int G, int NV>
__global__ void __launch_bounds__(256)
k_q8_rows(const Q8Args p) {
    constexpr int S = G * 8;                            // columns of one step
    const int lane = threadIdx.x % G;
    const int64_t row = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
    if (G == 64 && row >= p.M) return;                  // whole waves; 256-lane groups have a grid of M
    const T* x = static_cast<const T*>(p.x) + row * p.K;
    const T* res = RES ? static_cast<const T*>(p.res) + row * p.K : nullptr;
    const int64_t steps = NV ? NV : (p.K + S - 1) / S;

    float v[NV ? NV : 1][8];
    auto column = [&](int64_t k) { return k * S + 8 * lane; };
    auto load = [&](int64_t k, float* o) {
        ld8<T, VEC>(x, column(k), p.K, o);
        if constexpr (RES) {
            float r[8];
            ld8<T, VEC>(res, column(k), p.K, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += r[j];
        }
    };
    float rn = 1.0f;
    if constexpr (NV > 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k) load(k, v[k]);
#pragma unroll
        for (int k = 0; k < NV; ++k) ends8<VEC>(column(k), p.K, v[k]);
    }
    if constexpr (NORM) {
        float ss = 0.0f;
        auto squares = [&](int64_t k, const float* o) {
            float t = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) t = __builtin_fmaf(o[j], o[j], t);
            ss += column(k) < p.K ? t : 0.0f;
        };
        if constexpr (NV > 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) squares(k, v[k]);
        } else {
            for (int64_t k = 0; k < steps; ++k) {
                load(k, v[0]);
                ends8<VEC>(column(k), p.K, v[0]);
                squares(k, v[0]);
            }
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) ss += __shfl_xor(ss, o, 64);
        if constexpr (G == 256) {
            __shared__ float part[4];
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
            __syncthreads();
            ss = (part[0] + part[1]) + (part[2] + part[3]);
        }
        rn = 1.0f / __builtin_sqrtf(ss / (float)p.K + p.eps);
    }
    auto finish = [&](int64_t k, float* o) {
        const int64_t c = column(k);
        if constexpr (RES) st8<T, VEC>(static_cast<T*>(p.sum) + row * p.K, c, p.K, o);
        if constexpr (NORM) {
            float w[8];
            ld8<float, VEC>(p.w, c, p.K, w);
            ends8<VEC>(c, p.K, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = o[j] * rn * w[j];
        }
        const Q8Scale scale = q8_scale(top16(o));
        st8_q<VEC>(p.q + row * p.K, c, p.K, q8_eight<!NORM && sizeof(T) == 2>(o, scale));
        if (lane % 16 == 0 && c < p.K) p.scale[row * p.KB + c / 128] = scale.scale;
    };
    if constexpr (NV > 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k) finish(k, v[k]);
    } else {
        for (int64_t k = 0; k < steps; ++k) {
            load(k, v[0]);
            ends8<VEC>(column(k), p.K, v[0]);
            finish(k, v[0]);
        }
    }
}

// One 128 x 128 square per workgroup: 16 lanes across, the rows in turn. Lanes past the last
// row or column hold the last one instead, which leaves the largest magnitude as it is and the
// loads without branches between them. Bound by memory (10240 x 2560, bf16: 14.0 us, 5.6 TB/s,
// part of it from the last cache).
constexpr int kSquareThreads = 512;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSquareThreads)
k_q8_square(const Q8Args p) {
    constexpr int DOWN = kSquareThreads / 16, N = 128 / DOWN;
    const int cx = threadIdx.x % 16 * 8, ry = threadIdx.x / 16;
    const int64_t c = (int64_t)blockIdx.x * 128 + cx, r0 = (int64_t)blockIdx.y * 128 + ry;
    auto row = [&](int k) {
        const int64_t r = r0 + DOWN * k;
        return static_cast<const T*>(p.x) + (r < p.M ? r : p.M - 1) * p.K;
    };
    float v[N][8], top = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) ld8<T, VEC>(row(k), c, p.K, v[k]);
#pragma unroll
    for (int k = 0; k < N; ++k) ends8<VEC>(c, p.K, v[k]);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(v[k][j]));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, 64));
    __shared__ float part[kSquareThreads / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSquareThreads / 64; ++k) top = __builtin_fmaxf(top, part[k]);
    const Q8Scale scale = q8_scale(top);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t r = r0 + DOWN * k;
        const uint64_t u = q8_eight<sizeof(T) == 2>(v[k], scale);
        if (r < p.M) st8_q<VEC>(p.q + r * p.K, c, p.K, u);
    }
    if (threadIdx.x == 0) p.scale[(int64_t)blockIdx.y * p.KB + blockIdx.x] = scale.scale;
}

template <typename T, bool VEC, bool NORM, bool RES>
hipError_t launch_q8_rows(const LaunchQ8& p, const Q8Args& a) {
    hipStream_t st = static_cast<hipStream_t>(p.stream);
    // A wave per row where one step holds it (from memory, norm with residual, K 512: M 16384 13.6 us
    // in bf16 and 22.0 in fp32 against 22.9 and 27.2 with four waves, M 512 3.8 against 4.0 and 3.9) or,
    // with rows enough, two (K 768: M 16384 19.3 and 31.7 against 26.0 and 32.1, M 4096 7.2 and 11.2
    // against 8.4 and 10.9, M 1024 4.1 and 4.7 against 3.9 and 4.1). Else four waves (M 16384: K 1536 32.1 and 57.9
    // against 33.3 and 62.8, K 2560 53.1 and 97.9 against 54.2 and 105.7, K 4096 83.6 and 154 against 95.8 and
    // 167; M 1024, K 2560 6.1 and 10.1 against 7.3 and 11.6).
    const bool wave = p.K <= 512 || (p.M >= 4096 && p.K <= 1024);
    const int64_t steps = (p.K + (wave ? 512 : 2048) - 1) / (wave ? 512 : 2048);
    // a launch holds fewer than 2^32 lanes: rows past 2^22 go to launches of their own
    auto go = [&](auto kernel) {
        for (int64_t r = 0; r < p.M; r += kQ8LaunchRows) {
            Q8Args b = a;
            b.M = p.M - r < kQ8LaunchRows ? p.M - r : kQ8LaunchRows;
            b.x = static_cast<const T*>(a.x) + r * p.K;
            if (a.res) b.res = static_cast<const T*>(a.res) + r * p.K;
            if (a.sum) b.sum = static_cast<T*>(a.sum) + r * p.K;
            b.q = a.q + r * p.K;
            b.scale = a.scale + r * a.KB;
            hipLaunchKernelGGL(kernel, dim3((unsigned)(wave ? (b.M + 3) / 4 : b.M)), dim3(256), 0, st, b);
        }
    };
    if (wave) {
        if (steps <= 1) go(k_q8_rows<T, VEC, NORM, RES, 64, 1>);
        else go(k_q8_rows<T, VEC, NORM, RES, 64, 2>);
    } else {
        if (steps <= 1) go(k_q8_rows<T, VEC, NORM, RES, 256, 1>);
        else if (steps <= 2) go(k_q8_rows<T, VEC, NORM, RES, 256, 2>);
        else if (steps <= 4) go(k_q8_rows<T, VEC, NORM, RES, 256, 4>);
        else go(k_q8_rows<T, VEC, NORM, RES, 256, 0>);
    }
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t launch_q8_t(const LaunchQ8& p) {
    Q8Args a{p.x, p.res, p.w, p.q, p.scale, p.sum, p.M, p.K, (p.K + 127) / 128, p.eps};
    if (p.square) {
        hipLaunchKernelGGL((k_q8_square<T, VEC>), dim3((unsigned)a.KB, (unsigned)((p.M + 127) / 128)), dim3(kSquareThreads), 0,
                           static_cast<hipStream_t>(p.stream), a);
        return hipGetLastError();
    }
    if (!p.w) return launch_q8_rows<T, VEC, false, false>(p, a);
    return p.res ? launch_q8_rows<T, VEC, true, true>(p, a) : launch_q8_rows<T, VEC, true, false>(p, a);
}

}  // namespace selscan
