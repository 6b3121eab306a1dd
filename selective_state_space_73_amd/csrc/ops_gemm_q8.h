// Device code of the 8-bit product (ss_gemm_q8): Y[M, N] = X W^T (+ R) with
// X[m, k] = xs[m, k / 128] xq[m, k] and W[n, k] = ws[n / 128, k / 128] wq[n, k], the q e4m3.
//
// The scales are constant over blocks of 128 along k: the matrix cores sum a block's 128
// products from zero, and the vector units add the result to the running fp32 sum with its
// scale, acc += (xs ws) p. W rows are the first operand, so that a lane of a 16 x 16 result
// holds one row m of X (l % 16) and four consecutive rows n of W (4 (l / 16) + v): its block
// scale is one number.
//
// Precision of a block's sum. v_mfma_f32_16x16x128_f8f6f4 (as the older 16x16x32 fp8 form)
// adds the products of eight neighbouring k on a common exponent and drops what lies below
// 2^-13 of the largest of them (measured: a second product survives at 2^-13 and is lost at
// 2^-14 within eight k, at 2^-23 and 2^-24 further apart); normal data come out 1.5e-5 off, in
// the 2-norm. Outputs in bf16, which are rounded by 2^-9 or so anyway, take it. Outputs in
// fp32 convert the operands to bf16, which holds every e4m3 value, and take the bf16 form,
// whose products and sums keep fp32 (1e-8 off), at half the rate.
//
// Both operands are k-contiguous and a sum over k has no order of its own here, so a lane's
// 32 bytes of an operand may be any two 16-byte chunks of the block as long as both operands
// take the same two: lane l takes chunks l / 16 and l / 16 + 4 of its row.
#pragma once
#include "ops_internal.h"
#include "selscan_device.h"

namespace selscan {

typedef int gq_i8 __attribute__((ext_vector_type(8)));
typedef int gq_i4 __attribute__((ext_vector_type(4)));
typedef float gq_f4 __attribute__((ext_vector_type(4)));
typedef __bf16 gq_b8 __attribute__((ext_vector_type(8)));
typedef __bf16 gq_b2 __attribute__((ext_vector_type(2)));

// A lane's 32 bytes of one operand, as the matrix instruction of an output type takes them.
template <typename T> struct GqFrag;
template <> struct GqFrag<uint16_t> {
    gq_i8 v;
    __device__ __forceinline__ void set(gq_i4 a, gq_i4 b) { v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
    static __device__ __forceinline__ gq_f4 dot(const GqFrag& a, const GqFrag& b) {
        // operand formats 0, 0: e4m3; block exponents 0: the unscaled instruction
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, gq_f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
    }
};
template <> struct GqFrag<float> {
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
    static __device__ __forceinline__ gq_f4 dot(const GqFrag& a, const GqFrag& b) {
        gq_f4 q{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[j], b.v[j], q, 0, 0, 0);
        return q;
    }
};

struct GemmQ8Args {
    const uint8_t* xq; const float* xs; const uint8_t* wq; const float* ws;
    const void* R; void* Y0; void* Y1;
    int64_t split, M, N, K;
    int KB;                       // blocks along k
};

// Four consecutive columns n .. n + 3 of row m, n a multiple of 4.
template <typename T, bool RES>
__device__ __forceinline__ void gq_store(const GemmQ8Args& p, int64_t m, int64_t n, gq_f4 v) {
    if (m >= p.M || n >= p.N) return;
    const bool one = n >= p.split;
    const int64_t ld = one ? p.N - p.split : p.split, c = one ? n - p.split : n;
    T* y = static_cast<T*>(one ? p.Y1 : p.Y0) + m * ld + c;
    const T* r = RES ? static_cast<const T*>(p.R) + m * ld + c : nullptr;
    const bool whole = c + 4 <= ld && ((ld | p.split) & 3) == 0;      // the base is 16-byte aligned: aligned to four elements
    if (whole) {
        typedef T t4 __attribute__((ext_vector_type(4)));
        if (RES) {
            const t4 rv = *reinterpret_cast<const t4*>(r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += IO<T>::cvt(rv[j]);
        }
        t4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = IO<T>::bits(v[j]);
        *reinterpret_cast<t4*>(y) = o;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= p.N) break;
            const bool o2 = n + j >= p.split;
            const int64_t l2 = o2 ? p.N - p.split : p.split, at = m * l2 + (o2 ? n + j - p.split : n + j);
            float f = v[j];
            if (RES) f += IO<T>::ld(static_cast<const T*>(p.R) + at);
            IO<T>::st(static_cast<T*>(o2 ? p.Y1 : p.Y0) + at, f);
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup of WN x WM waves, each with 16 NF rows of W and 16 MF rows of X, the
// blocks of both staged in LDS, double buffered. Rows past the end repeat the last one, chunks
// past K are zero.
template <typename T, bool RES, int NF, int MF, int WN, int WM>
__global__ void __launch_bounds__(64 * WN * WM)
k_gemm_q8(const GemmQ8Args p, int tiles_m, int tiles_n) {
    constexpr int TN = 16 * NF * WN, TM = 16 * MF * WM, TH = 64 * WN * WM;
    constexpr int CW = TN * 8 / TH, CX = TM * 8 / TH;             // 16-byte chunks per thread and stage
    static_assert(128 % (16 * NF) == 0, "one scale of W per wave");
    __shared__ gq_i4 sW[2][TN * 8], sX[2][TM * 8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave / WM, wm = wave % WM;
    const int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
    const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TN;

    gq_i4 rw[CW], rx[CX];
    auto fetch = [&](int kb) {
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            const int idx = tid + TH * i, r = idx >> 3, ch = (idx & 7) ^ (r & 7);
            const int64_t row = n0 + r < p.N ? n0 + r : p.N - 1, k = (int64_t)kb * 128 + 16 * ch;
            rw[i] = k < p.K ? *reinterpret_cast<const gq_i4*>(p.wq + row * p.K + k) : gq_i4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < CX; ++i) {
            const int idx = tid + TH * i, r = idx >> 3, ch = (idx & 7) ^ (r & 7);
            const int64_t row = m0 + r < p.M ? m0 + r : p.M - 1, k = (int64_t)kb * 128 + 16 * ch;
            rx[i] = k < p.K ? *reinterpret_cast<const gq_i4*>(p.xq + row * p.K + k) : gq_i4{0, 0, 0, 0};
        }
    };
    auto stash = [&](int buf) {
#pragma unroll
        for (int i = 0; i < CW; ++i) sW[buf][tid + TH * i] = rw[i];
#pragma unroll
        for (int i = 0; i < CX; ++i) sX[buf][tid + TH * i] = rx[i];
    };
    const int fr = lane & 15, fc = lane >> 4;
    using Frag = GqFrag<T>;
    auto frag = [&](const gq_i4* s, int row0) {
        const int r = row0 + fr;
        Frag f;
        f.set(s[r * 8 + (fc ^ (r & 7))], s[r * 8 + ((fc + 4) ^ (r & 7))]);
        return f;
    };
    const float* xs[MF];
#pragma unroll
    for (int b = 0; b < MF; ++b) {
        const int64_t m = m0 + wm * 16 * MF + 16 * b + fr;
        xs[b] = p.xs + (m < p.M ? m : p.M - 1) * p.KB;
    }
    const int64_t nw = n0 + wn * 16 * NF;
    const float* ws = p.ws + (nw < p.N ? nw : p.N - 1) / 128 * p.KB;

    gq_f4 acc[NF][MF];
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b) acc[a][b] = gq_f4{0.f, 0.f, 0.f, 0.f};

    fetch(0);
    stash(0);
    float sc[MF];
#pragma unroll
    for (int b = 0; b < MF; ++b) sc[b] = xs[b][0] * ws[0];
    __syncthreads();
    for (int kb = 0; kb < p.KB; ++kb) {
        const int buf = kb & 1;
        const bool more = kb + 1 < p.KB;
        float nx[MF], nwv = 0.0f;
        if (more) {
            fetch(kb + 1);
#pragma unroll
            for (int b = 0; b < MF; ++b) nx[b] = xs[b][kb + 1];
            nwv = ws[kb + 1];
        }
        Frag fx[MF];
#pragma unroll
        for (int b = 0; b < MF; ++b) fx[b] = frag(sX[buf], wm * 16 * MF + 16 * b);
#pragma unroll
        for (int a = 0; a < NF; ++a) {
            const Frag fw = frag(sW[buf], wn * 16 * NF + 16 * a);
#pragma unroll
            for (int b = 0; b < MF; ++b) {
                const gq_f4 q = Frag::dot(fw, fx[b]);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[a][b][v] = __builtin_fmaf(q[v], sc[b], acc[a][b][v]);
            }
        }
        if (more) {
            stash(buf ^ 1);
#pragma unroll
            for (int b = 0; b < MF; ++b) sc[b] = nx[b] * nwv;
        }
        __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b)
            gq_store<T, RES>(p, m0 + wm * 16 * MF + 16 * b + fr, nw + 16 * a + 4 * fc, acc[a][b]);
}

// ---------------------------------------------------------------------------
// Few rows: W is read once, straight into registers. A workgroup has 16 NF rows of W and 16 MF
// rows of X; its WK waves take the blocks of k in turn and add their sums in LDS, in order.
template <typename T, bool RES, int NF, int MF, int WK>
__global__ void __launch_bounds__(64 * WK)
k_gemm_q8_thin(const GemmQ8Args p) {
    __shared__ gq_f4 part[WK][NF * MF][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fc = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NF), m0 = (int64_t)blockIdx.y * (16 * MF);
    const uint8_t* w[NF];
    const uint8_t* x[MF];
    const float* xs[MF];
#pragma unroll
    for (int a = 0; a < NF; ++a) {
        const int64_t n = n0 + 16 * a + fr;
        w[a] = p.wq + (n < p.N ? n : p.N - 1) * p.K;
    }
#pragma unroll
    for (int b = 0; b < MF; ++b) {
        const int64_t m = m0 + 16 * b + fr, at = m < p.M ? m : p.M - 1;
        x[b] = p.xq + at * p.K;
        xs[b] = p.xs + at * p.KB;
    }
    static_assert(128 % (16 * NF) == 0, "one scale of W per workgroup");
    const float* ws = p.ws + n0 / 128 * p.KB;

    gq_f4 acc[NF][MF];
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b) acc[a][b] = gq_f4{0.f, 0.f, 0.f, 0.f};

    struct Stage { gq_i4 w[NF][2], x[MF][2]; float s[MF], ws; };
    auto load = [&](int kb, Stage& s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = (int64_t)kb * 128 + 16 * (fc + 4 * h);
            const bool in = k < p.K;
#pragma unroll
            for (int a = 0; a < NF; ++a) s.w[a][h] = in ? *reinterpret_cast<const gq_i4*>(w[a] + k) : gq_i4{0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < MF; ++b) s.x[b][h] = in ? *reinterpret_cast<const gq_i4*>(x[b] + k) : gq_i4{0, 0, 0, 0};
        }
#pragma unroll
        for (int b = 0; b < MF; ++b) s.s[b] = xs[b][kb];
        s.ws = ws[kb];
    };
    auto use = [&](const Stage& s) {
        GqFrag<T> fw[NF];
#pragma unroll
        for (int a = 0; a < NF; ++a) fw[a].set(s.w[a][0], s.w[a][1]);
#pragma unroll
        for (int b = 0; b < MF; ++b) {
            GqFrag<T> fx;
            fx.set(s.x[b][0], s.x[b][1]);
            const float sc = s.s[b] * s.ws;
#pragma unroll
            for (int a = 0; a < NF; ++a) {
                const gq_f4 q = GqFrag<T>::dot(fw[a], fx);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[a][b][v] = __builtin_fmaf(q[v], sc, acc[a][b][v]);
            }
        }
    };
    // two blocks in flight
    Stage s0, s1;
    if (wave < p.KB) load(wave, s0);
    for (int kb = wave; kb < p.KB; kb += 2 * WK) {
        const bool second = kb + WK < p.KB;
        if (second) load(kb + WK, s1);
        use(s0);
        if (kb + 2 * WK < p.KB) load(kb + 2 * WK, s0);
        if (second) use(s1);
    }
#pragma unroll
    for (int a = 0; a < NF; ++a)
#pragma unroll
        for (int b = 0; b < MF; ++b) part[wave][a * MF + b][lane] = acc[a][b];
    __syncthreads();
    for (int t = wave; t < NF * MF; t += WK) {
        gq_f4 v = part[0][t][lane];
#pragma unroll
        for (int k = 1; k < WK; ++k) v += part[k][t][lane];
        const int a = t / MF, b = t % MF;
        gq_store<T, RES>(p, m0 + 16 * b + fr, n0 + 16 * a + 4 * fc, v);
    }
}

template <typename T, bool RES>
hipError_t launch_gemm_q8_t(const LaunchGemmQ8& p) {
    const GemmQ8Args a{p.xq, p.xs, p.wq, p.ws, p.R, p.Y[0], p.Y[1], p.split, p.M, p.N, p.K, (int)((p.K + 127) / 128)};
    hipStream_t st = static_cast<hipStream_t>(p.stream);
    if (p.M <= kGemmQ8ThinRows) {
        const unsigned gn = (unsigned)((p.N + 31) / 32);
        if (p.M <= 16) hipLaunchKernelGGL((k_gemm_q8_thin<T, RES, 2, 1, 8>), dim3(gn, 1), dim3(512), 0, st, a);
        else if (p.M <= 32) hipLaunchKernelGGL((k_gemm_q8_thin<T, RES, 2, 2, 4>), dim3(gn, 1), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_gemm_q8_thin<T, RES, 2, 4, 4>), dim3(gn, (unsigned)((p.M + 63) / 64)), dim3(256), 0, st, a);
    } else {
        const int tm = (int)((p.M + 127) / 128), tn = (int)((p.N + 127) / 128);
        hipLaunchKernelGGL((k_gemm_q8<T, RES, 4, 4, 2, 2>), dim3((unsigned)(tm * tn)), dim3(256), 0, st, a, tm, tn);
    }
    return hipGetLastError();
}

}  // namespace selscan
