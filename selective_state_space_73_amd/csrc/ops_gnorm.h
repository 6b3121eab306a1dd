// Device code of the norms around a layer (ss_gnorm_fwd, ss_gnorm_bwd).
//
//   p = y / sqrt(mean_group y^2 + eps) w,  h = p silu(gate),  s = residual + scale h,
//   n = s / sqrt(mean_row s^2 + eps) w_next
//
// Bound by memory: every value is read once and kept in registers through the sums it takes part in.
// The backward makes everything again from the inputs: it reads y, gate, residual, ds and dn and writes
// three gradients, no more bytes than with anything kept. Sums over rows (of w, scale, w_next) stay in
// the registers of a workgroup that goes through many rows, and meet in a second kernel in a fixed order.
// bf16 with gate and residual: 16384 x 2560 and both norms 89 us forward, 4.7 TB/s, and 247 us with its gradients, 4.4 TB/s
// (a large copy reaches 4.9; the backward's kernel alone, under a profiler, 165 to 181); 16384 x 5120 in heads of 128 87 us, 5.8 TB/s; 64 x 2560 4 us.
#pragma once
#include "ops_layer_internal.h"
#include "ops_rows.h"

namespace selscan {

struct GnormShape { int lanes, nv, threads, rows; };     // lanes of a row, eights a lane, of a workgroup: threads, rows

// A lane has eight columns: a row of up to 128 columns is 16 lanes, of up to 512 one wave, and above that as
// many waves as it needs, with two eights a lane from 8192 on. `whole`: a row is a workgroup, whatever its length.
inline GnormShape gnorm_shape(int64_t K, bool whole) {
    if (!whole && K <= 128) return {16, 1, 256, 16};
    if (!whole && K <= 512) return {64, 1, 256, 4};
    const int nv = K <= 8192 ? 1 : 2, t = (int)((K + 512 * nv - 1) / (512 * nv)) * 64;
    return {t, nv, t, 1};
}

// Eight values of the first norm's weight, which repeats with the groups (VEC: a group is whole eights).
template <bool VEC, bool GROUPED>
__device__ __forceinline__ void gnorm_w8(const float* w, int c, int K, int group, float* v) {
    if constexpr (!GROUPED) {
        ld8<float, VEC>(w, c, K, v);
        ends8<VEC>(c, K, v);
    } else if constexpr (VEC) {
        ld8<float, true>(w, c < K ? c % group : 0, group, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < K ? w[(c + j) % group] : 0.0f;
    }
}

// A lane's value from another of its 16: moves inside the vector unit, where a shuffle through LDS takes ten times as long.
template <int CTRL>
__device__ __forceinline__ float gnorm_dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float gnorm_sum16(float v) {
    v += gnorm_dpp<0xb1>(v);                               // lane ^ 1
    v += gnorm_dpp<0x4e>(v);                               // lane ^ 2
    v += gnorm_dpp<0x141>(v);                              // the other four of eight
    return v + gnorm_dpp<0x140>(v);                        // the other eight
}
__device__ __forceinline__ float gnorm_lane(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Sums over a row's lanes of N values at once. LANES 16 or 64: within a wave; 0: over the workgroup, `lds` of 16 floats a
// value, zeros behind the last wave's; calls that follow each other use other places.
template <int N, int LANES>
__device__ __forceinline__ void gnorm_sum(float* v, float* lds) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = gnorm_sum16(v[k]);
        if (LANES != 16) v[k] = (gnorm_lane(v[k], 0) + gnorm_lane(v[k], 16)) + (gnorm_lane(v[k], 32) + gnorm_lane(v[k], 48));
    }
    if constexpr (LANES == 0) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) lds[k * 16 + (threadIdx.x >> 6)] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = gnorm_lane(gnorm_sum16(lds[k * 16 + (threadIdx.x & 15)]), 0);
    }
}

// Zeros behind the last wave's places of the six sums (no wave writes there, so no barrier).
template <int LANES>
__device__ __forceinline__ void gnorm_zero(float* lds) {
    if (LANES == 0)
        for (int i = threadIdx.x; i < 96; i += 64)
            if (threadIdx.x < 64 && (i & 15) >= (int)(blockDim.x >> 6)) lds[i] = 0.0f;
}

// For each of a lane's values, the sum over its group: the eights' sums (VEC) or the values themselves meet in
// LDS, eight lanes sum a group, and every lane reads its groups' sums. buf: K / 8 (VEC) or K floats,
// tot: a float a group. One row a workgroup.
template <bool VEC, int NV>
__device__ __forceinline__ void gnorm_groups_sum(float (*v)[8], int K, int group, float* buf, float* tot) {
    const int tid = threadIdx.x, nth = blockDim.x;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * nth + tid) * 8;
        if constexpr (VEC) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[k][j];
            if (c < K) buf[c >> 3] = s;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < K) buf[c + j] = v[k][j];
        }
    }
    __syncthreads();
    const int per = VEC ? group >> 3 : group, groups = K / group;
    for (int g0 = 0; g0 < groups; g0 += nth >> 3) {
        const int gi = g0 + (tid >> 3);
        float s = 0.0f;
        if (gi < groups)
            for (int i = tid & 7; i < per; i += 8) s += buf[gi * per + i];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor(s, o, 64);
        if (gi < groups && (tid & 7) == 0) tot[gi] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * nth + tid) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = c + j < K ? tot[VEC ? c / group : (c + j) / group] : 0.0f;
    }
    __syncthreads();
}

// Eight values as they came; converted where they are used, so that a row's loads are in flight over the one before.
// What is not there is read from somewhere that is and masked, with no branch between the loads.
template <typename T, bool VEC> struct GnormRaw {
    float x[8];
    __device__ __forceinline__ void ld(const void* base, int64_t row, int c, int K) { ld8<T, VEC>(static_cast<const T*>(base) + row * K, c, K, x); }
    __device__ __forceinline__ void get(uint32_t mask, int c, int K, float* v) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x[j]) & mask);
        ends8<VEC>(c, K, v);
    }
};
template <> struct GnormRaw<uint16_t, true> {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    u4 u;
    __device__ __forceinline__ void ld(const void* base, int64_t row, int c, int K) {
        u = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(base) + row * K + (c < K ? c : K - 8));
    }
    __device__ __forceinline__ void get(uint32_t mask, int, int, float* v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __builtin_bit_cast(float, (u[j] & mask) << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, u[j] & mask & 0xffff0000u);
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void gnorm_ld(const void* base, int64_t row, int c, int K, float* v) {
    if (base) {
        ld8<T, VEC>(static_cast<const T*>(base) + row * K, c, K, v);
        ends8<VEC>(c, K, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
}

// Weights of the columns; `none` where there are none.
template <bool VEC>
__device__ __forceinline__ void gnorm_ldp(const float* w, int c, int K, float none, float* v) {
    if (w) {
        ld8<float, VEC>(w, c, K, v);
        ends8<VEC>(c, K, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none;
    }
}

// v_exp and v_rcp, each within one step. In fp32 the exponent in two parts, since its rounding alone would be |z| 2^-24 of e^-z: what
// the product with -log2 e rounds off, and what log2 e does, come back as a factor 1 + lo ln 2 (not where e^-z is infinite). For
// bf16 gates one part does: |z| 2^-24 is a thousandth of a bf16 step at the gates whose e^-z counts at all beside a row's other
// values (|z| < 16), and the second part would cost 6% (16384 x 2560, both norms: 88.6 and 94.6 us).
template <typename T>
__device__ __forceinline__ float gnorm_sigmoid(float z) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
    const float t = z * -1.44269504088896341f, lo = __builtin_fmaf(z, -1.925963033500011e-8f, __builtin_fmaf(z, -1.44269504088896341f, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_amdgcn_rcpf(1.0f + (t < 127.0f ? __builtin_fmaf(e, lo * 0.693147180559945309f, e) : e));
}

struct GnormArgs {
    const void *y, *gate, *residual, *ds, *dn;
    const float *w, *scale, *w_next;
    void *s, *n, *dy, *dgate, *dresidual;
    float* part;
    int64_t M;
    int K, group;
    int woff;                     // the backward: where the weights lie in LDS, in floats
    int per;                      // the forward by groups: groups of a row, whose scales follow each other
    float eps;
};

template <typename T, bool VEC, int LANES, int NV, bool GROUPED, int MAXT>
__global__ void __launch_bounds__(MAXT)
k_gnorm_fwd(const GnormArgs p) {
    extern __shared__ float lds[];
    const int nl = LANES ? LANES : blockDim.x, lane = threadIdx.x % nl, K = p.K;
    const int64_t at = (int64_t)blockIdx.x * (LANES ? MAXT / LANES : 1) + threadIdx.x / nl;
    const bool there = at < p.M;
    const int64_t row = there ? at : p.M - 1;
    const float* scale = p.scale ? p.scale + row % p.per * K : nullptr;
    const bool gated = p.gate != nullptr;
    gnorm_zero<LANES>(lds);
    float y[NV][8], z[NV][8], s[NV][8], q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nl + lane) * 8;
        gnorm_ld<T, VEC>(p.y, row, c, K, y[v]);
        gnorm_ld<T, VEC>(p.gate, row, c, K, z[v]);
        gnorm_ld<T, VEC>(p.residual, row, c, K, s[v]);
    }
    if constexpr (!VEC) {
        // a row's last lane reads columns that others may write in place: not before its values are here
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) asm volatile("" : : "v"(y[v][j]), "v"(z[v][j]), "v"(s[v][j]));
    }
    float ry[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const bool in = (v * nl + lane) * 8 < K;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ry[v][j] = in ? y[v][j] * y[v][j] : 0.0f;
            q[0] += ry[v][j];
        }
    }
    if constexpr (GROUPED) {
        gnorm_groups_sum<VEC, NV>(ry, K, p.group, lds + 96, lds + 96 + (VEC ? K / 8 : K));
    } else {
        gnorm_sum<1, LANES>(q, lds);
    }
    const float inv = 1.0f / (GROUPED ? p.group : K);
    const float r1 = GROUPED ? 0.0f : 1.0f / sqrtf(q[0] * inv + p.eps);
    q[0] = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nl + lane) * 8;
        float w[8], a[8];
        gnorm_w8<VEC, GROUPED>(p.w, c, K, p.group, w);
        gnorm_ldp<VEC>(scale, c, K, 1.0f, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float act = z[v][j] * gnorm_sigmoid<T>(z[v][j]);
            const float h = y[v][j] * (GROUPED ? 1.0f / sqrtf(ry[v][j] * inv + p.eps) : r1) * w[j] * (gated ? act : 1.0f);
            s[v][j] = __builtin_fmaf(a[j], h, s[v][j]);
            if (c < K) q[0] = __builtin_fmaf(s[v][j], s[v][j], q[0]);
        }
        if (there) st8<T, VEC>(static_cast<T*>(p.s) + row * K, c, K, s[v]);
    }
    if (!p.w_next) return;
    gnorm_sum<1, LANES>(q, lds + 32);
    const float r2 = 1.0f / sqrtf(q[0] / K + p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nl + lane) * 8;
        float w[8];
        gnorm_ldp<VEC>(p.w_next, c, K, 0.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= s[v][j] * r2;
        if (there) st8<T, VEC>(static_cast<T*>(p.n) + row * K, c, K, w);
    }
}

// A lane's columns are the same in every row: their sums over rows stay in its registers, and (AHEAD) the next row is on its way while this one is worked on.
template <typename T, bool VEC, int LANES, int NV, bool GROUPED, int MAXT, bool AHEAD, int WAVES>
__global__ void __launch_bounds__(MAXT, WAVES)
k_gnorm_bwd(const GnormArgs p) {
    extern __shared__ float lds[];
    constexpr int R = LANES ? MAXT / LANES : 1;
    const int nl = LANES ? LANES : blockDim.x, own = threadIdx.x % nl, K = p.K, slot = threadIdx.x / nl;
    const int64_t step = (int64_t)gridDim.x * R;
    float sw[NV][8] = {}, sa[NV][8] = {}, sn[NV][8] = {};
    // the weights by column, zeros past the last, in LDS (NV 1): three eights more in registers spill
    constexpr bool IN_LDS = NV == 1;
    float* lw = lds + p.woff;
    const int KP = nl * 8;
    auto weights = [&](int c, int which, float* x) {
        if constexpr (IN_LDS) {
            typedef float f4 __attribute__((ext_vector_type(4)));
            const f4 a = *reinterpret_cast<const f4*>(lw + which * KP + c), b = *reinterpret_cast<const f4*>(lw + which * KP + c + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) { x[j] = a[j]; x[4 + j] = b[j]; }
        } else if (which == 0) {
            gnorm_w8<VEC, GROUPED>(p.w, c, K, p.group, x);
        } else {
            gnorm_ldp<VEC>(which == 1 ? p.scale : p.w_next, c, K, which == 1 ? 1.0f : 0.0f, x);
        }
    };
    if constexpr (IN_LDS) {
        for (int c = threadIdx.x; c < KP; c += blockDim.x) {
            lw[c] = c < K ? p.w[GROUPED ? c % p.group : c] : 0.0f;
            lw[KP + c] = c < K ? p.scale ? p.scale[c] : 1.0f : 0.0f;
            lw[2 * KP + c] = c < K && p.w_next ? p.w_next[c] : 0.0f;
        }
        __syncthreads();
    }
    const float inv = 1.0f / (GROUPED ? p.group : K), invk = 1.0f / K;
    GnormRaw<T, VEC> raw[NV][5];
    const void* const from[5] = {p.y, p.gate ? p.gate : p.y, p.residual ? p.residual : p.y, p.ds ? p.ds : p.y, p.dn ? p.dn : p.y};
    const uint32_t mask[5] = {~0u, p.gate ? ~0u : 0u, p.residual ? ~0u : 0u, p.ds ? ~0u : 0u, p.dn ? ~0u : 0u};
    const bool gated = p.gate != nullptr;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int k = 0; k < 5; ++k) raw[v][k].ld(from[k], row, (v * nl + own) * 8, K);
    };
    gnorm_zero<LANES>(lds);
    const int64_t first = (int64_t)blockIdx.x * R + slot;
    if (AHEAD && first < p.M) fetch(first);
    for (int64_t row = first; row < p.M; row += step) {
        int lane = own;                               // columns are made again for every row: kept over the loop they would spill
        asm volatile("" : "+v"(lane));
        float y[NV][8], z[NV][8], s[NV][8], ds[NV][8], dn[NV][8], ry[GROUPED ? NV : 1][8], sg[NV][8], q[2] = {0.0f, 0.0f};
        if (!AHEAD) fetch(row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nl + lane) * 8;
            raw[v][0].get(mask[0], c, K, y[v]);
            raw[v][1].get(mask[1], c, K, z[v]);
            raw[v][2].get(mask[2], c, K, s[v]);
            raw[v][3].get(mask[3], c, K, ds[v]);
            raw[v][4].get(mask[4], c, K, dn[v]);
        }
        if (AHEAD) fetch(row + step < p.M ? row + step : row);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if ((v * nl + lane) * 8 < K) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[0] = __builtin_fmaf(y[v][j], y[v][j], q[0]);
            }
        if constexpr (GROUPED) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) ry[v][j] = y[v][j] * y[v][j];
            gnorm_groups_sum<VEC, NV>(ry, K, p.group, lds + 96, lds + 96 + (VEC ? K / 8 : K));
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) ry[v][j] = 1.0f / sqrtf(ry[v][j] * inv + p.eps);
        } else {
            gnorm_sum<1, LANES>(q, lds);
        }
        const float r1 = GROUPED ? 0.0f : 1.0f / sqrtf(q[0] * inv + p.eps);
        q[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nl + lane) * 8;
            float w[8], a[8], wn[8];
            weights(c, 0, w);
            weights(c, 1, a);
            weights(c, 2, wn);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[v][j] *= GROUPED ? ry[GROUPED ? v : 0][j] : r1;                  // y normed
                sg[v][j] = gnorm_sigmoid<T>(z[v][j]);
                const float h = y[v][j] * w[j] * (gated ? z[v][j] * sg[v][j] : 1.0f);
                s[v][j] = __builtin_fmaf(a[j], h, s[v][j]);
                if (c < K) {
                    q[0] = __builtin_fmaf(s[v][j], s[v][j], q[0]);
                    q[1] = __builtin_fmaf(s[v][j], dn[v][j] * wn[j], q[1]);
                }
            }
        }
        if (p.w_next) {
            gnorm_sum<2, LANES>(q, lds + 32);
            const float r2 = 1.0f / sqrtf(q[0] * invk + p.eps), m = q[1] * invk * r2 * r2;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float wn[8];
                weights((v * nl + lane) * 8, 2, wn);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sn[v][j] = __builtin_fmaf(dn[v][j], s[v][j] * r2, sn[v][j]);
                    ds[v][j] = __builtin_fmaf(r2, dn[v][j] * wn[j] - s[v][j] * m, ds[v][j]);
                }
            }
        }
        q[0] = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nl + lane) * 8;
            if (p.dresidual) st8<T, VEC>(static_cast<T*>(p.dresidual) + row * K, c, K, ds[v]);
            float w[8], a[8];
            weights(c, 0, w);
            weights(c, 1, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float dh = ds[v][j] * a[j], pp = y[v][j] * w[j];
                const float sig = sg[v][j], silu = z[v][j] * sig, act = gated ? silu : 1.0f;
                const float dp = dh * act, h = pp * act;
                z[v][j] = dh * pp * (sig + silu * (1.0f - sig));                   // gradient of the gate
                sa[v][j] = __builtin_fmaf(ds[v][j], h, sa[v][j]);
                sw[v][j] = __builtin_fmaf(dp, y[v][j], sw[v][j]);
                s[v][j] = dp * w[j];
                dn[v][j] = c < K ? s[v][j] * y[v][j] : 0.0f;
                q[0] += dn[v][j];
            }
            if (p.dgate) st8<T, VEC>(static_cast<T*>(p.dgate) + row * K, c, K, z[v]);
        }
        if constexpr (GROUPED) {
            gnorm_groups_sum<VEC, NV>(dn, K, p.group, lds + 96, lds + 96 + (VEC ? K / 8 : K));
        } else {
            gnorm_sum<1, LANES>(q, lds + 64);
        }
        const float m1 = q[0] * inv;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nl + lane) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[v][j] = (GROUPED ? ry[GROUPED ? v : 0][j] : r1) * (s[v][j] - y[v][j] * (GROUPED ? dn[v][j] * inv : m1));
            st8<T, VEC>(static_cast<T*>(p.dy) + row * K, c, K, s[v]);
        }
        if constexpr (LANES == 0) __syncthreads();        // the next row's sums go where this one's are still read
    }
    // the workgroup's sums of columns: its rows' slots one after the other
    float* out = p.part + (int64_t)blockIdx.x * 3 * K;
    for (int turn = 0; turn < R; ++turn) {
        if (slot == turn) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = (v * nl + own) * 8 + j;
                    if (R == 1) {
                        if (c < K) { out[c] = sw[v][j]; out[K + c] = sa[v][j]; out[2 * K + c] = sn[v][j]; }
                    } else if (c < K) {
                        float* l = lds + 96;
                        l[c] = turn ? l[c] + sw[v][j] : sw[v][j];
                        l[K + c] = turn ? l[K + c] + sa[v][j] : sa[v][j];
                        l[2 * K + c] = turn ? l[2 * K + c] + sn[v][j] : sn[v][j];
                    }
                }
        }
        if (R > 1) __syncthreads();
    }
    if (R > 1)
        for (int c = threadIdx.x; c < 3 * K; c += blockDim.x) out[c] = lds[96 + c];
}

// The sums of columns over the workgroups (and w's over the groups of a row), in a fixed order: 32 columns
// by 32 slices of the terms a workgroup, eight terms of a slice in flight.
__global__ void __launch_bounds__(1024)
k_gnorm_sum(const float* part, int64_t n, int K, int group, float* dw, float* dscale, float* dw_next) {
    __shared__ double lds[32][33];
    const int cols = blockIdx.y ? K : group;
    float* out = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? dscale : dw_next;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    if (!out || (int)blockIdx.x * 32 >= cols) return;
    const unsigned per = blockIdx.y ? 1 : K / group, terms = (unsigned)n * per;
    const float* at = part + (int64_t)blockIdx.y * K + (c < cols ? c : 0);
    double s = 0.0;                                    // thousands of terms
    for (unsigned i = slice; i < terms; i += 32 * 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const unsigned t = i + 32 * k < terms ? i + 32 * k : i;
            v[k] = at[(int64_t)(t / per) * 3 * K + (int64_t)(t % per) * group];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + 32 * k < terms) s += v[k];
    }
    lds[slice][threadIdx.x & 31] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += lds[k][threadIdx.x & 31];
        out[c] = (float)s;
    }
}

// Dynamic LDS above 64 KiB is asked for (rows of thousands of columns in groups that are not whole eights).
template <typename F>
hipError_t gnorm_lds(F kernel, size_t bytes) {
    if (bytes <= 65536) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, bool VEC>
hipError_t launch_gnorm_t(const LaunchGnorm& p) {
    GnormArgs a{p.y, p.gate, p.residual, p.ds, p.dn, p.w, p.scale, p.w_next, p.s, p.n, p.dy, p.dgate, p.dresidual, p.part,
                p.M, (int)p.K, (int)p.group, 0, 1, p.eps};
    hipStream_t st = static_cast<hipStream_t>(p.stream);
    bool grouped = p.group < p.K;
    if (grouped && !p.back && !p.w_next) {
        // no sum over the row: its groups are rows of their own
        a.per = (int)(p.K / p.group);
        a.M = p.M * a.per;
        a.K = (int)p.group;
        grouped = false;
    }
    GnormShape sh = gnorm_shape(a.K, grouped);
    const size_t sums = grouped ? (size_t)((VEC ? a.K / 8 : a.K) + a.K / a.group) * 4 : 0;
    if (p.back) {
        // groups of one column in rows of just under 8192 have as many sums as values: with the weights beside them they exceed
        // a CU's LDS, and two eights a lane, which read the weights from memory, do not
        if (grouped && sh.nv == 1 && 96 * 4 + sums + 16 + (size_t)3 * sh.lanes * 8 * 4 > 160 * 1024) {
            const int t = (int)((a.K + 1023) / 1024) * 64;
            sh = {t, 2, t, 1};
        }
        a.woff = (int)((96 * 4 + (grouped ? sums : sh.rows > 1 ? (size_t)3 * a.K * 4 : 0) + 15) / 16 * 4);
        const size_t shm = (size_t)a.woff * 4 + (sh.nv == 1 ? (size_t)3 * sh.lanes * 8 * 4 : 0);
        const int64_t n = gnorm_groups(p.M, p.K);
        hipError_t e = hipSuccess;
        auto go = [&](auto kernel) {
            if ((e = gnorm_lds(kernel, shm)) == hipSuccess) hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(sh.threads), shm, st, a);
        };
        if (grouped) {
            if (sh.nv == 2) go(k_gnorm_bwd<T, VEC, 0, 2, true, 1024, false, 4>);
            else if (sh.threads > 512) go(k_gnorm_bwd<T, VEC, 0, 1, true, 1024, false, 4>);
            else go(k_gnorm_bwd<T, VEC, 0, 1, true, 512, true, 2>);
        } else if (sh.lanes == 16) go(k_gnorm_bwd<T, VEC, 16, 1, false, 256, true, 2>);
        else if (sh.rows == 4) go(k_gnorm_bwd<T, VEC, 64, 1, false, 256, true, 2>);
        else if (sh.nv == 2) go(k_gnorm_bwd<T, VEC, 0, 2, false, 1024, false, 4>);
        else if (sh.threads > 512) go(k_gnorm_bwd<T, VEC, 0, 1, false, 1024, false, 4>);
        else go(k_gnorm_bwd<T, VEC, 0, 1, false, 512, true, 2>);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_gnorm_sum, dim3((unsigned)((p.K + 31) / 32), 3), dim3(1024), 0, st, p.part, n, (int)p.K, (int)p.group, p.dw,
                           p.dscale, p.dw_next);
        return hipGetLastError();
    }
    const size_t shm = 96 * 4 + sums;
    const int64_t n = (a.M + sh.rows - 1) / sh.rows;
    if (n >= (int64_t(1) << 32) / 1024) {
        // more rows than one launch holds lanes for: in pieces
        LaunchGnorm q = p;
        const int64_t half = p.M / 2, bytes = half * p.K * (int64_t)sizeof(T);
        auto on = [&](const void* v) { return v ? static_cast<const char*>(v) + bytes : nullptr; };
        q.M = half;
        const hipError_t e = launch_gnorm_t<T, VEC>(q);
        if (e != hipSuccess) return e;
        q.M = p.M - half;
        q.y = on(p.y); q.gate = on(p.gate); q.residual = on(p.residual);
        q.s = const_cast<char*>(on(p.s)); q.n = const_cast<char*>(on(p.n));
        return launch_gnorm_t<T, VEC>(q);
    }
    hipError_t e = hipSuccess;
    auto go = [&](auto kernel) {
        if ((e = gnorm_lds(kernel, shm)) == hipSuccess) hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(sh.threads), shm, st, a);
    };
    if (grouped) {
        if (sh.nv == 2) go(k_gnorm_fwd<T, VEC, 0, 2, true, 1024>);
        else go(k_gnorm_fwd<T, VEC, 0, 1, true, 1024>);
    } else if (sh.lanes == 16) go(k_gnorm_fwd<T, VEC, 16, 1, false, 256>);
    else if (sh.rows == 4) go(k_gnorm_fwd<T, VEC, 64, 1, false, 256>);
    else if (sh.nv == 2) go(k_gnorm_fwd<T, VEC, 0, 2, false, 1024>);
    else go(k_gnorm_fwd<T, VEC, 0, 1, false, 1024>);
    return e != hipSuccess ? e : hipGetLastError();
}

}  // namespace selscan
