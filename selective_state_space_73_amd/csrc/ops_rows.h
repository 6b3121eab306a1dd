// Eight values of a row at a time, for the kernels that go through rows of any length and alignment.
#pragma once
#include <stdint.h>

#include "selscan_device.h"

namespace selscan {

// VEC: rows start on 16 bytes and K is a multiple of 8. Else accesses of eight values are still
// one instruction (two for fp32), at the alignment of an element, which the memory pipeline takes
// (M 16384, K 2561, bf16, norm with residual, in the last cache: 59 us; element by element 189).
template <bool VEC> struct Q8Wide;
template <> struct Q8Wide<true> {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    typedef float f4 __attribute__((ext_vector_type(4)));
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    typedef uint64_t u8;
};
template <> struct Q8Wide<false> {
    typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef __bf16 b8 __attribute__((ext_vector_type(8), aligned(2)));
    typedef uint64_t u8 __attribute__((aligned(1)));
};

// Eight values of a row from column c on, or its last eight (K < 8 without VEC: what it has, then
// zeros): no condition between the loads of one lane. ends8 puts the lanes at the end right.
template <typename T, bool VEC>
__device__ __forceinline__ void ld8(const T* row, int64_t c, int64_t K, float* v) {
    using W = Q8Wide<VEC>;
    if (!VEC && K < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < K ? IO<T>::ld(row + c + j) : 0.0f;
        return;
    }
    const T* at = row + (c + 8 <= K ? c : K - 8);
    if constexpr (sizeof(T) == 2) {
        const typename W::u4 u = *reinterpret_cast<const typename W::u4*>(at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __builtin_bit_cast(float, u[j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, u[j] & 0xffff0000u);
        }
    } else {
        const typename W::f4 a = *reinterpret_cast<const typename W::f4*>(at), b = *reinterpret_cast<const typename W::f4*>(at + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
    }
}
// The eight values as they belong to column c: zeros past the end. With VEC only whole eights lie
// past it, which stand for nothing, and whose copies leave their block's largest magnitude as it is.
template <bool VEC>
__device__ __forceinline__ void ends8(int64_t c, int64_t K, float* v) {
    if (!VEC && K >= 8 && c + 8 > K) {
        const int by = c < K ? (int)(c + 8 - K) : 8;               // columns to move down: c's is at place `by`
#pragma unroll
        for (int s = 1; s <= 8; s *= 2)
            if (by & s) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = j + s < 8 ? v[j + s] : 0.0f;
            }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void st8(T* row, int64_t c, int64_t K, const float* v) {
    using W = Q8Wide<VEC>;
    if (c + 8 <= K) {
        if constexpr (sizeof(T) == 2) {
            typedef float f8 __attribute__((ext_vector_type(8)));
            typedef __bf16 b8 __attribute__((ext_vector_type(8)));
            f8 f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = v[j];
            *reinterpret_cast<typename W::b8*>(row + c) = __builtin_convertvector(f, b8);
        } else {
            *reinterpret_cast<typename W::f4*>(row + c) = typename W::f4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<typename W::f4*>(row + c + 4) = typename W::f4{v[4], v[5], v[6], v[7]};
        }
    } else if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < K) IO<T>::st(row + c + j, v[j]);
    }
}

}  // namespace selscan
