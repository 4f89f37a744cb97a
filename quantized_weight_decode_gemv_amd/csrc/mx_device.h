// Device helpers of the microscaled and 8-bit cache kernels: element types,
// E8M0 scales and exact splits of fp32 values into bf16 parts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_internal.h"

namespace qwg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int TYPE>
struct Elem;
template <>
struct Elem<kF32> {
    typedef float T;
    static constexpr int pieces = 3;  // bf16 parts that hold every bit of a value
};
template <>
struct Elem<kF16> {
    typedef _Float16 T;
    static constexpr int pieces = 2;
};
template <>
struct Elem<kBF16> {
    typedef __bf16 T;
    static constexpr int pieces = 1;
};

__device__ __forceinline__ float u2f(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t f2u(float v) { return __builtin_bit_cast(uint32_t, v); }

// The power of two 2^(e - 127) that the E8M0 byte e stands for; NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t e) {
    const uint32_t bits = e << 23;
    return u2f(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : bits);
}

// An fp32 value as three bf16 parts whose sum is exact: each part is the
// remainder's upper 16 bits (truncation, so no part overflows). An infinity or
// NaN goes into the first part alone.
__device__ __forceinline__ void split3(float v, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const uint32_t b = f2u(v);
    if ((b & 0x7f800000u) == 0x7f800000u) {
        hi = (b >> 16) | ((b & 0x7fffffu) ? 0x40u : 0u);
        mid = lo = 0;
        return;
    }
    hi = b >> 16;
    const float r = v - u2f(b & 0xffff0000u);
    mid = f2u(r) >> 16;
    lo = f2u(r - u2f(f2u(r) & 0xffff0000u)) >> 16;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    return (float)v;
}

// Eight values of a type from memory that is only aligned to the type (VEC =
// false) or to 16 bytes (VEC = true).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (VEC) {
        typedef T t8 __attribute__((ext_vector_type(8), aligned(16)));
        const t8 x = *(const t8 *)p;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
    }
}

// The other way, each value rounded once.
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (VEC) {
        typedef T t8 __attribute__((ext_vector_type(8), aligned(16)));
        t8 x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (T)v[i];
        *(t8 *)p = x;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = (T)v[i];
    }
}

}  // namespace qwg
