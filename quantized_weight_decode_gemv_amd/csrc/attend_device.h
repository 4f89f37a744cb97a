// Device helpers of attention on 32 x 32 tiles of scores (prompt.hip, kv8_shared.hip): a lane
// holds sixteen scores of one row, and the lane 32 on (or back) the row's other sixteen.
#pragma once

#include "mx_device.h"

namespace qwg {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Two fp32 values rounded to fp16 (HALF) or bf16 (nearest, ties to even) in one word.
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (HALF) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// 32 x 32 outputs of 16 products each from two operands of eight fp16 (HALF) or bf16 values a lane.
template <bool HALF>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (HALF)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// One instruction; a NaN stays one.
__device__ __forceinline__ float maximum3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

__device__ __forceinline__ float max_halves(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(f2u(v), f2u(v), false, false);
    return __builtin_elementwise_maximum(u2f(a[0]), u2f(a[1]));
}

__device__ __forceinline__ float sum_halves(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(f2u(v), f2u(v), false, false);
    return u2f(a[0]) + u2f(a[1]);
}

// N products whose first operands come from LDS, `ahead` of them on the way: `read(i)` is the i-th
// operand (READS LDS instructions), `use(i, operand)` its EACH products. The order is laid down: left to
// itself the compiler reads each operand just before its product and waits for LDS every time.
template <int N, int READS, int EACH, typename Read, typename Use>
__device__ __forceinline__ void products(Read read, Use use) {
    constexpr int A = N < 4 ? N : 4;
    u32x4 ring[A];
#pragma unroll
    for (int i = 0; i < A; ++i) ring[i] = read(i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        use(i, ring[i % A]);
        if (i + A < N) ring[i % A] = read(i + A);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, A * READS, 0);  // LDS reads
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, EACH, 0);  // matrix products
        if (i + A < N) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    }
}

constexpr int kSlack = 8;  // a maximum may grow by this many powers of two before sums shrink

// Where a row of a tile in LDS holds its 16-byte granule c: c ^ key, so that the granules that
// sixteen lanes read at once, one of each of sixteen rows, lie in all of the 256 bytes that LDS
// gives (for rows of 16 granules a multiple, of 8, and of 12).
template <int GRANULES>
__device__ __forceinline__ int row_key(int row) {
    return GRANULES % 16 == 0 ? row & 15 : GRANULES % 8 == 0 ? row >> 1 & 7 : row >> 2 & 3;
}

}  // namespace

}  // namespace qwg
