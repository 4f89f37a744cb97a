// What the kernels of attention over the 8-bit cache share (kv8.hip, kv8_shared.hip).
#pragma once

#include "mx_device.h"

namespace qwg {

namespace {

constexpr int kBlk = 64;          // positions a wavefront takes at once
constexpr int kMaxChunk = 4096;   // positions of a split, at most
constexpr int kMaxPages = (kMaxChunk + kBlk) / 16 + 1;
constexpr int kPageBytes = (kMaxPages * 8 + 15) & ~15;

// Bytes of a word that hold a NaN code, as 0x80 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Two fp32 values' upper halves in one word, the first one's low.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
    return __builtin_amdgcn_perm(f2u(b), f2u(a), 0x07060302u);
}

// Two fp32 values rounded to bf16 (nearest, ties to even) in one word, the first one low.
__device__ __forceinline__ uint32_t nearest_halves(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Floats of one split's partial result: rows of D sums, then a (maximum, total)
// pair per row, in whole 16 bytes.
__device__ __host__ __forceinline__ int64_t partial_floats(int64_t rows, int dim) {
    return (rows * (dim + 2) + 3) & ~(int64_t)3;
}

}  // namespace

}  // namespace qwg
