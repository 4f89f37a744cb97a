// C = A W^T for MXFP4 matrices A [n_rows, n_in] and W [n_out, n_in] (prefill:
// the activations of many tokens encoded to MXFP4), on the matrix cores' own
// microscaled form: v_mfma_scale_f32_16x16x128_f8f6f4 takes E2M1 operands and one
// E8M0 byte per lane for the 32 values that the lane holds.
#include "mx_device.h"

namespace qwg {

namespace {

// Four wavefronts, each 64 x 64 of C, operands from memory.
struct Frag {
    u32x4 c[4];
    uint32_t s;
};

template <bool WORDS>
__device__ __forceinline__ void load_frag(Frag &o, const uint8_t *codes, const uint8_t *scales,
                                          int b, int nblk) {
    if (WORDS && b + 4 <= nblk) {
        const u32x4 *p = (const u32x4 *)(codes + (int64_t)b * kMxCodeBytes);
#pragma unroll
        for (int q = 0; q < 4; ++q) o.c[q] = p[q];
        o.s = *(const uint32_t *)(scales + b);
        return;
    }
    o.s = 0x7f7f7f7fu;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        o.c[q] = u32x4{0, 0, 0, 0};
        if (b + q < nblk) {
            o.c[q] = *(const u32x4 *)(codes + (int64_t)(b + q) * kMxCodeBytes);
            o.s = (o.s & ~(255u << (8 * q))) | (uint32_t)scales[b + q] << (8 * q);
        }
    }
}

template <int Q>
__device__ __forceinline__ f32x4 product(const Frag &w, const Frag &a, f32x4 c) {
    const i32x8 x = {(int)w.c[Q][0], (int)w.c[Q][1], (int)w.c[Q][2], (int)w.c[Q][3], 0, 0, 0, 0};
    const i32x8 y = {(int)a.c[Q][0], (int)a.c[Q][1], (int)a.c[Q][2], (int)a.c[Q][3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, Q, (int)w.s, Q, (int)a.s);
}

template <int TYPE, bool WORDS>
__global__ __launch_bounds__(256) void mxfp4_matmul_kernel(MxMatmulArgs a) {
    typedef typename Elem<TYPE>::T T;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int nblk = a.n_in / kMxBlock;
    const int64_t out0 = (int64_t)blockIdx.x * 128 + (wave & 1) * 64;
    const int64_t row0 = (int64_t)blockIdx.y * 128 + (wave >> 1) * 64;
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    for (int b = g * 4; b - g * 4 < nblk; b += 16) {
        Frag w[4], x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t o = min(out0 + i * 16 + n, a.n_out - 1);
            const int64_t r = min(row0 + i * 16 + n, a.n_rows - 1);
            load_frag<WORDS>(w[i], a.w + o * nblk * kMxCodeBytes, a.w_scales + o * nblk, b, nblk);
            load_frag<WORDS>(x[i], a.a + r * nblk * kMxCodeBytes, a.a_scales + r * nblk, b, nblk);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = product<0>(w[i], x[j], acc[i][j]);
                acc[i][j] = product<1>(w[i], x[j], acc[i][j]);
                acc[i][j] = product<2>(w[i], x[j], acc[i][j]);
                acc[i][j] = product<3>(w[i], x[j], acc[i][j]);
            }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t r = row0 + j * 16 + n;
        if (r >= a.n_rows) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t o = out0 + i * 16 + g * 4 + e;
                if (o < a.n_out) ((T *)a.c)[r * a.n_out + o] = (T)acc[i][j][e];
            }
    }
}

template <int TYPE>
hipError_t launch(const MxMatmulArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.n_out + 127) / 128), (unsigned)((a.n_rows + 127) / 128));
    const bool words = a.n_in % (4 * kMxBlock) == 0 &&
                       ((uintptr_t)a.a_scales | (uintptr_t)a.w_scales) % 4 == 0;
    if (words)
        mxfp4_matmul_kernel<TYPE, true><<<grid, 256, 0, s>>>(a);
    else
        mxfp4_matmul_kernel<TYPE, false><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_matmul(const MxMatmulArgs &a, int type, hipStream_t s) {
    if (type == kF32) return launch<kF32>(a, s);
    if (type == kF16) return launch<kF16>(a, s);
    return launch<kBF16>(a, s);
}

}  // namespace qwg
