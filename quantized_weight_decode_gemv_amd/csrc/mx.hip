// MXFP4 (OCP Microscaling Formats v1.0: E2M1 elements, one E8M0 scale per 32
// values): encoder and decoder.
//
// encode: e = floor(log2(max |v|)) - 2, code = round-to-nearest-even of
// v / 2^e to {0, 1/2, 1, 3/2, 2, 3, 4, 6}, saturated at 6. With the biased fp32
// exponent E of the largest magnitude the stored scale is max(E - 2, 0): a
// block whose largest magnitude is below 2^-125 keeps the smallest scale
// 2^-127. A block with a NaN or an infinity has no E2M1 form: its scale is 255
// (NaN) and its codes 0.
#include "mx_device.h"

namespace qwg {

namespace {

// Four lanes per block, eight values each: the four magnitudes meet in two
// cross-lane steps, and the hardware conversion does the division by the scale,
// the rounding and the saturation.
template <int TYPE, bool VEC>
__global__ __launch_bounds__(256) void mxfp4_encode_kernel(uint8_t *codes, uint8_t *scales,
                                                           const typename Elem<TYPE>::T *x,
                                                           int64_t n_rows, int row_units,
                                                           int64_t x_stride) {
    const int64_t total = n_rows * row_units;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    // every lane of a group of four takes the same trips: total is a multiple of 4
    for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < total; u += step) {
        const int64_t row = u / row_units;
        float v[8];
        load8<typename Elem<TYPE>::T, VEC>(x + row * x_stride + (u - row * row_units) * 8, v);
        uint32_t top = 0;  // magnitudes as bits: their order is the values', NaN above infinity
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, f2u(v[i]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const uint32_t e = top >> 23;
        const bool none = e == 255;
        const uint32_t s = none ? 255 : e > 2 ? e - 2 : 0;
        const float scale = e8m0(none ? 127 : s);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
        __builtin_nontemporal_store(none ? 0 : c, (uint32_t *)codes + u);
        if ((u & 3) == 0) scales[u >> 2] = (uint8_t)s;
    }
}

// Eight values per lane. The product of a code's value and the scale is formed
// in fp32, which holds it exactly (down to its subnormals), and rounded once
// where the output type is narrower.
template <int TYPE>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const uint32_t *codes,
                                                            const uint8_t *scales,
                                                            typename Elem<TYPE>::T *dst,
                                                            int64_t units) {
    typedef typename Elem<TYPE>::T T;
    typedef T t8 __attribute__((ext_vector_type(8), aligned(16)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < units; u += step) {
        const uint32_t c = codes[u];
        const float s = e8m0(scales[u >> 2]);
        const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
        const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
        const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
        t8 o;
        o[0] = (T)(p0.x * s), o[1] = (T)(p0.y * s), o[2] = (T)(p1.x * s), o[3] = (T)(p1.y * s);
        o[4] = (T)(p2.x * s), o[5] = (T)(p2.y * s), o[6] = (T)(p3.x * s), o[7] = (T)(p3.y * s);
        __builtin_nontemporal_store(o, (t8 *)dst + u);
    }
}

constexpr int64_t kMaxGrid = 1 << 20;

unsigned grid_for(int64_t units) {
    const int64_t g = (units + 255) / 256;
    return (unsigned)(g < kMaxGrid ? g : kMaxGrid);
}

template <int TYPE>
hipError_t encode(uint8_t *codes, uint8_t *scales, const void *x, int64_t n_rows, int64_t n_in,
                  int64_t x_stride, hipStream_t s) {
    typedef typename Elem<TYPE>::T T;
    const int units = (int)(n_in / 8);
    const dim3 grid(grid_for(n_rows * units));
    // whole 16-byte loads where every row starts on one
    if (((uintptr_t)x | (uintptr_t)(n_rows > 1 ? x_stride * sizeof(T) : 0)) % 16 == 0)
        mxfp4_encode_kernel<TYPE, true><<<grid, 256, 0, s>>>(codes, scales, (const T *)x, n_rows,
                                                              units, x_stride);
    else
        mxfp4_encode_kernel<TYPE, false><<<grid, 256, 0, s>>>(codes, scales, (const T *)x, n_rows,
                                                               units, x_stride);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_encode(uint8_t *codes, uint8_t *scales, const void *x, int type,
                               int64_t n_rows, int64_t n_in, int64_t x_stride, hipStream_t s) {
    if (type == kF32) return encode<kF32>(codes, scales, x, n_rows, n_in, x_stride, s);
    if (type == kF16) return encode<kF16>(codes, scales, x, n_rows, n_in, x_stride, s);
    return encode<kBF16>(codes, scales, x, n_rows, n_in, x_stride, s);
}

hipError_t launch_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, void *dst, int type,
                                int64_t n, hipStream_t s) {
    const int64_t units = n / 8;
    const dim3 grid(grid_for(units));
    const uint32_t *c = (const uint32_t *)codes;
    if (type == kF32)
        mxfp4_dequant_kernel<kF32><<<grid, 256, 0, s>>>(c, scales, (float *)dst, units);
    else if (type == kF16)
        mxfp4_dequant_kernel<kF16><<<grid, 256, 0, s>>>(c, scales, (_Float16 *)dst, units);
    else
        mxfp4_dequant_kernel<kBF16><<<grid, 256, 0, s>>>(c, scales, (__bf16 *)dst, units);
    return hipGetLastError();
}

}  // namespace qwg
