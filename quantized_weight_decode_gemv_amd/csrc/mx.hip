// MXFP4 (OCP Microscaling Formats v1.0: E2M1 elements, one E8M0 scale per 32
// values): encoder and decoder.
//
// encode: e = floor(log2(max |v|)) - 2, code = round-to-nearest-even of
// v / 2^e to {0, 1/2, 1, 3/2, 2, 3, 4, 6}, saturated at 6. With the biased fp32
// exponent E of the largest magnitude the stored scale is max(E - 2, 0): a
// block whose largest magnitude is below 2^-125 keeps the smallest scale
// 2^-127. A block with a NaN or an infinity has no E2M1 form: its scale is 255
// (NaN) and its codes 0.
#include <algorithm>

#include "mx_device.h"

namespace qwg {

namespace {

// A lane takes 16 bytes of values: a quarter (16-bit types) or an eighth (fp32) of
// a block, so that a wavefront's loads and stores are whole lines.
template <int TYPE>
constexpr int kVals = TYPE == kF32 ? 4 : 8;
constexpr int kUnroll = 4;  // units a lane has on the way

template <int TYPE>
struct Packed {
    typename Elem<TYPE>::T v[kVals<TYPE>];
};

template <int TYPE, bool VEC>
__device__ __forceinline__ Packed<TYPE> load_unit(const typename Elem<TYPE>::T *p) {
    if constexpr (VEC) return __builtin_bit_cast(Packed<TYPE>, *(const u32x4 *)p);
    Packed<TYPE> o;
#pragma unroll
    for (int i = 0; i < kVals<TYPE>; ++i) o.v[i] = p[i];
    return o;
}

// Memory bounds both directions: 32000 x 2048 fp32 takes 48-50 us to encode (297 MB,
// 6.0 TB/s) and 43-49 us to decode (6.0-7.0 TB/s); with a whole block per lane, whose
// loads touch 64 lines at a time, decoding took 56. Non-temporal stores, ordinary
// loads (the hint on loads too gained nothing).
//
// The block's lanes find its largest magnitude in two or three cross-lane steps;
// the hardware conversion does the division by the scale, the rounding and the
// saturation. u: the unit's number in the outputs' order.
template <int TYPE>
__device__ __forceinline__ void encode_unit(uint8_t *codes, uint8_t *scales, int64_t u,
                                            const Packed<TYPE> &x) {
    constexpr int N = kVals<TYPE>, L = kMxBlock / N;  // lanes of a block
    float v[N];
    uint32_t top = 0;  // magnitudes as bits: their order is the values', NaN above infinity
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = to_f32(x.v[i]);
        top = max(top, f2u(v[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o < L; o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    const uint32_t e = top >> 23;
    const bool none = e == 255;
    const uint32_t s = none ? 255 : e > 2 ? e - 2 : 0;
    const float scale = e8m0(none ? 127 : s);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
    if constexpr (N == 8) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
        __builtin_nontemporal_store(none ? 0 : c, (uint32_t *)codes + u);
    } else {
        __builtin_nontemporal_store((uint16_t)(none ? 0 : c), (uint16_t *)codes + u);
    }
    if (u % L == 0) scales[u / L] = (uint8_t)s;
}

// Rows back to back: the values are one run. (The lanes of a block always take
// the same path: every count is a multiple of L.)
template <int TYPE>
__global__ __launch_bounds__(256) void mxfp4_encode_kernel(uint8_t *codes, uint8_t *scales,
                                                           const typename Elem<TYPE>::T *x,
                                                           int64_t units) {
    const int64_t step = (int64_t)gridDim.x * 256 * kUnroll;
    for (int64_t u = (int64_t)blockIdx.x * 256 * kUnroll + threadIdx.x; u < units; u += step) {
        Packed<TYPE> v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (u + k * 256 < units) v[k] = load_unit<TYPE, true>(x + (u + k * 256) * kVals<TYPE>);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (u + k * 256 < units) encode_unit<TYPE>(codes, scales, u + k * 256, v[k]);
    }
}

// Rows that lie apart, or values that do not start on 16 bytes.
template <int TYPE, bool VEC>
__global__ __launch_bounds__(256) void mxfp4_encode_rows_kernel(uint8_t *codes, uint8_t *scales,
                                                                const typename Elem<TYPE>::T *x,
                                                                int64_t n_rows, int row_units,
                                                                int64_t x_stride) {
    const int u = blockIdx.x * 256 + threadIdx.x;
    if (u >= row_units) return;
    for (int64_t r = blockIdx.y; r < n_rows; r += gridDim.y)
        encode_unit<TYPE>(codes, scales, r * row_units + u,
                          load_unit<TYPE, VEC>(x + r * x_stride + (int64_t)u * kVals<TYPE>));
}

// The product of a code's value and the scale is formed in fp32, which holds it
// exactly (down to its subnormals), and rounded once where the output type is
// narrower.
template <int TYPE>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const uint8_t *codes,
                                                            const uint8_t *scales,
                                                            typename Elem<TYPE>::T *dst,
                                                            int64_t units) {
    typedef typename Elem<TYPE>::T T;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    constexpr int N = kVals<TYPE>, L = kMxBlock / N;
    const int64_t step = (int64_t)gridDim.x * 256 * kUnroll;
    for (int64_t u = (int64_t)blockIdx.x * 256 * kUnroll + threadIdx.x; u < units; u += step) {
        uint32_t c[kUnroll], e[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (u + k * 256 < units) {
                c[k] = N == 8 ? ((const uint32_t *)codes)[u + k * 256]
                              : (uint32_t)((const uint16_t *)codes)[u + k * 256];
                e[k] = scales[(u + k * 256) / L];
            }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (u + k * 256 < units) {
                const float s = e8m0(e[k]);
                Packed<TYPE> o;
                auto pair = [&](const f32x2 &p, int i) { o.v[i] = (T)(p.x * s), o.v[i + 1] = (T)(p.y * s); };
                pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 0), 0);
                pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 1), 2);
                if constexpr (N == 8) {
                    pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 2), 4);
                    pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 3), 6);
                }
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o), (u32x4 *)dst + u + k * 256);
            }
    }
}

unsigned grid_for(int64_t units) {
    const int64_t g = (units + 256 * kUnroll - 1) / (256 * kUnroll);
    return (unsigned)std::min<int64_t>(g, 1 << 20);
}

template <int TYPE>
hipError_t encode(uint8_t *codes, uint8_t *scales, const void *x, int64_t n_rows, int64_t n_in,
                  int64_t x_stride, hipStream_t s) {
    typedef typename Elem<TYPE>::T T;
    const int units = (int)(n_in / kVals<TYPE>);
    const T *p = (const T *)x;
    const bool one_run = n_rows == 1 || x_stride == n_in;
    // whole 16-byte loads where every row starts on one (n_in is whole 16 bytes)
    const bool vec = ((uintptr_t)x | (uintptr_t)(one_run ? 0 : x_stride * sizeof(T))) % 16 == 0;
    if (one_run && vec) {
        mxfp4_encode_kernel<TYPE><<<grid_for(n_rows * units), 256, 0, s>>>(codes, scales, p, n_rows * units);
        return hipGetLastError();
    }
    const dim3 grid((units + 255) / 256, (unsigned)std::min<int64_t>(n_rows, 65535));
    if (vec)
        mxfp4_encode_rows_kernel<TYPE, true><<<grid, 256, 0, s>>>(codes, scales, p, n_rows, units, x_stride);
    else
        mxfp4_encode_rows_kernel<TYPE, false><<<grid, 256, 0, s>>>(codes, scales, p, n_rows, units, x_stride);
    return hipGetLastError();
}

template <int TYPE>
hipError_t dequant(const uint8_t *codes, const uint8_t *scales, void *dst, int64_t n, hipStream_t s) {
    const int64_t units = n / kVals<TYPE>;
    mxfp4_dequant_kernel<TYPE><<<grid_for(units), 256, 0, s>>>(codes, scales, (typename Elem<TYPE>::T *)dst, units);
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
    if (type == kF32) return dequant<kF32>(codes, scales, dst, n, s);
    if (type == kF16) return dequant<kF16>(codes, scales, dst, n, s);
    return dequant<kBF16>(codes, scales, dst, n, s);
}

}  // namespace qwg
