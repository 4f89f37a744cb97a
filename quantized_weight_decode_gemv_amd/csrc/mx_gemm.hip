// Y = X W^T for MXFP4 weights and 1..16 rows of fp32, fp16 or bf16 activations
// (decoding: the weights are the traffic).
//
// Every weight is exact in bf16 (two significand bits and a power of two), and
// an activation is the exact sum of one (bf16), two (fp16) or three (fp32) bf16
// parts. The matrix cores multiply the weights by the parts, one part of one
// activation row per column of the tile, and accumulate in fp32; a row's parts
// are added at the end. So a batch-1 fp32 product uses 3 of the 16 columns at no
// cost: a 16 x 512 piece of W takes 16 v_mfma_f32_16x16x32_bf16 (256 cycles)
// and 64 conversions either way, and HBM delivers its 4.3 KB to a SIMD no
// faster.
//
// A workgroup's wavefronts are wr x wk: wr groups of RT row tiles of 16 rows, wk
// wavefronts sharing each group's sum over n_in. Lane l of a wavefront takes row
// l % 16 and, of each 16 blocks of 32 weights, blocks 4(l / 16) .. +3: 64
// consecutive bytes of codes and one 32-bit word of scales. The order of the products
// within the sum is free as long as the activations follow it.
//
// Measured: 2048 -> 32000, one bf16 row (34.8 MB) 9.3-10.3 us, 3.5 TB/s, where a
// loop that only loads the same bytes takes 6.5-7.0: the start of 16 wavefronts per
// compute unit, the staged activations and the sums' meeting are the rest. 2048 ->
// 2048 fp32 4.9 us (launch, one trip to memory, the meeting). 4096 -> 14336, 11 rows
// of fp16 15.6 us: staging the 22 parts in every compute unit is 5 of them.
#include <algorithm>
#include <type_traits>

#include "mx_device.h"

namespace qwg {

namespace {

constexpr int kStepBlocks = 16;                       // blocks of a row per wavefront step
constexpr int kStep = kStepBlocks * kMxBlock;         // 512 weights
// Staged activation parts, at most (16 rows of fp32, 4096 x 14336: 37 us with 128 KB,
// 31 with 156).
constexpr int kLdsX = 156 * 1024;

// Where a wavefront takes more than kFold steps (of 16 products, each of 32 terms), its sums
// are added to a second set after every kFold of them and begin anew. One fp32 chain over
// all of a long row was off by 5.5e-5 of sum |w x| where the terms have one sign and repeat
// (65536 -> 32000; 14336 -> 70016 1.2e-5); chains of 64 products, and of up to 32 of
// those, by 1.5e-6 (2.1e-6 with 16 rows), for 0 to 1% of the time. One row tile and several
// column tiles keep one chain, of a step per chunk (16 x 14336 -> 4096 fp32 4.2e-6): there
// the second set leaves too few registers for the activations' reads, 34.2 us for 30.5.
constexpr int kFold = 4;
constexpr bool folds(int nt, int rt) { return nt == 1 || rt == 2; }

// Wavefronts of a workgroup at most: two row tiles' codes, twice (the next
// step's too), need more than the 128 registers that 16 wavefronts leave.
constexpr int kMaxWaves(int rt) { return rt == 1 ? 16 : 8; }

struct Codes {
    u32x4 c[4];
    uint32_t s;  // four E8M0 bytes
};

// A lane's 4 blocks from block `b` on; blocks from `nblk` on read as zero with scale 1.
template <bool WORDS>
__device__ __forceinline__ void load_codes(Codes &o, const uint8_t *codes, const uint8_t *scales,
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

// Eight weights (one 32-bit word of codes) as bf16, scaled.
__device__ __forceinline__ bf16x8 decode8(uint32_t c, float s) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
    return bf16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// LDS pitch in bytes of one activation part of `len` values: 16 bytes past a
// multiple of 1024, so that 16 columns' reads at one position meet no bank twice.
__device__ __host__ __forceinline__ int pitch_of(int len) { return len * 2 + 16; }

// Eight activations as they lie in memory.
template <int TYPE>
struct Unit {
    u32x4 w[TYPE == kF32 ? 2 : 1];
};

// Their bf16 parts, part p's eight values at to + p * pitch. Truncation, as
// split3, but without its test: an infinity (its remainder would be a NaN) is
// looked for in the whole unit and takes the other path.
template <int TYPE>
__device__ __forceinline__ void store_parts(uint8_t *to, int pitch, const Unit<TYPE> &u) {
    if constexpr (TYPE == kBF16) {
        *(u32x4 *)to = u.w[0];
    } else {
        constexpr int P = Elem<TYPE>::pieces;
        float v[8], top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (TYPE == kF32) v[e] = u2f(u.w[e / 4][e % 4]);
            else v[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u.w[0][e / 2] >> (e % 2 * 16)));
            top = fmaxf(top, __builtin_fabsf(v[e]));
        }
        u32x4 w[P];
        if (top == __builtin_inff()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a[3], b[3];
                split3(v[2 * j], a[0], a[1], a[2]);
                split3(v[2 * j + 1], b[0], b[1], b[2]);
#pragma unroll
                for (int p = 0; p < P; ++p) w[p][j] = a[p] | b[p] << 16;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a = v[2 * j], b = v[2 * j + 1];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    // the upper halves of a and b, and what they leave (a NaN leaves a NaN)
                    w[p][j] = __builtin_amdgcn_perm(f2u(b), f2u(a), 0x07060302u);
                    a -= u2f(f2u(a) & 0xffff0000u), b -= u2f(f2u(b) & 0xffff0000u);
                }
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) *(u32x4 *)(to + p * pitch) = w[p];
    }
}

// RT: row tiles that a wavefront takes together (one read of the activations
// for both); NT: 16-column tiles of activation parts.
template <int TYPE, int NT, int RT, bool WORDS, bool FOLD>
__global__ __launch_bounds__(kMaxWaves(RT) * 64) void mxfp4_gemm_kernel(MxGemmArgs a, int wk, int chunk) {
    typedef typename Elem<TYPE>::T T;
    constexpr int P = Elem<TYPE>::pieces;
    constexpr int kBatch = TYPE == kF32 ? 3 : 6;  // activation units a thread has on the way
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int waves = blockDim.x >> 6, wr = waves / wk;
    const int kw = wave % wk, rw = wave / wk;
    const int n = lane & 15, g = lane >> 4;
    const int nblk = a.n_in / kMxBlock;
    const uint8_t *codes[RT], *scales[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        // rows past the last one read the last one; they are not stored
        const int64_t row =
            min((((int64_t)blockIdx.x * wr + rw) * RT + r) * 16 + n, (int64_t)a.n_out - 1);
        codes[r] = a.codes + row * nblk * kMxCodeBytes;
        scales[r] = a.scales + row * nblk;
    }
    const int cols = a.batch * P;
    const int pitch = pitch_of(chunk);
    f32x4 acc[RT][NT], sum[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = sum[r][t] = f32x4{0, 0, 0, 0};
    int turns = 0;
    auto fold = [&] {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[r][t] += acc[r][t], acc[r][t] = f32x4{0, 0, 0, 0};
    };
    // a column past the last part reads some part; its sums are not used
    int col[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) col[t] = min(t * 16 + n, cols - 1) * pitch;

    for (int k0 = 0; k0 < a.n_in; k0 += chunk) {
        const int len = min(chunk, a.n_in - k0);
        const int steps = (len + kStep - 1) / kStep;
        const int units = steps * (kStep / 8), all = units * a.batch;
        // The activation rows of the chunk, eight values a unit, zero past n_in. The
        // first of them are asked for before the first two steps' weights, which
        // take longer to come.
        Unit<TYPE> v[kBatch];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int h = 0; h < kBatch; ++h) {
                const int i = i0 + h * blockDim.x, b = i / units, u = i - b * units;
                v[h] = {};
                if (i < all && u * 8 < len)
                    v[h] = *(const Unit<TYPE> *)((const T *)a.x + (int64_t)b * a.n_in + k0 + u * 8);
            }
        };
        auto put = [&](int i0) {
#pragma unroll
            for (int h = 0; h < kBatch; ++h) {
                const int i = i0 + h * blockDim.x, b = i / units, u = i - b * units;
                if (i < all) store_parts<TYPE>(lds + b * P * pitch + u * 16, pitch, v[h]);
            }
        };
        fetch(threadIdx.x);
        int st = kw;
        Codes cur[RT], next[RT];
        auto load = [&](Codes(&c)[RT], int s) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
                load_codes<WORDS>(c[r], codes[r], scales[r],
                                  k0 / kMxBlock + s * kStepBlocks + g * 4, nblk);
        };
        if (st < steps) load(cur, st);
        if (st + wk < steps) load(next, st + wk);
        if (k0) __syncthreads();
        put(threadIdx.x);
        for (int i = threadIdx.x + kBatch * blockDim.x; i < all; i += kBatch * blockDim.x) {
            fetch(i);
            put(i);
        }
        __syncthreads();
        for (; st < steps; st += wk) {
            const int at = (st * kStepBlocks + g * 4) * kMxBlock * 2;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float s[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) s[r] = e8m0((cur[r].s >> (8 * q)) & 255);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    bf16x8 w[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) w[r] = decode8(cur[r].c[q][j], s[r]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const bf16x8 x = *(const bf16x8 *)(lds + col[t] + at + q * 64 + j * 16);
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            acc[r][t] =
                                __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[r], x, acc[r][t], 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) cur[r] = next[r];
            if (st + 2 * wk < steps) load(next, st + 2 * wk);
            if (FOLD && ++turns % kFold == 0) fold();
        }
    }
    if constexpr (FOLD) fold();
    // every wavefront's sums meet in LDS: [wave][row tile][column][row]
    __syncthreads();
    float *sums = (float *)lds;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            *(f32x4 *)(sums + (((wave * RT + r) * NT + t) * 16 + n) * 16 + g * 4) = (FOLD ? sum : acc)[r][t];
    __syncthreads();
    for (int i = threadIdx.x; i < wr * RT * 16 * a.batch; i += blockDim.x) {
        const int m = i & 15, w = (i >> 4) % (wr * RT), b = (i >> 4) / (wr * RT);
        const int64_t out = ((int64_t)blockIdx.x * wr * RT + w) * 16 + m;
        if (out >= a.n_out) continue;
        float y = 0;
        // the small parts first
#pragma unroll
        for (int p = P - 1; p >= 0; --p) {
            float s = 0;
            for (int k = 0; k < wk; ++k)
                s += sums[((((w / RT) * wk + k) * RT + w % RT) * NT * 16 + b * P + p) * 16 + m];
            y += s;
        }
        ((T *)a.y)[(int64_t)b * a.n_out + out] = (T)y;
    }
}

// One workgroup of up to 16 wavefronts per compute unit: its activations are
// staged once. `tp` row tiles per workgroup, and as many wavefronts as fit
// share each tile's sum. (Two workgroups of eight per unit: 2048 -> 32000 9.5 us,
// 4096 -> 14336 10.0 against 9.6, 2048 -> 5632 fp32 5.2 against 4.9.)
constexpr int kWorkgroups = 256;

template <int TYPE, int NT, int RT>
hipError_t launch(const MxGemmArgs &a, int wr, hipStream_t s) {
    constexpr int P = Elem<TYPE>::pieces;
    const int64_t tiles = ((int64_t)a.n_out + 15) / 16;
    const int steps = (a.n_in + kStep - 1) / kStep;
    int wk = kMaxWaves(RT) / wr;
    if (wk > steps) wk = steps;
    // The steps whose activations fit LDS: all, or whole turns of the wavefronts, or
    // even parts.
    int fit = kLdsX / (a.batch * P) / 2 / kStep;
    if (fit >= steps) fit = steps;
    else if (fit > wk) fit -= fit % wk;
    else fit = (steps + (steps + fit - 1) / fit - 1) / ((steps + fit - 1) / fit);
    const int chunk = fit * kStep;
    size_t lds = (size_t)a.batch * P * pitch_of(chunk);
    const size_t join = (size_t)wk * wr * RT * NT * 16 * 16 * 4;
    if (lds < join) lds = join;
    const unsigned grid = (unsigned)((tiles + wr * RT - 1) / (wr * RT));
    const bool words = a.n_in % (4 * kMxBlock) == 0 && (uintptr_t)a.scales % 4 == 0;
    auto run = [&](auto fold) {
        if (words) mxfp4_gemm_kernel<TYPE, NT, RT, true, fold.value><<<grid, wk * wr * 64, lds, s>>>(a, wk, chunk);
        else mxfp4_gemm_kernel<TYPE, NT, RT, false, fold.value><<<grid, wk * wr * 64, lds, s>>>(a, wk, chunk);
        return hipGetLastError();
    };
    if constexpr (folds(NT, RT)) {
        // the steps of one wavefront at most: every wk-th of each chunk
        const int turns = (steps + fit - 1) / fit * ((fit + wk - 1) / wk);
        if (turns > kFold) return run(std::true_type{});
    }
    return run(std::false_type{});
}

template <int TYPE, int NT>
hipError_t launch(const MxGemmArgs &a, hipStream_t s) {
    const int64_t tiles = ((int64_t)a.n_out + 15) / 16;
    const int64_t tp = (tiles + kWorkgroups - 1) / kWorkgroups;
    // two row tiles per wavefront where the activations' LDS reads would bound it
    if constexpr (NT > 1) {
        if (tp >= 2) return launch<TYPE, NT, 2>(a, (int)std::min<int64_t>((tp + 1) / 2, kMaxWaves(2)), s);
    }
    return launch<TYPE, NT, 1>(a, (int)std::min<int64_t>(tp, kMaxWaves(1)), s);
}

}  // namespace

hipError_t launch_mxfp4_gemm(const MxGemmArgs &a, int type, hipStream_t s) {
    if (type == kF32) {
        if (a.batch * 3 <= 16) return launch<kF32, 1>(a, s);
        if (a.batch * 3 <= 32) return launch<kF32, 2>(a, s);
        return launch<kF32, 3>(a, s);
    }
    if (type == kF16) {
        if (a.batch * 2 <= 16) return launch<kF16, 1>(a, s);
        return launch<kF16, 2>(a, s);
    }
    return launch<kBF16, 1>(a, s);
}

}  // namespace qwg
