// C = A W^T for MXFP4 matrices A [n_rows, n_in] and W [n_out, n_in] (prefill:
// the activations of many tokens encoded to MXFP4), on the matrix cores' own
// microscaled form: v_mfma_scale_f32_16x16x128_f8f6f4 takes E2M1 operands and one
// E8M0 byte per lane for the 32 values that the lane holds, and accumulates in
// fp32 (65,536 operations in 16 cycles: 10 PFLOP/s on the chip).
//
// 8192 x 4096 -> 28672 (bf16 C) takes 545-565 us, 3.4-3.5 PFLOP/s. Without its stores
// (470 MB, 100 us at copy rate, which one workgroup per compute unit overlaps little)
// it takes 451, without stores and loads 371: the products alone, at the 7 PFLOP/s
// that the chip's power leaves them on random data (9.5 on zeros), would take 275.
// 509 x 2048 -> 5632: 10.2 us, launch and eight stages' latency.
//
// An output is one chain of n_in / 128 fp32 sums (the accumulators of a large tile leave no
// registers for a second set): where terms of one sign repeat it is off by 1.8e-6 of their
// sum at an n_in of 4096, 6.2e-6 at 14336, 3.3e-5 at 65536.
//
// A workgroup holds BM x BN of C and walks n_in in stages of 256: 128 bytes of
// codes and 8 of scales per row. Codes come by LDS DMA, a whole 128-byte line per
// row, into the other of two buffers; the 16-byte granules of a row
// are permuted so that a tile's operand reads meet no bank twice. Lane l takes
// the 32-value blocks 2(l/16), 2(l/16)+1 of a stage's eight: two products.
//
// Rows within a group of 64 (four 16-row tiles) are dealt so that row m of tile i
// is row 16(m/4) + 4i + m%4. The result lane's four rows in each of four tiles are
// then 16 consecutive outputs, and four tiles' scales of a lane lie in one 8-byte
// word, whose bytes the product instruction selects by itself.
#include <algorithm>

#include "mx_device.h"
#include "mx_lds.h"

namespace qwg {

namespace {

constexpr int kStageBlocks = 8;                                // blocks of a row per stage
constexpr int kStageBytes = kStageBlocks * kMxCodeBytes;       // 128

template <int Q, int I, int J>
__device__ __forceinline__ f32x4 product(u32x4 w, u32x4 a, u32x2 ws, u32x2 as, f32x4 c) {
    const i32x8 x = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 y = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        x, y, c, 4, 4, (I & 1) * 2 + Q, (int)ws[(I >> 1) & 1], (J & 1) * 2 + Q, (int)as[(J >> 1) & 1]);
}

// f(integral constant) for 0 .. N-1
template <int I>
struct Int {
    static constexpr int v = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F &&f) {
    if constexpr (I < N) {
        f(Int<I>{});
        each<N, I + 1>(f);
    }
}

// TM, TN: 16-row tiles of A and of W that a wavefront takes; WM x WN wavefronts.
template <int TYPE, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void mxfp4_matmul_kernel(MxMatmulArgs a, int row_tiles,
                                                                    int out_tiles) {
    typedef typename Elem<TYPE>::T T;
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16, R = BM + BN, W = WM * WN;
    static_assert(BM % 64 == 0 && BN % 64 == 0 && TN % 4 == 0 && R <= W * 64, "tiles");
    constexpr int kBuffer = R * kStageBytes + R * 8;  // codes [row][128], then scales
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int nblk = a.n_in / kMxBlock, stages = nblk / kStageBlocks;
    const int64_t row_bytes = (int64_t)nblk * kMxCodeBytes;

    // Workgroups go round the eight XCDs: give each a contiguous run of tiles,
    // in bands of eight row tiles, so that its L2 holds what its workgroups share.
    int row_tile, out_tile;
    {
        const int total = row_tiles * out_tiles, id = blockIdx.x;
        const int xcd = id & 7, q = total >> 3, r = total & 7;
        const int at = xcd * q + min(xcd, r) + (id >> 3);
        const int band = at / (8 * out_tiles), in = at - band * 8 * out_tiles;
        const int high = min(8, row_tiles - band * 8);
        out_tile = __builtin_amdgcn_readfirstlane(in / high);
        row_tile = __builtin_amdgcn_readfirstlane(band * 8 + in % high);
    }
    const int64_t row0 = (int64_t)row_tile * BM, out0 = (int64_t)out_tile * BN;
    const uint8_t *a_codes = a.a + row0 * row_bytes, *w_codes = a.w + out0 * row_bytes;
    const int a_last = (int)min<int64_t>(BM - 1, a.n_rows - 1 - row0);
    const int w_last = (int)min<int64_t>(BN - 1, a.n_out - 1 - out0);

    // LDS row r: A's rows, then W's. Rows past the last one read the last one.
    constexpr int ND = R / 8 / W;  // DMAs (eight rows) of a wavefront per stage
    static_assert(R % (8 * W) == 0, "whole DMAs");
    uint32_t from[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        const int r = (wave * ND + i) * 8 + (lane >> 3), gran = (lane & 7) ^ ((r & 3) | (r >> 4 & 1) << 2);
        const int at = r < BM ? min(r, a_last) : min(r - BM, w_last);
        from[i] = (uint32_t)(at * row_bytes) + gran * 16;
    }
    auto issue = [&](int s, int buf) {
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            const int r = (wave * ND + i) * 8;  // a DMA's rows are all A's or all W's
            dma16((r < BM ? a_codes : w_codes) + (int64_t)s * kStageBytes, from[i],
                  buf * kBuffer + r * kStageBytes);
        }
    };
    // a thread's row of scales: eight bytes a stage at any alignment
    const int sr = threadIdx.x;
    const bool has_row = R == W * 64 || sr < R;
    const uint8_t *scales = sr < BM ? a.a_scales + (row0 + min(sr, a_last)) * nblk
                                    : a.w_scales + (out0 + min(sr - BM, w_last)) * nblk;
    auto fetch_scales = [&](int s) {
        uint64_t v = 0;
        if (has_row) __builtin_memcpy(&v, scales + (int64_t)s * kStageBlocks, 8);
        return v;
    };
    // [64-row group][lane group][lane % 16][tile] two bytes
    auto put_scales = [&](uint64_t v, int buf) {
        uint8_t *to = lds + buf * kBuffer + R * kStageBytes + (sr >> 6) * 512 +
                      ((sr >> 4 & 3) * 4 + (sr & 3)) * 8 + (sr >> 2 & 3) * 2;
        if (has_row) {
#pragma unroll
            for (int h = 0; h < 4; ++h) *(uint16_t *)(to + h * 128) = (uint16_t)(v >> (16 * h));
        }
    };
    const int key = (n & 3) | (n >> 2 & 1) << 2;
    const int lane_row = (n >> 2) * 16 + (n & 3);
    struct LaneScales {
        u32x2 w[TN / 4], x[(TM + 3) / 4];
    };
    auto read_scales = [&](LaneScales &v, int buf) {
        const uint8_t *sc = lds + buf * kBuffer + R * kStageBytes + g * 128 + n * 8;
#pragma unroll
        for (int i = 0; i < TN / 4; ++i) v.w[i] = *(const u32x2 *)(sc + (BM / 64 + wn * (TN / 4) + i) * 512);
#pragma unroll
        for (int j = 0; j < (TM + 3) / 4; ++j) v.x[j] = *(const u32x2 *)(sc + (wm * TM / 4 + j) * 512);
        if constexpr (TM == 2) {  // half a group: its tiles are 0, 1 or 2, 3
            if (wm & 1) v.x[0][0] = v.x[0][1];
        }
        if constexpr (TM == 1) v.x[0][0] = (wm & 2 ? v.x[0][1] : v.x[0][0]) >> (wm & 1) * 16;
    };
    const uint8_t *const base_w = lds + (BM + wn * TN * 16) * kStageBytes + lane_row * kStageBytes;
    const uint8_t *const base_x = lds + (wm * TM / 4 * 64 + wm * TM % 4 * 4) * kStageBytes + lane_row * kStageBytes;
    auto read_w = [&](u32x4(&w)[TN], int buf, int q) {
        const uint8_t *p = base_w + buf * kBuffer + ((g * 2 + q) ^ key) * 16;
#pragma unroll
        for (int i = 0; i < TN; ++i) w[i] = *(const u32x4 *)(p + (i / 4 * 64 + i % 4 * 4) * kStageBytes);
    };
    auto read_x = [&](u32x4 &x, int buf, int q, int j) {
        const uint8_t *p = base_x + buf * kBuffer + ((g * 2 + q) ^ key) * 16;
        x = *(const u32x4 *)(p + (j / 4 * 64 + j % 4 * 4) * kStageBytes);
    };
    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    // A stage is 2 TM steps, each the products of one tile of A with TN of W. A
    // step's operand is asked for kAhead steps before; `mid` comes when the last
    // one has been, so that under the last steps' products the wavefronts meet,
    // the buffer takes the stage after the next, and the next stage's first
    // operands are on their way. The products touch no memory: only the
    // scheduling barriers keep them in their steps.
    constexpr int kSteps = 2 * TM, kAhead = TM < 4 ? 1 : 3, kRing = kAhead + 1;
    static_assert(kSteps % kRing == 0, "ring");
    u32x4 w0[TN], w1[TN], x[kRing];
    LaneScales cur, ahead;
    auto start = [&](int buf) {
        read_scales(ahead, buf);
        read_w(w0, buf, 0);
#pragma unroll
        for (int t = 0; t < kAhead; ++t) read_x(x[t], buf, 0, t);
    };
    auto stage = [&](int buf, auto &&mid, auto more) {
        cur = ahead;
        each<kSteps>([&](auto t) {
            constexpr int S = t.v, J = S % TM, N = S + kAhead;
            if constexpr (N < kSteps) {
                read_x(x[N % kRing], buf, N / TM, N % TM);
                if constexpr (N == TM) read_w(w1, buf, 1);
            } else {
                if constexpr (N == kSteps) {
                    mid();
                    if constexpr (more.v) read_scales(ahead, buf ^ 1), read_w(w0, buf ^ 1, 0);
                }
                if constexpr (more.v) read_x(x[N % kRing], buf ^ 1, 0, N - kSteps);
            }
            __builtin_amdgcn_sched_barrier(0);
            each<TN>([&](auto i) {
                acc[i.v][J] = product<S / TM, i.v, J>(S < TM ? w0[i.v] : w1[i.v], x[S % kRing],
                                                      cur.w[i.v / 4], cur.x[J / 4], acc[i.v][J]);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    if (stages > 0) {
        issue(0, 0);
        uint64_t next = fetch_scales(0);
        wait_vmcnt<0>();
        put_scales(next, 0);
        __syncthreads();
        if (stages > 1) {
            next = fetch_scales(1);
            issue(1, 1);
        }
        start(0);
        int s = 0;
        auto meet = [&] {  // stage s + 1 has come, stage s's buffer is free
            wait_vmcnt<0>();
            put_scales(next, (s & 1) ^ 1);
            __syncthreads();
        };
        for (; s + 2 < stages; ++s)
            stage(s & 1, [&] {
                meet();
                next = fetch_scales(s + 2);
                issue(s + 2, s & 1);
            }, Int<1>{});
        if (s + 1 < stages) {
            stage(s & 1, meet, Int<1>{});
            ++s;
        }
        stage(s & 1, [&] { __syncthreads(); }, Int<0>{});
    }
    if (const int left = nblk - stages * kStageBlocks) {
        // the last blocks: what lies past them is zero with scale 1
        for (int f = threadIdx.x; f < R * kStageBlocks; f += W * 64) {
            const int r = f >> 3, b = (f & 7) ^ ((r & 3) | (r >> 4 & 1) << 2);
            const uint8_t *p = r < BM ? a_codes + min(r, a_last) * row_bytes
                                      : w_codes + min(r - BM, w_last) * row_bytes;
            u32x4 v = {0, 0, 0, 0};
            if (b < left) v = *(const u32x4 *)(p + (int64_t)stages * kStageBytes + b * kMxCodeBytes);
            *(u32x4 *)(lds + f * 16) = v;
        }
        uint64_t v = 0x7f7f7f7f7f7f7f7full;
        for (int b = 0; has_row && b < left; ++b)
            v = (v & ~(255ull << (8 * b))) | (uint64_t)scales[stages * kStageBlocks + b] << (8 * b);
        put_scales(v, 0);
        __syncthreads();
        start(0);
        stage(0, [] {}, Int<0>{});
    }

#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const int64_t r = row0 + (wm * TM + j) / 4 * 64 + (wm * TM + j) % 4 * 4 + lane_row;
        if (r >= a.n_rows) continue;
#pragma unroll
        for (int i = 0; i < TN; i += 4) {
            // sixteen consecutive outputs
            const int64_t o = out0 + (wn * TN + i) / 4 * 64 + g * 16;
            T *to = (T *)a.c + r * a.n_out + o;
            typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
            if (o + 16 <= a.n_out) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const f32x4 v = acc[i + h][j];
                    *(t4 *)(to + h * 4) = t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
                }
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (o + h * 4 + e < a.n_out) to[h * 4 + e] = (T)acc[i + h][j][e];
            }
        }
    }
}

// Few tiles: 32 x 32 of C per workgroup, whose wavefronts share n_in. A wavefront
// takes 512 columns of the 64 rows at a time, straight from memory into the
// operands, lane l of a row's sixteen blocks 4(l/16) .. +3 (64 consecutive bytes;
// with 16 bytes of 64-byte pieces per lane group instead, 128 outputs of 32 rows of
// 8192 took 16.4 us). A compute unit alone draws 30-40 GB/s, so the smallest tile
// that the operands' form allows, on as many units as there are, is what counts.
// us here and in 64 x 128 tiles: 4096 outputs of 64 rows of 14336 18.6 and 38.3, 1024
// of 32 of 2048 5.5 and 6.3, of 512 (one wavefront's columns) 5.2 and 3.7; 4096 of 128
// of 2048 (512 tiles) 7.9 and 6.6.
constexpr int kFewWaves = 16;
constexpr int kFewMinIn = 2048;

template <int TYPE, bool WORDS>
__global__ __launch_bounds__(kFewWaves * 64) void mxfp4_matmul_few_kernel(MxMatmulArgs a) {
    typedef typename Elem<TYPE>::T T;
    __shared__ __align__(16) float sums[kFewWaves][32][32 + 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int nblk = a.n_in / kMxBlock, steps = (nblk + 15) / 16;
    const int64_t row0 = (int64_t)blockIdx.y * 32, out0 = (int64_t)blockIdx.x * 32;
    // rows past the last one read the last one
    const uint8_t *codes[4], *scales[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = i < 2 ? min(out0 + i * 16 + n, a.n_out - 1) : min(row0 + (i - 2) * 16 + n, a.n_rows - 1);
        codes[i] = (i < 2 ? a.w : a.a) + r * nblk * kMxCodeBytes;
        scales[i] = (i < 2 ? a.w_scales : a.a_scales) + r * nblk;
    }
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    for (int s = wave; s < steps; s += waves) {
        const int b = s * 16 + g * 4;
        u32x4 c[4][4];
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (WORDS && b + 4 <= nblk) {
#pragma unroll
                for (int q = 0; q < 4; ++q) c[i][q] = *(const u32x4 *)(codes[i] + (int64_t)(b + q) * kMxCodeBytes);
                e[i] = *(const uint32_t *)(scales[i] + b);
            } else {
                e[i] = 0x7f7f7f7fu;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    c[i][q] = u32x4{0, 0, 0, 0};
                    if (b + q < nblk) {
                        c[i][q] = *(const u32x4 *)(codes[i] + (int64_t)(b + q) * kMxCodeBytes);
                        e[i] = (e[i] & ~(255u << (8 * q))) | (uint32_t)scales[i][b + q] << (8 * q);
                    }
                }
            }
        }
        each<4>([&](auto q) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = product<q.v & 1, q.v / 2, q.v / 2>(c[i][q.v], c[2 + j][q.v], u32x2{e[i], 0}, u32x2{e[2 + j], 0}, acc[i][j]);
        });
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) *(f32x4 *)&sums[wave][j * 16 + n][i * 16 + g * 4] = acc[i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 32; i += blockDim.x) {
        const int r = i >> 5, o = i & 31;
        if (row0 + r >= a.n_rows || out0 + o >= a.n_out) continue;
        float v = 0;
        for (int w = 0; w < waves; ++w) v += sums[w][r][o];
        ((T *)a.c)[(row0 + r) * a.n_out + out0 + o] = (T)v;
    }
}

constexpr int64_t kUnits = 256;  // compute units

template <int TYPE>
hipError_t launch_few(const MxMatmulArgs &a, hipStream_t s) {
    const int steps = (a.n_in / kMxBlock + 15) / 16;
    const dim3 grid((unsigned)((a.n_out + 31) / 32), (unsigned)((a.n_rows + 31) / 32));
    const bool words = a.n_in % (4 * kMxBlock) == 0 && ((uintptr_t)a.a_scales | (uintptr_t)a.w_scales) % 4 == 0;
    if (words)
        mxfp4_matmul_few_kernel<TYPE, true><<<grid, std::min(steps, kFewWaves) * 64, 0, s>>>(a);
    else
        mxfp4_matmul_few_kernel<TYPE, false><<<grid, std::min(steps, kFewWaves) * 64, 0, s>>>(a);
    return hipGetLastError();
}

template <int TYPE, int TM, int TN, int WM, int WN>
hipError_t launch(const MxMatmulArgs &a, hipStream_t s) {
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    const int64_t rt = (a.n_rows + BM - 1) / BM, ot = (a.n_out + BN - 1) / BN;
    constexpr size_t lds = 2 * (BM + BN) * (kStageBytes + 8);
    mxfp4_matmul_kernel<TYPE, TM, TN, WM, WN>
        <<<(unsigned)(rt * ot), WM * WN * 64, lds, s>>>(a, (int)rt, (int)ot);
    return hipGetLastError();
}

template <int TYPE>
hipError_t launch(const MxMatmulArgs &a, hipStream_t s) {
    // The largest tile that keeps five eighths of the compute units busy in every round
    // (us in 256 x 256, 128 x 128, 64 x 128 and 64 x 64 tiles: 3606 x 2016 -> 3162, 195
    // large tiles, 27.0, 30.6, 34.3, 39.3; 2048 x 4096 -> 4096, 128 of them, 34.9, 27.0,
    // 34.3, 39.6; 509 x 2048 -> 5632, 176 of 128 x 128, 19.3, 10.1, 11.2, 10.8), and the
    // smallest where there is at most one to a unit (140 x 5568 -> 2875: 43.4, 21.6,
    // 21.2, 13.5; 200 x 14336 -> 4096: 88.4, 43.3, 39.0, 32.2).
    auto tiles = [&](int64_t m, int64_t n) {
        return ((a.n_rows + m - 1) / m) * ((a.n_out + n - 1) / n);
    };
    if (a.n_in >= kFewMinIn && tiles(32, 32) <= kUnits) return launch_few<TYPE>(a, s);
    if (tiles(64, 64) <= kUnits) return launch<TYPE, 1, 4, 4, 1>(a, s);
    const int64_t large = tiles(256, 256), rounds = (large + kUnits - 1) / kUnits;
    if (large * 8 >= rounds * kUnits * 5) return launch<TYPE, 8, 4, 2, 4>(a, s);
    if (tiles(128, 128) * 8 >= kUnits * 5) return launch<TYPE, 4, 4, 2, 2>(a, s);
    return launch<TYPE, 2, 4, 2, 2>(a, s);
}

}  // namespace

hipError_t launch_mxfp4_matmul(const MxMatmulArgs &a, int type, hipStream_t s) {
    if (type == kF32) return launch<kF32>(a, s);
    if (type == kF16) return launch<kF16>(a, s);
    return launch<kBF16>(a, s);
}

}  // namespace qwg
