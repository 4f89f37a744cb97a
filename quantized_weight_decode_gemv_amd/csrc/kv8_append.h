// Appending to the 8-bit key/value cache, as it is (kv8.hip) or rotating keys on the way
// (kv8_rotary.hip). The layout of a page: kv8.hip.
#pragma once

#include <type_traits>

#include "mx_device.h"

namespace qwg {

namespace {

// The biased exponent of the smallest power of two s with top / s <= 448 =
// 1.75 * 2^8, `top` given as the bits of a finite magnitude.
__device__ __forceinline__ uint32_t page_exponent(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e > 0 ? (uint32_t)e : 0;
}

// Four codes of a value each, the first in the low byte. NaN and infinity become
// NaN codes.
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d, float scale) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    s16x2 v = {0, 0};
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, a, b, scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, v);
}

// The four codes of a word, times `shift`, as codes.
__device__ __forceinline__ uint32_t fp8_shifted(uint32_t w, float shift) {
    return fp8_codes(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * shift,
                     __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * shift,
                     __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * shift,
                     __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * shift, 1.0f);
}

// The largest of a workgroup's values.
template <int threads>
__device__ __forceinline__ uint32_t top_of_all(uint32_t top, uint32_t *tops) {
#pragma unroll
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < threads / 64; ++w) top = max(top, tops[w]);
    return top;
}

// Where a page's scale rises, the codes of its first `old` slots are rounded to the new one.
template <int threads>
__device__ __forceinline__ void raise_codes(uint8_t *codes, bool is_v, int old, int dim, int page,
                                            uint32_t before, uint32_t now) {
    if (!old || now <= before) return;
    const float shift = __builtin_ldexpf(1.0f, (int)before - (int)now);
    if (!is_v) {
        for (int i = threadIdx.x; i < old * dim / 4; i += threads)
            ((uint32_t *)codes)[i] = fp8_shifted(((uint32_t *)codes)[i], shift);
    } else {
        const int words = (old + 3) >> 2;
        for (int i = threadIdx.x; i < words * dim; i += threads) {
            const int ch = i / words, s = (i - ch * words) * 4;
            uint8_t *at = codes + ch * page + s;
            if (s + 4 <= old) {
                *(uint32_t *)at = fp8_shifted(*(uint32_t *)at, shift);
            } else {  // the word's other slots may be getting new codes
                for (int t = 0; s + t < old; ++t) at[t] = (uint8_t)fp8_shifted(at[t], shift);
            }
        }
    }
}

// sin and cos of 2 pi t, t in turns. A position times a frequency is exact enough in 64
// bits alone (position 10^5 at one radian each: fp32 leaves 2^-8 of a radian), and there the
// rest is cheap too: the quarter turn comes off exactly, and the Taylor sums of what is
// left, at most pi/4, end where the next term is below 2^-45.
__device__ __forceinline__ void sincos_turns(double t, double &s, double &c) {
    const double quarter = __builtin_rint(t * 4.0);
    const double x = __builtin_fma(quarter, -0.25, t) * 6.283185307179586, x2 = x * x;
    double a = 1.0 / 6227020800.0, b = -1.0 / 87178291200.0;
    a = __builtin_fma(a, x2, -1.0 / 39916800.0);
    b = __builtin_fma(b, x2, 1.0 / 479001600.0);
    a = __builtin_fma(a, x2, 1.0 / 362880.0);
    b = __builtin_fma(b, x2, -1.0 / 3628800.0);
    a = __builtin_fma(a, x2, -1.0 / 5040.0);
    b = __builtin_fma(b, x2, 1.0 / 40320.0);
    a = __builtin_fma(a, x2, 1.0 / 120.0);
    b = __builtin_fma(b, x2, -1.0 / 720.0);
    a = __builtin_fma(a, x2, -1.0 / 6.0);
    b = __builtin_fma(b, x2, 1.0 / 24.0);
    b = __builtin_fma(b, x2, -0.5);
    a = __builtin_fma(a * x2, x, x);  // sin x
    b = __builtin_fma(b, x2, 1.0);    // cos x
    const double round = quarter * 0.25;
    const int k = (int)((round - __builtin_floor(round)) * 4.0);  // quarter mod 4
    const double u = k & 1 ? b : a, w = k & 1 ? a : b;
    s = k & 2 ? -u : u;
    c = (k + 1) & 2 ? -w : w;
}

constexpr double kTurnsPerRadian = 0.15915494309189535;
// how the channels of a head pair up: not at all, the first half with the second, neighbours
constexpr int kPlain = 0, kHalves = 1, kNeighbours = 2;
constexpr int kHeadsAtOnce = 4;  // whose loads are under way together

// The channels of a thread's unit: eight from `d`, and with `two` the eight that they pair with,
// half a rotary width on.
template <int ROT>
struct Unit {
    int d;
    bool two, turns;
    __device__ __forceinline__ Unit(int u, int half, int rotary) {
        d = ROT == kHalves && u >= half / 8 ? u * 8 + half : u * 8;
        two = ROT == kHalves && d < half;
        turns = ROT == kHalves ? two : d < rotary;
    }
    static __device__ __forceinline__ int count(int dim, int half) {
        return (ROT == kHalves ? dim - half : dim) / 8;
    }
};
// angles of a unit: pair e is values (e, e + 8) of halves, (2 e, 2 e + 1) of neighbours
constexpr int pairs_of(int rot) { return rot == kHalves ? 8 : 4; }
constexpr int first_of(int rot, int e) { return rot == kHalves ? e : 2 * e; }
constexpr int second_of(int rot, int e) { return rot == kHalves ? e + 8 : 2 * e + 1; }

// The tokens of a sequence, rotated, to q_out or k_out: a.slice heads at most of one chunk
// of `page` tokens after another. A thread takes a unit of a.per_thread heads of one token
// under the same angles, which cost what four heads' loads and stores do.
template <typename T, int ROT, int threads>
__device__ __forceinline__ void rotate_rows(const T *x, int64_t x_stride, T *to, int64_t to_stride, int heads,
                                            const Kv8RotaryArgs &a, int64_t first, int64_t count, int64_t held) {
    const int dim = a.cache.dim, page = a.cache.page, half = a.rotary / 2;
    const bool vec = (((uintptr_t)x | (uintptr_t)to | (uintptr_t)x_stride * sizeof(T) |
                       (uintptr_t)to_stride * sizeof(T)) & 15) == 0;
    const int units = Unit<ROT>::count(dim, half);
    const int sets = (heads + a.per_thread - 1) / a.per_thread;
    auto load = [&](const T *p, float *v) {
        float (&w)[8] = *(float (*)[8])v;
        vec ? load8<T, true>(p, w) : load8<T, false>(p, w);
    };
    auto store = [&](T *p, const float *v) {
        const float (&w)[8] = *(const float (*)[8])v;
        vec ? store8<T, true>(p, w) : store8<T, false>(p, w);
    };
    for (int64_t i0 = (int64_t)blockIdx.x * page; i0 < count; i0 += (int64_t)gridDim.x * page) {
        const int items = (int)min((int64_t)page, count - i0) * sets * units;
        for (int i = threadIdx.x; i < items; i += threads) {
            const int u = i % units, r = i / units, set = r % sets;
            const int64_t token = i0 + r / sets;
            const Unit<ROT> unit(u, half, a.rotary);
            const T *p = x + (first + token) * x_stride + unit.d;
            T *o = to + (first + token) * to_stride + unit.d;
            const int stop = min((set + 1) * a.per_thread, heads);
            float cs[pairs_of(ROT)], sn[pairs_of(ROT)];
            if (unit.turns) {
                const double pos = (double)(held + token);
#pragma unroll
                for (int e = 0; e < pairs_of(ROT); ++e) {
                    double sd, cd;
                    sincos_turns(pos * (a.freqs[(ROT == kHalves ? unit.d : unit.d / 2) + e] * kTurnsPerRadian), sd, cd);
                    cs[e] = (float)cd, sn[e] = (float)sd;
                }
            }
            for (int h0 = set * a.per_thread; h0 < stop; h0 += kHeadsAtOnce) {
                float v[kHeadsAtOnce][16];
#pragma unroll
                for (int h = 0; h < kHeadsAtOnce; ++h)
                    if (h0 + h < stop) {
                        load(p + (h0 + h) * dim, v[h]);
                        if (unit.two) load(p + (h0 + h) * dim + half, v[h] + 8);
                    }
#pragma unroll
                for (int h = 0; h < kHeadsAtOnce; ++h)
                    if (h0 + h < stop) {
                        if (unit.turns) {
#pragma unroll
                            for (int e = 0; e < pairs_of(ROT); ++e) {
                                float &x0 = v[h][first_of(ROT, e)], &x1 = v[h][second_of(ROT, e)];
                                const float y = __builtin_fmaf(x0, cs[e], -(x1 * sn[e]));
                                x1 = __builtin_fmaf(x1, cs[e], x0 * sn[e]);
                                x0 = y;
                            }
                        }
                        store(o + (h0 + h) * dim, v[h]);
                        if (unit.two) store(o + (h0 + h) * dim + half, v[h] + 8);
                    }
            }
        }
    }
}

// A value of 64 bits rounded to fp32 such that a further rounding to few bits is that of the
// value itself: towards zero, with the last bit set where something was cut off.
__device__ __forceinline__ float odd_f32(double x) {
    const float f = (float)x;
    const double back = (double)f;
    uint32_t b = f2u(f);
    if (back != x && fabsf(f) < __builtin_inff()) b = (b - (fabs(back) > fabs(x))) | 1;
    return u2f(b);
}

// kv8_append_kernel's work on a page of K where the keys are rotated on the way: the rotated
// keys wait in LDS (a.rows of them; a page that gets more takes them in turns, twice) for the
// page's largest. In registers, four positions of sixteen channels a thread, they left
// a compute unit four wavefronts (9 prompts of up to 2000 tokens, 8 heads of 128: 103 us).
template <typename T, bool VEC, int ROT, int threads>
__device__ __forceinline__ void append_keys(const Kv8RotaryArgs &a, const T *x0, int64_t pos0, int old, int stop,
                                            uint8_t *codes, uint8_t *scale, uint32_t *tops, float *keys) {
    const int dim = a.cache.dim, half = a.rotary / 2;
    const int units = Unit<ROT>::count(dim, half);
    uint32_t top = 0;
    auto fill = [&](int begin, int end) {
        for (int i = threadIdx.x; i < (end - begin) * units; i += threads) {
            const int r = i / units, slot = begin + r;
            const Unit<ROT> unit(i - r * units, half, a.rotary);
            float v[16];
            float (&v0)[8] = *(float (*)[8])v, (&v1)[8] = *(float (*)[8])(v + 8);
            const T *p = x0 + slot * a.k_stride + unit.d;
            load8<T, VEC>(p, v0);
#pragma unroll
            for (int e = 0; e < 8; ++e) v1[e] = 0;
            if (unit.two) load8<T, VEC>(p + half, v1);
            if (unit.turns) {
                const double pos = (double)(pos0 + slot);
#pragma unroll
                for (int e = 0; e < pairs_of(ROT); ++e) {
                    double s, c;
                    sincos_turns(pos * (a.freqs[(ROT == kHalves ? unit.d : unit.d / 2) + e] * kTurnsPerRadian), s, c);
                    const double x = v[first_of(ROT, e)], y = v[second_of(ROT, e)];
                    v[first_of(ROT, e)] = odd_f32(__builtin_fma(x, c, -(y * s)));
                    v[second_of(ROT, e)] = odd_f32(__builtin_fma(y, c, x * s));
                }
            }
            float *to = keys + r * dim + unit.d;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                if (e < 8 || unit.two)
                    *(f32x4 *)(to + (e < 8 ? e : half + e - 8)) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t m = f2u(v[e]) & 0x7fffffffu;
                top = max(top, m < 0x7f800000u ? m : 0u);
            }
        }
    };
    for (int r = old; r < stop; r += a.rows) fill(r, min(r + a.rows, stop));
    top = top_of_all<threads>(top, tops);  // (and every key is in LDS)
    const uint32_t before = old ? *scale : 0;
    const uint32_t now = max(before, page_exponent(top));
    const float sc = e8m0(now);
    for (int r = old; r < stop; r += a.rows) {
        const int end = min(r + a.rows, stop);
        if (stop - old > a.rows) {
            __syncthreads();
            fill(r, end);
            __syncthreads();
        }
        for (int i = threadIdx.x; i < (end - r) * dim / 16; i += threads) {
            const f32x4 *w = (const f32x4 *)(keys + i * 16);
            u32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 v = w[e];
                x[e] = fp8_codes(v[0], v[1], v[2], v[3], sc);
            }
            *(u32x4 *)(codes + r * dim + i * 16) = x;
        }
    }
    raise_codes<threads>(codes, false, old, dim, a.cache.page, before, now);
    __syncthreads();  // every thread has read the scale, and the keys
    if (threadIdx.x == 0) *scale = (uint8_t)now;
}

// The tokens that a sequence appends.
__device__ __forceinline__ void new_tokens(const Kv8AppendArgs &a, int64_t seq, int64_t &first, int64_t &count) {
    if (a.starts) {
        first = max((int64_t)a.starts[seq], (int64_t)0);
        count = min((int64_t)a.starts[seq + 1], a.n_tokens) - first;
    } else {
        count = a.n_tokens / a.n_seqs;
        first = seq * count;
    }
}

// One slice of the heads of q, or behind those of k.
template <typename T, int ROT, int threads>
__device__ __forceinline__ void rotate_slice(const Kv8RotaryArgs &a, int slice, int64_t first, int64_t count,
                                             int64_t position) {
    const int of_q = (a.n_heads + a.slice - 1) / a.slice;
    const bool q = slice < of_q;
    const int h0 = (q ? slice : slice - of_q) * a.slice, heads = (q ? a.n_heads : a.cache.n_kv) - h0;
    const int64_t at = (int64_t)h0 * a.cache.dim;
    rotate_rows<T, ROT, threads>((const T *)(q ? a.q : a.k) + at, q ? a.q_stride : a.k_stride,
                                 (T *)(q ? a.q_out : a.k_out) + at, q ? a.q_out_stride : a.k_out_stride,
                                 min(heads, a.slice), a, first, count, position);
}

template <int ROT>
struct AppendArgs {
    typedef Kv8RotaryArgs type;
};
template <>
struct AppendArgs<kPlain> {
    typedef Kv8AppendArgs type;
};

// One workgroup per (page of a sequence, sequence, head of K or V). A thread
// takes four consecutive positions of eight channels: 8-byte stores to a K page,
// 4-byte stores (one per channel) to a transposed V page. The page's largest new
// magnitude comes first (one pass over the values, a cross-lane and an LDS step);
// a thread's last tile stays in registers meanwhile, so that a page of up to `threads`
// tiles is read once. Memory bounds it where there is much: 9 prompts of up to 2000
// tokens, 8 heads of 128, bf16 (62 MB read and written): 17.4 us, 3.5 TB/s. One token
// each of 33 sequences takes 5.4 us: the launch and four round trips in a row (length,
// page number, values, exponent).
// VEC: the values of a token start on 16 bytes.
// ROT: keys are rotated on the way, in 64 bits, so that a code is the exact key's; workgroups
// past the heads' rotate q and, where asked for, k into q_out and k_out. One launch: the
// rotation of 32 query heads beside them keeps memory busy while the keys' angles keep the vector
// units (9 prompts of up to 2000 tokens, 8 and 32 heads of 128, bf16, 273 MB: 76 us, 3.6
// TB/s; in two launches 34 and 49).
template <int TYPE, bool VEC, int threads, int ROT>
__global__ __launch_bounds__(threads) void kv8_append_kernel(typename AppendArgs<ROT>::type a) {
    typedef typename Elem<TYPE>::T T;
    __shared__ uint32_t tops[threads / 64];
    extern __shared__ __align__(16) float keys[];
    const Kv8 &c = a.cache;
    const int64_t seq = blockIdx.y;
    const int head = (int)blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int64_t held = a.lens[seq];
    int64_t first, count;
    new_tokens(a, seq, first, count);
    int64_t before = 0;
    if constexpr (ROT != kPlain) {
        if (a.before) before = a.before[0];
        if ((int)blockIdx.z >= 2 * c.n_kv) {
            rotate_slice<T, ROT, threads>(a, (int)blockIdx.z - 2 * c.n_kv, first, count, held + before);
            return;
        }
    }
    if (held < 0 || count <= 0) return;
    const T *x = (const T *)(is_v ? a.v : a.k) + (int64_t)head * c.dim;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const int64_t end = min(held + count, a.width * c.page);
    const int octs = c.dim / 8;
    for (int64_t p = held / c.page + blockIdx.x; p * c.page < end; p += gridDim.x) {
        const int64_t id = a.table[seq * a.width + p];
        if (id < 0 || id >= c.n_pages) continue;
        const int64_t pos0 = p * c.page;
        const int old = (int)max((int64_t)0, held - pos0);               // slots filled before
        const int stop = (int)min((int64_t)c.page, end - pos0);          // slots filled after
        uint8_t *codes = (is_v ? c.v : c.k) + (id * c.n_kv + head) * (int64_t)c.page * c.dim;
        uint8_t *scale = (is_v ? c.v_scales : c.k_scales) + id * c.n_kv + head;
        const T *x0 = x + (first + pos0 - held) * stride;                // token of slot 0
        if constexpr (ROT != kPlain) {
            if (!is_v) {
                append_keys<T, VEC, ROT, threads>(a, x0, before + pos0, old, stop, codes, scale, tops, keys);
                continue;
            }
        }
        // tiles: groups of four slots from the one that holds slot `old`, by channel octets;
        // neighbouring threads take neighbouring octets of K, neighbouring slots of V
        const int g0 = old >> 2, groups = ((stop + 3) >> 2) - g0, tiles = groups * octs;
        float v[4][8];
        auto load = [&](int i, int &slot, int &d) {
            const int by = is_v ? groups : octs, q = i / by, r = i - q * by;
            slot = (g0 + (is_v ? r : q)) * 4, d = (is_v ? q : r) * 8;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[t][e] = 0;
                if (slot + t >= old && slot + t < stop)
                    load8<T, VEC>(x0 + (slot + t) * stride + d, v[t]);
            }
        };
        uint32_t top = 0;
        // the last tile of a thread is loaded last, and kept for the second pass
        const int last = (int)threadIdx.x < tiles
                             ? (int)threadIdx.x + (tiles - 1 - (int)threadIdx.x) / threads * threads
                             : -1;
        int slot = 0, d = 0;
        for (int i = threadIdx.x; i < tiles; i += threads) {
            load(i, slot, d);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t m = f2u(v[t][e]) & 0x7fffffffu;
                    top = max(top, m < 0x7f800000u ? m : 0u);
                }
        }
        top = top_of_all<threads>(top, tops);
        const uint32_t before = old ? *scale : 0;
        const uint32_t now = max(before, page_exponent(top));
        const float sc = e8m0(now);
        for (int i = last; i >= 0; i -= threads) {
            if (i != last) load(i, slot, d);
            const int lo = max(old - slot, 0), hi = min(stop - slot, 4);
            if (!is_v) {
                for (int t = lo; t < hi; ++t) {
                    u32x2 w = {0, 0};
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (s == t)
                            w = u32x2{fp8_codes(v[s][0], v[s][1], v[s][2], v[s][3], sc),
                                      fp8_codes(v[s][4], v[s][5], v[s][6], v[s][7], sc)};
                    *(u32x2 *)(codes + (slot + t) * c.dim + d) = w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t w = fp8_codes(v[0][e], v[1][e], v[2][e], v[3][e], sc);
                    uint8_t *to = codes + (d + e) * c.page + slot;
                    if (lo == 0 && hi == 4) {
                        *(uint32_t *)to = w;
                    } else {
                        for (int t = lo; t < hi; ++t) to[t] = (uint8_t)(w >> (8 * t));
                    }
                }
            }
        }
        raise_codes<threads>(codes, is_v, old, c.dim, c.page, before, now);
        __syncthreads();  // every thread has read the scale
        if (threadIdx.x == 0) *scale = (uint8_t)now;
    }
}

template <int TYPE, int ROT, typename Args>
hipError_t append(const Args &a, hipStream_t s) {
    // pages that max_new tokens touch at most; a sequence with more of them takes more trips
    int64_t pages = a.max_new / a.cache.page + 2;
    if (a.max_new <= 1) pages = 1;
    if (pages > a.width) pages = a.width;
    if (pages > 4096) pages = 4096;
    int heads = a.cache.n_kv * 2;
    size_t lds = 0;
    if constexpr (ROT != kPlain) {
        lds = (size_t)a.rows * a.cache.dim * 4;  // 128 KB at most
        int slices = (a.n_heads + a.slice - 1) / a.slice;
        if (a.k_out) slices += (a.cache.n_kv + a.slice - 1) / a.slice;
        heads += slices;
    }
    const dim3 grid((unsigned)pages, (unsigned)a.n_seqs, (unsigned)heads);
    const uintptr_t size = sizeof(typename Elem<TYPE>::T);
    // (head_dim values are whole 16 bytes in every type)
    const bool vec = ((uintptr_t)a.k | (uintptr_t)a.v) % 16 == 0 &&
                     (a.n_tokens == 1 || (a.k_stride * size % 16 == 0 && a.v_stride * size % 16 == 0));
    // a thread per tile of a full page, or per two (44 prompts of up to 491 tokens on
    // pages of 16, 4 heads of 96, fp16: 32.8 us with 256 threads for the 48 tiles, 14.6
    // with 64; 34 of 44 on pages of 64, 8 heads of 192: 20.9 with 1024 for the 384, 11.5
    // with 512)
    const int tiles = a.cache.page * a.cache.dim / 32;
    auto run = [&](auto threads) {
        if (vec) kv8_append_kernel<TYPE, true, threads.value, ROT><<<grid, threads.value, lds, s>>>(a);
        else kv8_append_kernel<TYPE, false, threads.value, ROT><<<grid, threads.value, lds, s>>>(a);
    };
    if (tiles <= 64 || (ROT != kPlain && a.max_new <= 1)) run(std::integral_constant<int, 64>{});
    else if (tiles <= 256) run(std::integral_constant<int, 256>{});
    else run(std::integral_constant<int, 512>{});
    return hipGetLastError();
}

}  // namespace

}  // namespace qwg
