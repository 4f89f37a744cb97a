// An 8-bit key/value cache in pages: append (encode new tokens into their
// pages) and attend (single-token or few-token attention over it).
//
// A page holds `page` positions of one sequence. Per page and key/value head
// there is one E8M0 scale for K and one for V, the smallest power of two that
// brings every magnitude of the page to 448 or less, so that no value saturates;
// values are e4m3. K pages are [n_kv][page][dim]; V pages are transposed,
// [n_kv][dim][page]: attention's second product sums over positions, and with
// consecutive positions of a channel in consecutive bytes both products take
// their operands from memory as they lie.
#include <algorithm>
#include <type_traits>

#include "mx_device.h"
#include "mx_lds.h"

namespace qwg {

namespace {

// ------------------------------------------------------------------- append

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
template <int TYPE, bool VEC, int threads>
__global__ __launch_bounds__(threads) void kv8_append_kernel(Kv8AppendArgs a) {
    typedef typename Elem<TYPE>::T T;
    __shared__ uint32_t tops[threads / 64];
    const Kv8 &c = a.cache;
    const int64_t seq = blockIdx.y;
    const int head = (int)blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int64_t held = a.lens[seq];
    int64_t first, count;
    if (a.starts) {
        first = max((int64_t)a.starts[seq], (int64_t)0);
        count = min((int64_t)a.starts[seq + 1], a.n_tokens) - first;
    } else {
        count = a.n_tokens / a.n_seqs;
        first = seq * count;
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
#pragma unroll
        for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < threads / 64; ++w) top = max(top, tops[w]);
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
        if (old && now > before) {
            // the page's scale rises: its earlier codes are rounded to the new one
            const float shift = __builtin_ldexpf(1.0f, (int)before - (int)now);
            if (!is_v) {
                for (int i = threadIdx.x; i < old * c.dim / 4; i += threads)
                    ((uint32_t *)codes)[i] = fp8_shifted(((uint32_t *)codes)[i], shift);
            } else {
                const int words = (old + 3) >> 2;
                for (int i = threadIdx.x; i < words * c.dim; i += threads) {
                    const int ch = i / words, s = (i - ch * words) * 4;
                    uint8_t *at = codes + ch * c.page + s;
                    if (s + 4 <= old) {
                        *(uint32_t *)at = fp8_shifted(*(uint32_t *)at, shift);
                    } else {  // the word's other slots may be getting new codes
                        for (int t = 0; s + t < old; ++t) at[t] = (uint8_t)fp8_shifted(at[t], shift);
                    }
                }
            }
        }
        __syncthreads();  // every thread has read the scale
        if (threadIdx.x == 0) *scale = (uint8_t)now;
    }
}

// ------------------------------------------------------------------- attend

// Eight e4m3 codes (two words) as bf16, exact.
__device__ __forceinline__ bf16x8 fp8x8(uint32_t a, uint32_t b) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf16x8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

constexpr int kBlk = 64;          // positions a wavefront takes at once
constexpr int kMaxChunk = 4096;   // positions of a split, at most
constexpr int kMaxPages = (kMaxChunk + kBlk) / 16 + 1;
constexpr int kPageBytes = (kMaxPages * 8 + 15) & ~15;

// Bytes of a word that hold a NaN code, as 0x80 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// The largest of the four lanes' values with the same lane % 16, without LDS.
__device__ __forceinline__ float max_groups(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(f2u(v), f2u(v), false, false);
    v = fmaxf(u2f(a[0]), u2f(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(f2u(v), f2u(v), false, false);
    return fmaxf(u2f(b[0]), u2f(b[1]));
}

// Two fp32 values' upper halves in one word, the first one's low.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
    return __builtin_amdgcn_perm(f2u(b), f2u(a), 0x07060302u);
}

// Two fp32 values rounded to bf16 (nearest, ties to even) in one word, the first one low.
__device__ __forceinline__ uint32_t nearest_halves(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// The block of positions that the first row's window starts in: what some row
// sees is from there to the end, and the splits begin there.
__device__ __forceinline__ int first_seen(int len, int q_len, int window) {
    return window > 0 ? max(0, len - q_len + 1 - window) & -kBlk : 0;
}

// Floats of one split's partial result: rows of D sums, then a (maximum, total)
// pair per row, in whole 16 bytes.
__device__ __host__ __forceinline__ int64_t partial_floats(int64_t rows, int dim) {
    return (rows * (dim + 2) + 3) & ~(int64_t)3;
}

// LDS of an attention workgroup: Q parts, the split's pages, then per wavefront a
// block's K and V (V of 96 channels on 16-token pages takes padded rows).
constexpr int q_bytes(int type, int d, int r) {
    return r * (d / 32) * (type == kF32 ? 3 : type == kF16 ? 2 : 1) * 1024;
}
constexpr int k_zone(int d) { return d * kBlk; }
constexpr int v_zone(int d) { return (d == 96 ? 128 : d) * kBlk; }
// Wavefronts of a workgroup: four, two such workgroups to a compute unit (one's
// start and end then overlap the other's middle); eight for two tiles of 128
// channels, whose Q would not fit twice; three or four for two of 256, as LDS
// holds. Eight where every workgroup has a compute unit to itself and takes a
// whole sequence (one of 517 positions, 4 heads of 64: 10.0 us with four, 8.3 with
// eight, 8.7 with sixteen); two, and so more workgroups at once, where short
// sequences are many (100 of up to 200 positions, 8 heads of 256: 33.0 us with four,
// 25.6 with two; of up to 86, 8 of 128: 13.3 and 9.1).
constexpr int waves_of(int d, int r, int type) {
    return d == 128 && r == 2 ? 8 : d == 256 && r == 2 && type != kBF16 ? 3 : 4;
}

// One workgroup: one split (`chunk` positions) of one sequence, one key/value
// head, R tiles of 16 rows; a row is a (query token, head of the group) pair.
//
// A wavefront takes 64 positions at a time. S^T = K Q^T: the K operand's row m of
// tile u (u = 0..3) is position 16(m/4) + 4u + m%4, so that lane l's sixteen
// results, column l%16, are the scores of one row at the consecutive positions
// 16(l/16) .. +15. They are the B operand of O^T = V^T P^T as they stand: the
// A operand's lane takes the same sixteen positions of channel l%16, sixteen
// consecutive bytes of the transposed V page. No value crosses lanes but the
// row maxima.
//
// K and V come by LDS DMA in the order of memory (four lanes to 64 bytes where
// the page has them: read straight into the operands' lanes every 16 bytes were
// an access of their own, and the L1 bound the kernel at 4 TB/s), the 16-byte
// granules of a line permuted so that the operands' reads meet no bank twice. A
// block's K is asked for as soon as the block before has read its own, V
// likewise.
//
// It is bound by memory where the cache is long: 32 ragged sequences of up to 8192
// positions, 8 heads of 128, four queries' heads each (324 MB): 58.9 us and 4.6 to
// join the splits, 5.1 TB/s (a large copy reaches 4.7); one of 131,071, 4 tokens of 64
// heads: 52-54 us and 4.6. A short call is bound by its chain of round trips (length,
// page numbers, exponents, K and V, the sums' meeting): 8.2 us for 517 positions.
// Asking for the first K and V before the exponents took a barrier more and 0.3-0.9
// us more.
//
// Queries and probabilities enter as bf16 parts (one to three) that hold all
// their bits, or the nearest value of two parts for the 16-bit types' probabilities (off by
// 2^-17 of it at most); e4m3 is exact in bf16.
//
// ONCE: this workgroup takes all rows of its key/value head, whose lines are then
// read once (with the hint 32 ragged sequences of up to 8192 positions took 60 us,
// without it 68; three row tiles, which share the lines, 61 and 56).
template <int TYPE, int D, int R, int W, bool ONCE>
__global__ __launch_bounds__(W * 64) void kv8_attend_kernel(Kv8AttendArgs a) {
    typedef typename Elem<TYPE>::T T;
    constexpr int PQ = Elem<TYPE>::pieces;      // parts of a query
    constexpr int PP = TYPE == kF32 ? 3 : 2;    // parts of a probability
    constexpr int KS = D / 32;                  // steps of the first product
    constexpr int DT = D / 16;                  // channel tiles of the second
    constexpr int C = D / 16;                   // 16-byte granules of a K row
    constexpr int NK = D / 16;                  // DMAs (1 KB) of a block's K
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const Kv8 &c = a.cache;
    const int group = a.n_heads / c.n_kv;
    const int rows = a.q_len * group;
    const int64_t seq = blockIdx.z;
    const int tiles = (rows + 16 * R - 1) / (16 * R);
    const int head = (int)blockIdx.y / tiles, row0 = (int)blockIdx.y % tiles * 16 * R;
    const int shift = __builtin_ctz(c.page);
    const int len0 = a.lens[seq], cap = (int)a.width << shift;
    const bool bad = len0 < 0 || len0 > cap;  // no such length: the rows become NaN
    const int len = bad ? 0 : len0;
    const int window = (int)min(a.window, (int64_t)1 << 30);  // 0: all
    const int low = first_seen(len, a.q_len, window);
    const int splits = max(1, (len - low + a.chunk - 1) / a.chunk);
    const int split = blockIdx.x;
    if (split >= splits) return;
    const int begin = low + split * a.chunk, end = min(begin + a.chunk, len);

    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t *const q_lds = lds;
    // the split's pages: number (-1: no page of the pool), exponents of K and V
    uint2 *const pages = (uint2 *)(lds + q_bytes(TYPE, D, R));
    const uint32_t zone = q_bytes(TYPE, D, R) + kPageBytes + wave * (k_zone(D) + v_zone(D));
    uint8_t *const k_lds = lds + zone, *const v_lds = k_lds + k_zone(D);
    const int first_page = begin >> shift;
    for (int i = threadIdx.x; i < kMaxPages; i += W * 64) {
        const int pos = (first_page + i) << shift;
        uint2 e = {0, 0x7f7f};  // past the end: any page does, its codes are masked
        if (pos < end) {
            const int id = a.table[seq * a.width + first_page + i];
            if (id < 0 || id >= c.n_pages) {
                e.x = ~0u;
            } else {
                const int64_t at = (int64_t)id * c.n_kv + head;
                e.x = id, e.y = c.k_scales[at] | (uint32_t)c.v_scales[at] << 8;
            }
        }
        pages[i] = e;
    }
    // Q parts: [tile][step][part][lane] 16 bytes, as the lanes take them
    {
        const T *q = (const T *)a.q;
        const bool vec = ((uintptr_t)q | (uintptr_t)a.q_stride * sizeof(T)) % 16 == 0;
        for (int i = threadIdx.x; i < R * KS * 64; i += W * 64) {
            const int l = i & 63, ks = (i >> 6) % KS, r = (i >> 6) / KS;
            const int row = row0 + r * 16 + (l & 15), lg = l >> 4;
            // a pair of steps takes 64 channels, 16 consecutive ones per lane
            // group; an odd last step 32, 8 per lane group
            const int d = (D % 64 && ks == KS - 1) ? ks * 32 + lg * 8
                                                   : (ks >> 1) * 64 + lg * 16 + (ks & 1) * 8;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (row < rows) {
                const int t = row / group, h = head * group + row % group;
                const T *p = q + (seq * a.q_len + t) * a.q_stride + (int64_t)h * D + d;
                vec ? load8<T, true>(p, v) : load8<T, false>(p, v);
            }
            uint32_t w[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t h0, m0, l0, h1, m1, l1;
                split3(v[2 * j], h0, m0, l0);
                split3(v[2 * j + 1], h1, m1, l1);
                w[0][j] = h0 | h1 << 16, w[1][j] = m0 | m1 << 16, w[2][j] = l0 | l1 << 16;
            }
#pragma unroll
            for (int p = 0; p < PQ; ++p)
                *(u32x4 *)(q_lds + (((r * KS + ks) * PQ + p) * 64 + l) * 16) =
                    u32x4{w[p][0], w[p][1], w[p][2], w[p][3]};
        }
    }
    __syncthreads();

    const float to_log2 = a.scale * 1.4426950408889634f;
    float top[R], sum[R];
    f32x4 out[R][DT];
    int last[R];  // the last position that this lane's row sees
#pragma unroll
    for (int r = 0; r < R; ++r) {
        top[r] = -__builtin_inff();
        sum[r] = 0;
#pragma unroll
        for (int t = 0; t < DT; ++t) out[r][t] = f32x4{0, 0, 0, 0};
        const int row = row0 + r * 16 + n;
        last[r] = row < rows ? len - a.q_len + row / group : -1;
    }
    const int64_t head_bytes = (int64_t)c.page * D;
    auto page_at = [&](int pos) { return pages[(pos >> shift) - first_page]; };
    auto page_base = [&](const uint8_t *p, int pos) {
        return p + ((int64_t)max((int)page_at(pos).x, 0) * c.n_kv + head) * head_bytes;
    };

    // K in LDS: granule s of row r (a position of the block) holds granule s ^
    // key(r) of the row: eight lanes of a tile's reads (rows 16a + 4u + b, two a
    // and four b) then meet eight different 16-byte banks.
    auto k_key = [](int b, int a1) {
        if constexpr (D % 128 == 0) return b | a1 << 2;
        else if constexpr (D == 96) return a1;
        else return b >> 1 | a1 << 1;
    };
    auto dma = [](const uint8_t *p, uint32_t to) { ONCE ? dma16_once(p, to) : dma16(p, to); };
    auto issue_k = [&](int b0) {
        const uint8_t *base[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            base[q] = page_base(c.k, b0 + q * 16) + ((b0 + q * 16) & (c.page - 1)) * D;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int f = i * 64 + lane, r = f / C, s = f - r * C;
            const int q0 = i * 64 / (16 * C), q1 = (i * 64 + 63) / (16 * C);
            const uint8_t *p = q0 == q1 || f < q1 * 16 * C ? base[q0] : base[q1];
            dma(p + (r & 15) * D + (s ^ k_key(r & 3, (r >> 4) & 1)) * 16, zone + i * 1024);
        }
    };
    // V in LDS: [16-position pieces that lie in other pages][channel][pieces of
    // one page row], `pg` pieces of a row side by side, permuted like K's.
    const int pg_log = min(shift - 4, 2), pg = 1 << pg_log;
    const int v_runs = (D * pg + 63) / 64;  // DMAs of one page row's pieces
    const int v_piece = lane & (pg - 1);
    auto issue_v = [&](int b0) {
        const int d0 = lane >> pg_log;
        const int piece = pg_log == 2 ? v_piece ^ (d0 >> 1 & 3) : pg_log == 1 ? v_piece ^ (d0 >> 2 & 1) : 0;
        uint32_t to = zone + k_zone(D);
        for (int o = 0; o < 4 >> pg_log; ++o) {
            const int pos = b0 + (o * pg + piece) * 16;
            const uint8_t *p = page_base(c.v, pos) + (pos & (c.page - 1));
            for (int i = 0; i < v_runs; ++i, to += 1024) {
                const int d = min(d0 + i * (64 >> pg_log), D - 1);
                dma(p + d * c.page, to);
            }
        }
    };
    // waits: V's DMAs are the younger ones when K is needed, the next K's when V is
    auto wait_k = [&] {
        if (D == 96 && pg == 1) wait_vmcnt<8>();
        else wait_vmcnt<D / 16>();
    };
    const int key = k_key(n & 3, (n >> 2) & 1);
    const uint8_t *const k_row = k_lds + ((n >> 2) * 16 + (n & 3)) * D;
    const int v_key = pg_log == 2 ? n >> 1 & 3 : pg_log == 1 ? n >> 2 & 1 : 0;
    const uint8_t *const v_row = v_lds + (g >> pg_log) * v_runs * 1024 +
                                 ((n << pg_log) + ((g & (pg - 1)) ^ v_key)) * 16;

    int b0 = begin + wave * kBlk;
    if (b0 < end) {
        issue_k(b0);
        issue_v(b0);
    }
    for (; b0 < end; b0 += W * kBlk) {
        const int vpos = b0 + g * 16, next = b0 + W * kBlk;
        wait_k();
        u32x4 kc[4][D / 64];
        u32x2 kt[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                kc[u][j] = *(const u32x4 *)(k_row + u * 4 * D + ((j * 4 + g) ^ key) * 16);
            if constexpr (D % 64 != 0)
                kt[u] = *(const u32x2 *)(k_row + u * 4 * D + ((D / 64 * 4 + (g >> 1)) ^ key) * 16 + (g & 1) * 8);
        }
        const uint2 page = page_at(vpos);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // K is in registers
        if (next < end) issue_k(next);

        f32x4 s[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[r][u] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const bool odd = D % 64 != 0 && k == KS - 1;
            bf16x8 kv[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                kv[u] = odd ? fp8x8(kt[u][0], kt[u][1])
                            : fp8x8(kc[u][k >> 1][(k & 1) * 2], kc[u][k >> 1][(k & 1) * 2 + 1]);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int p = PQ - 1; p >= 0; --p) {
                    const bf16x8 q = *(const bf16x8 *)(q_lds + (((r * KS + k) * PQ + p) * 64 + lane) * 16);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        s[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv[u], q, s[r][u], 0, 0, 0);
                }
        }

        const bool lost = (int)page.x < 0;  // this lane's sixteen positions have no page
        float ks = e8m0(page.y & 255) * to_log2;
        const float vs = e8m0(page.y >> 8 & 255);
        if (lost) ks = __builtin_nanf("");
        // every row sees the whole block, or the rows' masks decide
        const bool whole = b0 + kBlk <= len - a.q_len + 1 && (window <= 0 || b0 >= len - window);
        uint32_t seen[R];  // of this lane's sixteen positions, which lie in one page
#pragma unroll
        for (int r = 0; r < R; ++r) seen[r] = 0xffffu;
        if (!whole) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int hi = last[r] - vpos;
                const int lo = window > 0 ? max(0, hi - window + 1) : 0;
                uint32_t m = hi < 0 ? 0u : hi >= 15 ? 0xffffu : (2u << hi) - 1u;
                m &= lo >= 16 ? 0u : 0xffffu << lo;
                seen[r] = m;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float m = -__builtin_inff();
#pragma unroll
            for (int u = 0; u < 4; ++u) s[r][u] *= ks;
            if (!whole) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(seen[r] >> (u * 4 + i) & 1)) s[r][u][i] = -__builtin_inff();
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = fmaxf(m, s[r][u][i]);
            m = max_groups(m);
            if (__any(m > top[r])) {  // a new maximum in some row: what was summed shrinks
                const float now = fmaxf(top[r], m);
                const float alpha = now == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top[r] - now);
                top[r] = now;
                sum[r] *= alpha;
#pragma unroll
                for (int t = 0; t < DT; ++t) out[r][t] *= alpha;
            }
            const float base = top[r] == -__builtin_inff() ? 0.0f : top[r];
            f32x4 part = {0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][u][i] = __builtin_amdgcn_exp2f(s[r][u][i] - base);
                part += s[r][u];
            }
            sum[r] += (part[0] + part[1]) + (part[2] + part[3]);
        }
        // p * vs as bf16 parts: never infinite (p <= 1, vs a power of two), and a NaN stays
        // one. Two parts are each rounded to nearest, which leaves 2^-17 of p, as often up
        // as down; cut off they left up to 2^-15, and outputs too small by 2^-17 of
        // themselves, the sum of the probabilities being whole. Three hold every bit; for
        // the 16-bit types they cost more than outputs of 8 or 11 bits show (32 x 8192, bf16:
        // 64.6 us for 63.4, and 0.6e-5 off the rounded exact result for 5.1e-5, a plain fp32
        // softmax being 4.5e-5 off; 131,071 x 4 tokens: 65.0 us for 60.3).
        u32x4 pp[R][2][PP];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a page that the row does not see counts for nothing: not even its
                    // scale may (0 times a NaN scale is NaN)
                    const float f = seen[r] ? vs : 1.0f;
                    const float p0 = s[r][k * 2 + i / 2][i % 2 * 2] * f;
                    const float p1 = s[r][k * 2 + i / 2][i % 2 * 2 + 1] * f;
                    const uint32_t w = PP == 2 ? nearest_halves(p0, p1) : upper_halves(p0, p1);
                    const float r0 = p0 - u2f(w << 16), r1 = p1 - u2f(w & 0xffff0000u);
                    pp[r][k][0][i] = w;
                    if constexpr (PP == 2) {
                        pp[r][k][1][i] = nearest_halves(r0, r1);
                    } else {
                        pp[r][k][1][i] = upper_halves(r0, r1);
                        pp[r][k][2][i] = upper_halves(r0 - u2f(f2u(r0) & 0xffff0000u),
                                                      r1 - u2f(f2u(r1) & 0xffff0000u));
                    }
                }

        if (next < end) wait_vmcnt<NK>();
        else wait_vmcnt<0>();
        u32x4 vc[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t) vc[t] = *(const u32x4 *)(v_row + (t << pg_log) * 256);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // V is in registers
        if (next < end) issue_v(next);
        // a NaN in V that some rows see and others do not must reach the former alone
        if (!whole) {
            // codes past the end are whatever the pool held: none of them may
            // reach the product
            const int keep = min(max(len - vpos, 0), 16);
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int k = keep - w * 4;
                const uint32_t m = k >= 4 ? ~0u : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    vc[t][w] &= m;
                    any |= nan_bytes(vc[t][w]);
                }
            }
            if (__any(any != 0)) {
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    u32x4 flags;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t nb = nan_bytes(vc[t][w]) >> 7;  // 1 per NaN byte
                        flags[w] = nb * 0x38u;                          // e4m3 1.0
                        vc[t][w] &= ~(nb * 0xffu);
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        f32x4 hit = {0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            bf16x8 see;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                see[i] = (__bf16)(seen[r] >> (k * 8 + i) & 1 ? 1.0f : 0.0f);
                            hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                fp8x8(flags[k * 2], flags[k * 2 + 1]), see, hit, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (hit[i] > 0) out[r][t][i] = __builtin_nanf("");
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bf16x8 v = fp8x8(vc[t][k * 2], vc[t][k * 2 + 1]);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int p = PP - 1; p >= 0; --p)
                        out[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            v, __builtin_bit_cast(bf16x8, pp[r][k][p]), out[r][t], 0, 0, 0);
            }
    }

    // join the wavefronts: [wave][row][D] sums, then their maxima and totals
    __syncthreads();
    constexpr int RP = D + 4;  // row pitch: four floats past a multiple of 32 banks
    float *so = (float *)lds;
    float *sm = so + W * R * 16 * RP;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float t = sum[r];
        t += __shfl_xor(t, 16);
        t += __shfl_xor(t, 32);
        const int row = wave * R * 16 + r * 16 + n;
        if (g == 0) sm[row * 2] = top[r], sm[row * 2 + 1] = t;
#pragma unroll
        for (int d = 0; d < DT; ++d) *(f32x4 *)(so + row * RP + d * 16 + g * 4) = out[r][d];
    }
    __syncthreads();
    const int64_t row_base = seq * a.q_len;
    const int64_t all = (int64_t)a.q_len * a.n_heads;
    float *part = a.partial + (seq * a.max_splits + split) * partial_floats(all, D);
    for (int i = threadIdx.x; i < R * 16 * (D / 4); i += W * 64) {
        const int d = i % (D / 4) * 4, lr = i / (D / 4), row = row0 + lr;
        if (row >= rows) continue;
        float m = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, sm[(w * R * 16 + lr) * 2]);
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float total = 0;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[(w * R * 16 + lr) * 2] - base);
            total += f * sm[(w * R * 16 + lr) * 2 + 1];
            o += f * *(const f32x4 *)(so + (w * R * 16 + lr) * RP + d);
        }
        const int t = row / group, h = head * group + row % group;
        if (splits == 1) {
            T *dst = (T *)a.out + ((row_base + t) * a.n_heads + h) * D + d;
            const float inv = bad ? __builtin_nanf("") : 1.0f / total;
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = (T)(total == 0 && !bad ? 0.0f : o[e] * inv);
        } else {
            const int64_t at = (int64_t)t * a.n_heads + h;
            *(f32x4 *)(part + at * D + d) = o;
            if (d == 0) part[all * D + at * 2] = m, part[all * D + at * 2 + 1] = total;
        }
    }
}

// Joins the splits of a sequence: one workgroup per (query token, head), its
// wavefronts taking the splits in turn. 4.6 us for 32 x 32 rows of 128 channels in
// up to nine splits (5 MB at most, from the last-level cache), most of it the launch
// and two round trips; in this launch and not in the last workgroup to end, so that
// no counter has to be cleared and the order of the sums is fixed.
template <int TYPE, int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8AttendArgs a) {
    typedef typename Elem<TYPE>::T T;
    constexpr int V = D / 4;   // lanes that hold one row, four channels each
    constexpr int S = 64 / V;  // splits that a wavefront reads at once
    __shared__ float sums[4 * S][D + 1];
    __shared__ float red[2][4];
    const int64_t seq = blockIdx.y;
    const int row = blockIdx.x;  // token * n_heads + head
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int len0 = a.lens[seq];
    const int len = len0 < 0 || len0 > a.width * a.cache.page ? 0 : len0;
    const int low = first_seen(len, a.q_len, (int)min(a.window, (int64_t)1 << 30));
    const int splits = max(1, (len - low + a.chunk - 1) / a.chunk);
    if (splits == 1) return;
    const int64_t rows = (int64_t)a.q_len * a.n_heads, each = partial_floats(rows, D);
    const float *part = a.partial + seq * a.max_splits * each;
    const float *ml = part + rows * D + row * 2;
    float m = -__builtin_inff();
    for (int s = threadIdx.x; s < splits; s += 256) m = fmaxf(m, ml[s * each]);
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (lane == 0) red[0][wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float total = 0;
    for (int s = threadIdx.x; s < splits; s += 256)
        total += __builtin_amdgcn_exp2f(ml[s * each] - base) * ml[s * each + 1];
#pragma unroll
    for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o);
    if (lane == 0) red[1][wave] = total;
    f32x4 o = {0, 0, 0, 0};
    const int sub = lane / V, d = lane % V * 4;
    if (sub < S) {
        for (int s = wave * S + sub; s < splits; s += 4 * S)
            o += __builtin_amdgcn_exp2f(ml[s * each] - base) *
                 *(const f32x4 *)(part + s * each + (int64_t)row * D + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave * S + sub][d + e] = o[e];
    }
    __syncthreads();
    total = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    for (int d = threadIdx.x; d < D; d += 256) {
        float o = 0;
#pragma unroll
        for (int s = 0; s < 4 * S; ++s) o += sums[s][d];
        ((T *)a.out)[(seq * rows + row) * D + d] = (T)(total == 0 ? 0.0f : o / total);
    }
}

template <int TYPE, int D, int R, int W = waves_of(D, R, TYPE)>
hipError_t attend(const Kv8AttendArgs &a, hipStream_t s) {
    if constexpr (W == waves_of(D, R, TYPE)) {
        if (a.brief) return attend<TYPE, D, R, 2>(a, s);
    }
    if constexpr (D <= 128 && W == 4) {
        if (a.few) return attend<TYPE, D, R, 8>(a, s);
    }
    const int rows = a.q_len * (a.n_heads / a.cache.n_kv);
    const int tiles = (rows + 16 * R - 1) / (16 * R);
    constexpr size_t work = q_bytes(TYPE, D, R) + kPageBytes + W * (k_zone(D) + v_zone(D));
    constexpr size_t join = (size_t)W * R * 16 * (D + 4 + 2) * 4;
    static_assert(work <= 160 * 1024 && join <= 160 * 1024, "LDS");
    const dim3 grid(a.max_splits, a.cache.n_kv * tiles, (unsigned)a.n_seqs);
    const size_t lds = work > join ? work : join;
    if constexpr (R == 1 && D <= 128) {  // (16 rows at most)
        kv8_attend_kernel<TYPE, D, R, W, true><<<grid, W * 64, lds, s>>>(a);
    } else if constexpr (R == 2 && D > 128) {  // (more than 32)
        kv8_attend_kernel<TYPE, D, R, W, false><<<grid, W * 64, lds, s>>>(a);
    } else {
        if (tiles == 1)
            kv8_attend_kernel<TYPE, D, R, W, true><<<grid, W * 64, lds, s>>>(a);
        else
            kv8_attend_kernel<TYPE, D, R, W, false><<<grid, W * 64, lds, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.max_splits == 1) return e;
    kv8_join_kernel<TYPE, D><<<dim3(a.q_len * a.n_heads, (unsigned)a.n_seqs), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int TYPE>
hipError_t attend_dim(const Kv8AttendArgs &a, hipStream_t s) {
    const bool two = a.row_tiles == 2;
    switch (a.cache.dim) {
        case 64: return two ? attend<TYPE, 64, 2>(a, s) : attend<TYPE, 64, 1>(a, s);
        case 96: return two ? attend<TYPE, 96, 2>(a, s) : attend<TYPE, 96, 1>(a, s);
        case 128: return two ? attend<TYPE, 128, 2>(a, s) : attend<TYPE, 128, 1>(a, s);
        case 192: return two ? attend<TYPE, 192, 2>(a, s) : attend<TYPE, 192, 1>(a, s);
        default: return two ? attend<TYPE, 256, 2>(a, s) : attend<TYPE, 256, 1>(a, s);
    }
}

template <int TYPE>
hipError_t append(const Kv8AppendArgs &a, hipStream_t s) {
    // pages that max_new tokens touch at most; a sequence with more of them takes more trips
    int64_t pages = a.max_new / a.cache.page + 2;
    if (a.max_new <= 1) pages = 1;
    if (pages > a.width) pages = a.width;
    if (pages > 4096) pages = 4096;
    const dim3 grid((unsigned)pages, (unsigned)a.n_seqs, (unsigned)(a.cache.n_kv * 2));
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
        if (vec) kv8_append_kernel<TYPE, true, threads.value><<<grid, threads.value, 0, s>>>(a);
        else kv8_append_kernel<TYPE, false, threads.value><<<grid, threads.value, 0, s>>>(a);
    };
    if (tiles <= 64) run(std::integral_constant<int, 64>{});
    else if (tiles <= 256) run(std::integral_constant<int, 256>{});
    else run(std::integral_constant<int, 512>{});
    return hipGetLastError();
}

}  // namespace

bool kv8_dim_supported(int dim) {
    return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

hipError_t launch_kv8_append(const Kv8AppendArgs &a, int type, hipStream_t s) {
    if (type == kF32) return append<kF32>(a, s);
    if (type == kF16) return append<kF16>(a, s);
    return append<kBF16>(a, s);
}

// Splits. A workgroup's start and end cost as much as three or four of its turns,
// and the launch that joins splits two more, so splits are as long as the chip
// stays busy: what a round of resident workgroups shares evenly; twice that, or
// 1024 positions, where two workgroups share a compute unit and the sequences are
// few or uneven (us: 2 x 32,000, 8 heads of 128, splits of 256 / 512 / 1024 / 2048:
// 37.6, 31.5, 27.9, 26.3; 32 x 8192: 97, 72, 65, 68; one of 4000: 9.9, 11.6, 15.8,
// 24.1, there 256 is twice the share). Whole sequences where they fill the chip by
// themselves (256 x 1500, 8 heads of 128: 93, in splits of 1024 137; 30 x 3000, 4
// heads of 256: 32.0 and 41.5) and, up to 1024 positions, everywhere (64 x 900, 8
// heads of 128: 22, in splits of 256 35) but where a workgroup of four wavefronts
// would take more than two turns with three quarters of the compute units idle (900
// positions, 4 heads of 256: 19.4 whole, 12.3 in splits of 256).
void kv8_attend_plan(Kv8AttendArgs &a, int64_t max_len, int cus) {
    const int rows = a.q_len * (a.n_heads / a.cache.n_kv);
    // positions that a sequence's rows see together, at most and as far as known
    int64_t cap = a.width * a.cache.page;
    if (a.window > 0 && a.window < cap) cap = std::min(cap, a.window + a.q_len + kBlk - 2);
    if (max_len <= 0 || max_len > cap) max_len = cap;
    // Row tiles that a workgroup takes together: two where there are more than 16 rows
    // per key/value head; of more than 128 channels (one wavefront to a SIMD) where it
    // saves a third of the passes over the cache and that is what counts (us: 8 x 6018,
    // 40 rows, 8 heads of 256: 74, one by one 120; 32 rows of 16 x 3000, 8 heads of 192:
    // 39 and 42; 32 rows of 2 x 500, 4 heads of 256: 26 and 14).
    const int64_t alone = a.n_seqs * a.cache.n_kv * ((rows + 15) / 16);
    const int r = rows > 16 && (a.cache.dim <= 128 || (rows > 32 && alone * max_len >= cus * 1024)) ? 2 : 1;
    a.row_tiles = r;
    const int64_t groups = a.n_seqs * a.cache.n_kv * ((rows + 16 * r - 1) / (16 * r));
    const bool two = a.cache.dim <= 128 && !(a.cache.dim == 128 && r == 2);  // to a compute unit
    const int64_t slots = two ? 2 * cus : cus;
    int64_t chunk = (max_len * groups + slots - 1) / slots;
    const bool full = two ? groups >= slots : 2 * groups > slots;
    if (max_len <= kMaxChunk && full) chunk = max_len;
    else if (two && (chunk <= 1024 || a.n_seqs > 1)) chunk = std::min<int64_t>(2 * chunk, 1024);
    chunk = (chunk + 255) / 256 * 256;
    const bool idle = a.cache.dim > 128 && groups * 4 <= cus;
    if (max_len <= (idle ? 512 : 1024)) chunk = 1024;
    // Sequences of one split as far as known stay whole in longer ones, and the table needs
    // fewer of those (32 of 500 positions, 8 heads of 128, max_len 500, a table of 131,072:
    // 268 us in splits of 1024 and, most of them empty, workgroups of eight wavefronts; 150).
    if (chunk > kMaxChunk || (max_len <= chunk && cap > chunk)) chunk = kMaxChunk;
    a.chunk = (int)chunk;
    a.max_splits = (int)((cap + chunk - 1) / chunk);
    a.few = max_len <= chunk && groups * a.max_splits <= cus;
    a.brief = max_len <= 512 && groups > slots;
}

int64_t kv8_attend_partial_bytes(const Kv8AttendArgs &a) {
    if (a.max_splits <= 1) return 0;
    return a.n_seqs * a.max_splits * partial_floats((int64_t)a.q_len * a.n_heads, a.cache.dim) * 4;
}

hipError_t launch_kv8_attend(const Kv8AttendArgs &a, int type, hipStream_t s) {
    if (type == kF32) return attend_dim<kF32>(a, s);
    if (type == kF16) return attend_dim<kF16>(a, s);
    return attend_dim<kBF16>(a, s);
}

}  // namespace qwg
