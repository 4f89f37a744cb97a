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
#include "mx_device.h"

namespace qwg {

namespace {

// ------------------------------------------------------------------- append

// The biased exponent of the smallest power of two s with top / s <= 448 =
// 1.75 * 2^8, `top` given as the bits of a finite magnitude.
__device__ __forceinline__ uint32_t page_exponent(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e > 0 ? (uint32_t)e : 0;
}

__device__ __forceinline__ uint32_t fp8_code(float v, float scale) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const s16x2 z = {0, 0};
    // NaN and infinity become the NaN code
    return __builtin_bit_cast(
               uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, v, v, scale, false)) & 255u;
}

__device__ __forceinline__ float fp8_value(uint32_t code) {
    return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

// One workgroup per (page of a sequence, sequence, head of K or V).
template <int TYPE>
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8AppendArgs a) {
    typedef typename Elem<TYPE>::T T;
    __shared__ uint32_t tops[4];
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
    for (int64_t p = held / c.page + blockIdx.x; p * c.page < end; p += gridDim.x) {
        const int64_t id = a.table[seq * a.width + p];
        if (id < 0 || id >= c.n_pages) continue;
        const int64_t pos0 = p * c.page;
        const int old = (int)max((int64_t)0, held - pos0);               // slots filled before
        const int stop = (int)min((int64_t)c.page, end - pos0);          // slots filled after
        const int64_t tok0 = first + pos0 - held;                        // token of slot 0
        uint8_t *codes = (is_v ? c.v : c.k) + (id * c.n_kv + head) * (int64_t)c.page * c.dim;
        uint8_t *scale = (is_v ? c.v_scales : c.k_scales) + id * c.n_kv + head;
        uint32_t top = 0;
        for (int i = threadIdx.x; i < (stop - old) * c.dim; i += blockDim.x) {
            const int s = old + i / c.dim, d = i % c.dim;
            const uint32_t m = f2u(to_f32(x[(tok0 + s) * stride + d])) & 0x7fffffffu;
            if (m < 0x7f800000u) top = max(top, m);
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
        const uint32_t before = old ? *scale : 0;
        const uint32_t now = max(before, page_exponent(top));
        if (old && now > before) {
            // the page's scale rises: its codes are rounded to the new one
            const float shift = __builtin_ldexpf(1.0f, (int)before - (int)now);
            for (int i = threadIdx.x; i < old * c.dim; i += blockDim.x) {
                const int64_t at = is_v ? (int64_t)(i / old) * c.page + i % old : i;
                codes[at] = (uint8_t)fp8_code(fp8_value(codes[at]) * shift, 1.0f);
            }
        }
        const float sc = e8m0(now);
        for (int i = threadIdx.x; i < (stop - old) * c.dim; i += blockDim.x) {
            const int n = stop - old;
            const int s = old + (is_v ? i % n : i / c.dim), d = is_v ? i / n : i % c.dim;
            const float v = to_f32(x[(tok0 + s) * stride + d]);
            codes[is_v ? d * c.page + s : s * c.dim + d] = (uint8_t)fp8_code(v, sc);
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

constexpr int kBlk = 64;     // positions a wavefront takes at once
constexpr int kWaves = 4;

// Bytes of a word that hold a NaN code, as 0x80 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
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
// row maxima, and nothing but Q goes through LDS.
//
// Queries and probabilities enter as bf16 parts (one to three) that hold all
// their bits, or 16 of the probabilities' for the 16-bit types; e4m3 is exact in bf16.
template <int TYPE, int D, int R>
__global__ __launch_bounds__(kWaves * 64) void kv8_attend_kernel(Kv8AttendArgs a) {
    typedef typename Elem<TYPE>::T T;
    constexpr int PQ = Elem<TYPE>::pieces;      // parts of a query
    constexpr int PP = TYPE == kF32 ? 3 : 2;    // parts of a probability
    constexpr int KS = D / 32;                  // steps of the first product
    constexpr int DT = D / 16;                  // channel tiles of the second
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const Kv8 &c = a.cache;
    const int group = a.n_heads / c.n_kv;
    const int rows = a.q_len * group;
    const int64_t seq = blockIdx.z;
    const int tiles = (rows + 16 * R - 1) / (16 * R);
    const int head = (int)blockIdx.y / tiles, row0 = (int)blockIdx.y % tiles * 16 * R;
    const int64_t len0 = a.lens[seq], cap = a.width * c.page;
    const bool bad = len0 < 0 || len0 > cap;  // no such length: the rows become NaN
    const int64_t len = bad ? 0 : len0;
    const int splits = max(1, (int)((len + a.chunk - 1) / a.chunk));
    const int split = blockIdx.x;
    if (split >= splits) return;
    // positions that some row sees: those below len, from the first row's window on
    const int64_t low = a.window > 0 ? max((int64_t)0, len - a.q_len + 1 - a.window) : 0;
    const int64_t begin = max((int64_t)split * a.chunk, low / kBlk * kBlk);
    const int64_t end = min((int64_t)(split + 1) * a.chunk, len);

    extern __shared__ __align__(16) uint8_t lds[];
    // Q parts: [tile][step][part][lane] 16 bytes, as the lanes take them
    {
        const T *q = (const T *)a.q;
        for (int i = threadIdx.x; i < R * KS * 64; i += kWaves * 64) {
            const int l = i & 63, ks = (i >> 6) % KS, r = (i >> 6) / KS;
            const int row = row0 + r * 16 + (l & 15), lg = l >> 4;
            // a pair of steps takes 64 channels, 16 consecutive ones per lane
            // group; an odd last step 32, 8 per lane group
            const int d = (D % 64 && ks == KS - 1) ? ks * 32 + lg * 8
                                                   : (ks >> 1) * 64 + lg * 16 + (ks & 1) * 8;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (row < rows) {
                const int t = row / group, h = head * group + row % group;
                load8<T, false>(q + (seq * a.q_len + t) * a.q_stride + (int64_t)h * D + d, v);
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
                *(u32x4 *)(lds + (((r * KS + ks) * PQ + p) * 64 + l) * 16) =
                    u32x4{w[p][0], w[p][1], w[p][2], w[p][3]};
        }
    }
    __syncthreads();

    const float to_log2 = a.scale * 1.4426950408889634f;
    float top[R], sum[R];
    f32x4 out[R][DT];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        top[r] = -__builtin_inff();
        sum[r] = 0;
#pragma unroll
        for (int t = 0; t < DT; ++t) out[r][t] = f32x4{0, 0, 0, 0};
    }
    // the last position that each of this lane's rows sees
    int64_t last[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r * 16 + n;
        last[r] = row < rows ? len - a.q_len + row / group : -1;
    }
    const int32_t *table = a.table + seq * a.width;
    const int64_t head_bytes = (int64_t)c.page * D;
    // page of a position: 0 for positions past the end, -1 for a number that is no page
    auto page_of = [&](int64_t pos) -> int64_t {
        if (pos >= len) return 0;
        const int64_t id = table[pos / c.page];
        return id < 0 || id >= c.n_pages ? -1 : id;
    };

    for (int64_t b0 = begin + wave * kBlk; b0 < end; b0 += kWaves * kBlk) {
        const int64_t kpos = b0 + (n >> 2) * 16, vpos = b0 + g * 16;
        int64_t kid = page_of(kpos), vid = page_of(vpos);
        const bool lost = vid < 0;  // this lane's sixteen positions have no page
        kid = max(kid, (int64_t)0), vid = max(vid, (int64_t)0);
        const uint8_t *kp = c.k + (kid * c.n_kv + head) * head_bytes + (kpos % c.page + (n & 3)) * D + g * 16;
        const uint8_t *vp = c.v + (vid * c.n_kv + head) * head_bytes + (int64_t)n * c.page + vpos % c.page;
        float ks = e8m0(c.k_scales[vid * c.n_kv + head]) * to_log2;
        // where there is no page its V counts for nothing: not even its scale may
        // (0 times a NaN scale is NaN)
        const float vs = lost || vpos >= len ? 1.0f : e8m0(c.v_scales[vid * c.n_kv + head]);
        if (lost) ks = __builtin_nanf("");
        u32x4 kc[4][D / 64];
        u32x2 kt[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j) kc[u][j] = *(const u32x4 *)(kp + u * 4 * D + j * 64);
            if constexpr (D % 64 != 0)
                kt[u] = *(const u32x2 *)(kp - g * 8 + u * 4 * D + (D / 64) * 64);
        }
        u32x4 vc[DT];
#pragma unroll
        for (int t = 0; t < DT; ++t) vc[t] = *(const u32x4 *)(vp + (int64_t)t * 16 * c.page);

        f32x4 s[R][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][u] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const bool odd = D % 64 != 0 && k == KS - 1;
                const bf16x8 kv = odd ? fp8x8(kt[u][0], kt[u][1])
                                      : fp8x8(kc[u][k >> 1][(k & 1) * 2], kc[u][k >> 1][(k & 1) * 2 + 1]);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int p = PQ - 1; p >= 0; --p) {
                        const bf16x8 q = *(const bf16x8 *)(lds + (((r * KS + k) * PQ + p) * 64 + lane) * 16);
                        s[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, q, s[r][u], 0, 0, 0);
                    }
            }
        }
        // every row sees the whole block, or the rows' masks decide
        const bool whole = b0 + kBlk <= len - a.q_len + 1 && (a.window <= 0 || b0 >= len - a.window);
        if (!whole) {
            // codes past the end are whatever the pool held: none of them may
            // reach the products
            const int64_t left = len - vpos;
            const int keep = left < 0 ? 0 : left > 16 ? 16 : (int)left;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int k = keep - w * 4;
                const uint32_t m = k >= 4 ? ~0u : k <= 0 ? 0u : (1u << (8 * k)) - 1u;
#pragma unroll
                for (int t = 0; t < DT; ++t) vc[t][w] &= m;
            }
        }
        uint32_t seen[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            seen[r] = 0xffffu;
            if (!whole) {
                const int64_t hi = last[r] - vpos;
                const int64_t lo = a.window > 0 ? max((int64_t)0, last[r] - a.window + 1 - vpos) : 0;
                uint32_t m = hi < 0 ? 0u : hi >= 15 ? 0xffffu : (2u << hi) - 1u;
                m &= lo >= 16 ? 0u : 0xffffu << lo;
                seen[r] = m & 0xffffu;
            }
            float m = -__builtin_inff();
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = s[r][u][i] * ks;
                    if (!whole && !(seen[r] >> (u * 4 + i) & 1)) v = -__builtin_inff();
                    s[r][u][i] = v;
                    m = fmaxf(m, v);
                }
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            const float now = fmaxf(top[r], m);
            const float base = now == -__builtin_inff() ? 0.0f : now;
            const float alpha = __builtin_amdgcn_exp2f(top[r] - base);
            top[r] = now;
            float part = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = __builtin_amdgcn_exp2f(s[r][u][i] - base);
                    s[r][u][i] = p;
                    part += p;
                }
            sum[r] = sum[r] * alpha + part;
#pragma unroll
            for (int t = 0; t < DT; ++t) out[r][t] *= alpha;
        }
        // a NaN in V that some rows see and others do not must reach the former alone
        bool some_nan = false;
        if (!whole) {
            uint32_t any = 0;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int w = 0; w < 4; ++w) any |= nan_bytes(vc[t][w]);
            some_nan = __any(any != 0);
        }
        if (some_nan) {
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
                        for (int i = 0; i < 8; ++i) see[i] = (__bf16)(seen[r] >> (k * 8 + i) & 1 ? 1.0f : 0.0f);
                        hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            fp8x8(flags[k * 2], flags[k * 2 + 1]), see, hit, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (hit[i] > 0) out[r][t][i] = __builtin_nanf("");
                }
            }
        }
        bf16x8 pp[R][2][PP];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = s[r][k * 2 + i / 4][i % 4] * vs;
                    uint32_t h, m, l;
                    split3(p, h, m, l);
                    pp[r][k][0][i] = __builtin_bit_cast(__bf16, (uint16_t)h);
                    pp[r][k][1][i] = __builtin_bit_cast(__bf16, (uint16_t)m);
                    if constexpr (PP == 3) pp[r][k][2][i] = __builtin_bit_cast(__bf16, (uint16_t)l);
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
                        out[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pp[r][k][p], out[r][t], 0, 0, 0);
            }
    }

    // join the wavefronts: [wave][row][D] sums, then their maxima and totals
    __syncthreads();
    constexpr int RP = D + 4;  // row pitch: four floats past a multiple of 32 banks
    float *so = (float *)lds;
    float *sm = so + kWaves * R * 16 * RP;
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
    for (int i = threadIdx.x; i < R * 16 * (D / 4); i += kWaves * 64) {
        const int d = i % (D / 4) * 4, lr = i / (D / 4), row = row0 + lr;
        if (row >= rows) continue;
        float m = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sm[(w * R * 16 + lr) * 2]);
        const float base = m == -__builtin_inff() ? 0.0f : m;
        float total = 0;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[(w * R * 16 + lr) * 2] - base);
            total += f * sm[(w * R * 16 + lr) * 2 + 1];
            o += f * *(const f32x4 *)(so + (w * R * 16 + lr) * RP + d);
        }
        const int t = row / group, h = head * group + row % group;
        if (splits == 1) {
            T *dst = (T *)a.out + ((row_base + t) * a.n_heads + h) * D + d;
            const float inv = bad ? __builtin_nanf("") : total == 0 ? 0.0f : 1.0f / total;
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = (T)(total == 0 && !bad ? 0.0f : o[e] * inv);
        } else {
            float *dst = a.partial + ((seq * a.max_splits + split) * a.q_len * a.n_heads + (int64_t)t * a.n_heads + h) * (D + 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[2 + d + e] = o[e];
            if (d == 0) dst[0] = m, dst[1] = total;
        }
    }
}

// Joins the splits of a sequence: one wavefront per (query token, head).
template <int TYPE, int D>
__global__ __launch_bounds__(64) void kv8_join_kernel(Kv8AttendArgs a) {
    typedef typename Elem<TYPE>::T T;
    const int64_t seq = blockIdx.y;
    const int row = blockIdx.x;  // token * n_heads + head
    const int64_t len0 = a.lens[seq];
    const int64_t len = len0 < 0 || len0 > a.width * a.cache.page ? 0 : len0;
    const int splits = max(1, (int)((len + a.chunk - 1) / a.chunk));
    if (splits == 1) return;
    const int64_t rows = (int64_t)a.q_len * a.n_heads;
    const float *p = a.partial + (seq * a.max_splits * rows + row) * (D + 2);
    float m = -__builtin_inff();
    for (int s = 0; s < splits; ++s) m = fmaxf(m, p[s * rows * (D + 2)]);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float total = 0;
    for (int s = 0; s < splits; ++s)
        total += __builtin_amdgcn_exp2f(p[s * rows * (D + 2)] - base) * p[s * rows * (D + 2) + 1];
    for (int d = threadIdx.x; d < D; d += 64) {
        float o = 0;
        for (int s = 0; s < splits; ++s)
            o += __builtin_amdgcn_exp2f(p[s * rows * (D + 2)] - base) * p[s * rows * (D + 2) + 2 + d];
        ((T *)a.out)[(seq * rows + row) * D + d] = (T)(total == 0 ? 0.0f : o / total);
    }
}

template <int TYPE, int D, int R>
hipError_t attend(const Kv8AttendArgs &a, hipStream_t s) {
    const int rows = a.q_len * (a.n_heads / a.cache.n_kv);
    const int tiles = (rows + 16 * R - 1) / (16 * R);
    constexpr size_t q = (size_t)R * (D / 32) * Elem<TYPE>::pieces * 64 * 16;
    constexpr size_t join = (size_t)kWaves * R * 16 * (D + 4 + 2) * 4;
    const dim3 grid(a.max_splits, a.cache.n_kv * tiles, (unsigned)a.n_seqs);
    kv8_attend_kernel<TYPE, D, R><<<grid, kWaves * 64, q > join ? q : join, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.max_splits == 1) return e;
    kv8_join_kernel<TYPE, D><<<dim3(a.q_len * a.n_heads, (unsigned)a.n_seqs), 64, 0, s>>>(a);
    return hipGetLastError();
}

template <int TYPE>
hipError_t attend_dim(const Kv8AttendArgs &a, hipStream_t s) {
    switch (a.cache.dim) {
        case 64: return attend<TYPE, 64, 1>(a, s);
        case 96: return attend<TYPE, 96, 1>(a, s);
        case 128: return attend<TYPE, 128, 1>(a, s);
        case 192: return attend<TYPE, 192, 1>(a, s);
        default: return attend<TYPE, 256, 1>(a, s);
    }
}

}  // namespace

bool kv8_dim_supported(int dim) {
    return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

hipError_t launch_kv8_append(const Kv8AppendArgs &a, int type, hipStream_t s) {
    // pages that max_new tokens touch at most; a sequence with more of them takes more trips
    int64_t pages = a.max_new / a.cache.page + 2;
    if (a.max_new <= 1) pages = 1;
    if (pages > a.width) pages = a.width;
    if (pages > 4096) pages = 4096;
    const dim3 grid((unsigned)pages, (unsigned)a.n_seqs, (unsigned)(a.cache.n_kv * 2));
    if (type == kF32)
        kv8_append_kernel<kF32><<<grid, 256, 0, s>>>(a);
    else if (type == kF16)
        kv8_append_kernel<kF16><<<grid, 256, 0, s>>>(a);
    else
        kv8_append_kernel<kBF16><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

// Splits: enough workgroups for about four per compute unit, of at least
// 256 positions (one block for each wavefront).
void kv8_attend_plan(Kv8AttendArgs &a, int64_t max_len, int cus) {
    const int rows = a.q_len * (a.n_heads / a.cache.n_kv);
    const int64_t cap = a.width * a.cache.page;
    if (max_len <= 0 || max_len > cap) max_len = cap;
    const int64_t groups = a.n_seqs * a.cache.n_kv * ((rows + 15) / 16);
    const int64_t want = (4 * (int64_t)cus + groups - 1) / groups;
    int64_t chunk = (max_len + want - 1) / want;
    chunk = (chunk + 255) / 256 * 256;
    a.chunk = (int)chunk;
    a.max_splits = (int)((cap + chunk - 1) / chunk);
}

int64_t kv8_attend_partial_bytes(const Kv8AttendArgs &a) {
    if (a.max_splits <= 1) return 0;
    return a.n_seqs * a.max_splits * a.q_len * a.n_heads * (int64_t)(a.cache.dim + 2) * 4;
}

hipError_t launch_kv8_attend(const Kv8AttendArgs &a, int type, hipStream_t s) {
    if (type == kF32) return attend_dim<kF32>(a, s);
    if (type == kF16) return attend_dim<kF16>(a, s);
    return attend_dim<kBF16>(a, s);
}

}  // namespace qwg
