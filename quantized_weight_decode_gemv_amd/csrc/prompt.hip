// Causal attention over whole prompts, packed one behind another, before their keys and
// values are held in 8 bits: out[t, h] = sum_j softmax_j(scale q[t, h] . k[j, h / group])
// v[j, h / group] over the positions j <= t of the same sequence (the last `window` of them).
#include <algorithm>
#include <type_traits>

#include "attend_device.h"
#include "mx_device.h"
#include "mx_lds.h"

namespace qwg {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Four positions of one channel each from a [position][channel] tile of 16-bit values: of
// sixteen lanes, lane i gives the address of four channels of position i / 4 and takes channel i.
__device__ __forceinline__ u32x2 read_turned(const uint8_t *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4 *)p));
}

// Positions of a block of keys and values in LDS. In fp32 two blocks of 64 leave room for one
// workgroup a compute unit from 96 channels on (4 prompts of 2000 tokens, 16 heads, us with 32 and 64
// positions: of 64 channels 280 and 220, of 96 302 and 318, of 128 397 and 406; of more, 64 do not fit).
constexpr int block_of(int type, int d) { return type == kF32 && d > 64 ? 32 : 64; }

// The first token of a sequence, its length and which of its tiles the workgroup takes:
// false past the last tile. Every wavefront looks for itself. Equal lengths need no search; of
// others a lane takes eight sequences at once (where both were searched one to a lane, 32 heads of 128,
// bf16: 640 prompts of 32 tokens took 169 us, now 112, 300 of up to 60 68 and 63, 21 of up to 900 87 and 89).
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int64_t at, int tile_rows, int group,
                                          int64_t &first, int &len, int &tile) {
    if (!a.starts) {
        const int64_t each = a.n_tokens / a.n_seqs, tiles = (each * group + tile_rows - 1) / tile_rows;
        const int64_t s = at / tiles;
        first = s * each, len = (int)each;
        tile = (int)(tiles - 1 - (at - s * tiles));  // the tiles that see the most come first
        return s < a.n_seqs;
    }
    const int lane = threadIdx.x & 63;
    constexpr int S = 8;
    auto tiles_of = [&](int n) { return (int)((uint32_t)(n * group + tile_rows - 1) / (uint32_t)tile_rows); };  // (2^28 rows at most)
    for (int64_t s0 = 0; s0 < a.n_seqs; s0 += 64 * S) {
        int edge[S + 1], upto = 0;
#pragma unroll
        for (int j = 0; j <= S; ++j)
            edge[j] = min(max(a.starts[min(s0 + lane * S + j, a.n_seqs)], 0), (int)a.n_tokens);
#pragma unroll
        for (int j = 0; j < S; ++j) upto += tiles_of(max(edge[j + 1] - edge[j], 0));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o);
            if (lane >= o) upto += v;
        }
        const uint64_t past = __ballot(at < upto);
        if (past) {
            const int l = __builtin_ctzll(past);
            int left = (int)at - (l ? __builtin_amdgcn_readlane(upto, l - 1) : 0);
#pragma unroll
            for (int j = 0; j < S; ++j) {
                first = __builtin_amdgcn_readlane(edge[j], l);
                len = max(__builtin_amdgcn_readlane(edge[j + 1], l) - (int)first, 0);
                const int tiles = tiles_of(len);
                tile = tiles - 1 - left;
                if (tile >= 0) return true;
                left -= tiles;
            }
        }
        at -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// One workgroup: one tile of rows of one sequence and key/value head; a row is a (token, head
// of the group) pair, so that the heads that read the same keys take them from LDS together. A
// wavefront holds R x 32 rows (their queries and sums in registers); all share the blocks of keys
// and values, which come by LDS DMA, two blocks in turn.
//
// S^T = K Q^T on 32 x 32 tiles gives a lane sixteen scores of one row, at positions
// 8(i/4) + 4(lane/32) + i%4: with the other half lane's a whole row of them, so that maximum and sum
// cross lanes once. The lane's scores eight by eight are the B operand of O^T = V^T P^T as they
// stand; the A operand's eight positions of a channel are two transposing reads of V.
//
// Probabilities of the 16-bit types are rounded to that type (by 2^-8 or 2^-11
// of themselves at most, as often up as down: the output's own rounding once more); their
// sum is taken before.
//
// Non-finite values in V where some row of the tile does not see them are set to zero in
// LDS (0 times infinity is NaN) and added at the end for the rows that do see them.
//
// Bound by the matrix cores and the exponentials between them where prompts are long, at the clock that the
// card's power leaves: one of 12,000 tokens, 32 heads of 128, bf16: 1170-1230 us, 0.96-1.0 PFLOP/s of
// what the rows see (a large library product: 1.13); the matrix cores are busy for half of the cycles.
// 3 of up to 2500 in fp32, a window of 1000: 376-400 us, the matrix cores busy for 80% of the compute units'
// cycles, 6% of them with positions that no row sees.
// Short ones by a tile's start and end, 10 us of which memory is the larger part (a block costs 1.9
// more): 21 of up to 900 take 89 us. One of 77 tokens takes 7.7: the launch and two trips to memory.
// Of 256 channels, and in fp32 of 192, one wavefront to a SIMD: with two the sums spill (4 x 2000, 16
// heads of 256: bf16 316 us for 137, fp32 1815 for 816). Of 192 in 16 bits two spill as well, 20 bytes a
// lane (4 x 2000, 16 heads: bf16 160 us, 155 with one; one of 6000, 32 heads: 543 and 535). The scores of the
// next block ahead of this one's exponentials, wavefronts set out of step, results by way of LDS
// (21 x 900: 95 us for 87) and non-temporal ones (in a loop of calls 111 for 105) were no faster.
template <int TYPE, int D, int W, int R>
__global__ __launch_bounds__(W * 64, (TYPE == kF32 ? D >= 192 : D == 256) ? 1 : 2) void prompt_kernel(PromptArgs a) {
    typedef typename Elem<TYPE>::T T;
    constexpr int B = block_of(TYPE, D);
    constexpr int U = B / 32;                       // score tiles of a block
    constexpr int G = D * (int)sizeof(T) / 16;      // 16-byte granules of a row
    constexpr int kTile = B * G * 16;               // bytes of a block's K (or V)
    constexpr int DT = D / 32;                      // channel tiles
    constexpr int E = 16 / (int)sizeof(T);          // values of a granule
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n = lane & 31, g = lane >> 5;
    const int group = a.n_heads / a.n_kv;
    const int head = (int)(blockIdx.x % a.n_kv);
    int64_t first;
    int len, tile;
    if (!find_tile(a, blockIdx.x / a.n_kv, W * R * 32, group, first, len, tile)) return;
    // (as scalars: left to itself the compiler keeps some of what follows from them in vector registers, and
    // 5 prompts of up to 4000 take 503 us for 483)
    first = __builtin_amdgcn_readfirstlane((int)first);
    len = __builtin_amdgcn_readfirstlane(len), tile = __builtin_amdgcn_readfirstlane(tile);
    const int64_t rows = (int64_t)len * group;
    const int64_t row0 = (int64_t)tile * (W * R * 32), wrow0 = row0 + wave * R * 32;
    // tokens of the workgroup's rows and of the wavefront's
    const int t_lo = (int)(row0 / group), t_hi = (int)min((row0 + W * R * 32 - 1) / group, (int64_t)len - 1);
    const int w_lo = (int)(wrow0 / group), w_hi = (int)min((wrow0 + R * 32 - 1) / group, (int64_t)len - 1);
    const bool idle = wrow0 >= rows;
    const int window = (int)min(a.window, (int64_t)1 << 30);  // 0: all

    extern __shared__ __align__(16) uint8_t lds[];
    int *const dirty = (int *)(lds + 4 * kTile);
    if (threadIdx.x == 0) *dirty = 0;

    // granule f of a tile in LDS holds granule (f % G) ^ key of row f / G; what thirty-two lanes
    // read of V at once, 32 bytes of each of four rows twice, lies in 256 bytes too
    auto k_key = [](int row) { return row_key<G>(row); };
    auto v_key = [](int row) {
        return TYPE == kF32 ? 0 : G % 16 == 0 ? (row & 3) * 4 : G % 8 == 0 ? (row & 3) * 2 : 0;
    };
    const T *const kp = (const T *)a.k + first * a.k_stride + (int64_t)head * D;
    const T *const vp = (const T *)a.v + first * a.v_stride + (int64_t)head * D;
    // A wavefront's DMAs of a block. Where they lie whole 16 rows apart, and so their granules' keys
    // are the same, one offset serves all of them.
    constexpr int N = (B * G / 64 + W - 1) / W;
    constexpr bool kEven = W * 64 % G == 0 && W * 64 / G % 16 == 0;
    auto offset = [&](int i, bool of_v, int last) {  // last: the block's last position, or the sequence's
        const int f = (i * W + wave) * 64 + lane, row = f / G, c = f - row * G;
        const uint32_t pos = min(row, last);  // past the end: masked
        return (pos * (uint32_t)(of_v ? a.v_stride : a.k_stride) + (c ^ (of_v ? v_key(row) : k_key(row))) * E) * (uint32_t)sizeof(T);
    };
    uint32_t k_off[kEven ? 1 : N], v_off[kEven ? 1 : N];
#pragma unroll
    for (int i = 0; i < (kEven ? 1 : N); ++i) k_off[i] = offset(i, false, B), v_off[i] = offset(i, true, B);
    auto fetch = [&](bool of_v, int b0, uint32_t to) {
        const int64_t stride = of_v ? a.v_stride : a.k_stride;
        const T *const p0 = (of_v ? vp : kp) + b0 * stride;
        to += wave * 1024;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (B * G / 64 % W != 0 && i * W + wave >= B * G / 64) break;
            const bool whole = b0 + B <= len;
            const T *const p = kEven && whole ? p0 + i * (W * 64 / G) * stride : p0;
            const uint32_t off = whole ? (of_v ? v_off : k_off)[kEven ? 0 : i] : offset(i, of_v, len - 1 - b0);
            if (a.vec) {
                dma16(p, off, to + i * W * 1024);
            } else {
                T x[E];
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = p[off / sizeof(T) + e];
                __builtin_memcpy(lds + to + i * W * 1024 + lane * 16, x, 16);
            }
        }
    };
    // a block of keys, or of values, into the first or second of its two places
    auto issue_k = [&](int b0, int buf) { fetch(false, b0, buf * 2 * kTile); };
    auto issue_v = [&](int b0, int buf) { fetch(true, b0, buf * 2 * kTile + kTile); };

    const int low = window > 0 ? max(0, t_lo - window + 1) / B * B : 0;
    issue_k(low, 0);  // (ahead of the queries: one trip to memory for both)
    issue_v(low, 0);

    // queries: the B operand's lane takes row n, eight channels (four of fp32) per half
    const bool flip = a.scale < 0;  // the maximum is taken before the scale
    // (never zero: -infinity, of what is masked, has to stay what it is; the smallest number moves no
    // score by more than 2^-21; a NaN stays one)
    const float to_log2 = __builtin_elementwise_maximum(fabsf(a.scale) * 1.4426950408889634f, 0x1p-149f);
    u32x4 q[R][G / 2];
    int token[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = wrow0 + r * 32 + n;
        token[r] = row < rows ? (int)(row / group) : -1;
        const T *p = (const T *)a.q + (first + max(token[r], 0)) * a.q_stride +
                     (int64_t)(head * group + (int)(row % group)) * D;
#pragma unroll
        for (int s = 0; s < G / 2; ++s) {
            u32x4 w = {0, 0, 0, 0};
            if (token[r] >= 0) {
                if (a.vec) {
                    w = *(const u32x4 *)(p + (s * 2 + g) * E);
                } else {
                    T v[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] = p[(s * 2 + g) * E + e];
                    __builtin_memcpy(&w, v, 16);
                }
            }
            const uint32_t sign = flip ? (sizeof(T) == 4 ? 0x80000000u : 0x80008000u) : 0u;
            q[r][s] = w ^ sign;
        }
    }

    float top[R], sum[R];  // maximum times to_log2, sum of this half lane's probabilities
    f32x16 out[R][DT];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        top[r] = -__builtin_inff();
        sum[r] = 0;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) out[r][t][i] = 0;
    }
    // whether every one of the tokens from lo to hi sees the whole block
    auto whole = [&](int b0, int lo, int hi) { return b0 + B - 1 <= lo && (window == 0 || b0 > hi - window); };

    // Where a lane reads a tile: of K granule g of row n, of V (the first) four channels of the position
    // of its quarter. The granules of other steps and channel tiles lie an exclusive or away.
    const int v_row = g * 4 + (n >> 2 & 3);
    const int k_at = (n * G + (g ^ k_key(n))) * 16;
    const int v_at = (v_row * G + (((n >> 4) * 2 + (n >> 1 & 1)) ^ v_key(v_row))) * 16 + (n & 1) * 8;
    auto key = [&](const uint8_t *k_lds, int i) {  // the i-th operand of the first product: tile i % U, step i / U
        const int c = i / U * 2;
        const int at = G % 16 == 0 && c < 16 ? k_at ^ c * 16 : (n * G + ((c + g) ^ k_key(n))) * 16;
        return *(const u32x4 *)(k_lds + at + i % U * 32 * G * 16);
    };
    auto value = [&](const uint8_t *v_lds, int i) {  // of the second: step i / DT, channel tile i % DT
        const int c = i % DT * 4;
        const int at = G % 16 == 0 && c < 16 ? v_at ^ c * 16
                                             : (v_row * G + ((c + (n >> 4) * 2 + (n >> 1 & 1)) ^ v_key(v_row))) * 16 + (n & 1) * 8;
        const uint8_t *v = v_lds + at + i / DT * 16 * G * 16;
        const u32x2 x = read_turned(v), y = read_turned(v + 8 * G * 16);
        return u32x4{x[0], x[1], y[0], y[1]};
    };

    // infinities and NaNs of a block of values that some row does not see all of: to zero
    auto clean = [&](uint8_t *v_lds) {
        bool found = false;
        for (int f = threadIdx.x; f < B * G; f += W * 64) {
            u32x4 w = *(u32x4 *)(v_lds + f * 16);
            bool here = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                constexpr uint32_t x = TYPE == kF32 ? 0x7f800000u : TYPE == kF16 ? 0x7c00u : 0x7f80u;
                if constexpr (TYPE == kF32) {
                    if ((w[e] & x) == x) w[e] = 0, here = true;
                } else {
                    if ((w[e] & x) == x) w[e] &= 0xffff0000u, here = true;
                    if ((w[e] >> 16 & x) == x) w[e] &= 0xffffu, here = true;
                }
            }
            if (here) *(u32x4 *)(v_lds + f * 16) = w, found = true;
        }
        if (found) *dirty = 1;
        __syncthreads();
    };
    auto scores = [&](f32x16 (&s)[R][U], const uint8_t *k_lds) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[r][u][i] = 0;
        // the tiles' operands of a step in turn: a chain of sums each
        products<U * G / 2, 1, R * (TYPE == kF32 ? 4 : 1)>(
            [&](int i) { return key(k_lds, i); },
            [&](int i, u32x4 k) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    f32x16 &x = s[r][i % U];
                    if constexpr (TYPE == kF32) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x = __builtin_amdgcn_mfma_f32_32x32x2f32(u2f(k[e]), u2f(q[r][i / U][e]), x, 0, 0, 0);
                    } else {
                        x = mfma32<TYPE == kF16>(k, q[r][i / U], x);
                    }
                }
            });
    };
    // what a row does not see becomes -infinity
    auto mask = [&](int r, f32x16 (&s)[U], int b0) {
        // the positions that the lane's row sees, from the lane's first of the block
        const int hi = token[r] - b0 - g * 4, lo = window > 0 ? hi - window : -1;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int pos = u * 32 + (i >> 2) * 8 + (i & 3);
                if (pos > hi || pos <= lo) s[u][i] = -__builtin_inff();
            }
    };
    float base[R];  // what the exponents are taken from: the maximum, or zero before there is one
    // takes a block's largest scores in: where one is far above the maximum so far, what was summed shrinks
    auto raise = [&](int r, float largest) {
        const float t = max_halves(largest);
        const float scaled = t == -__builtin_inff() ? t : t * to_log2;
        if (__any(scaled > top[r] + kSlack)) {  // (every number is more than -infinity)
            const float now = fmaxf(top[r], scaled);
            const float alpha = now == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top[r] - now);
            top[r] = now;
            sum[r] *= alpha;
#pragma unroll
            for (int t = 0; t < DT; ++t) out[r][t] *= alpha;
        }
        base[r] = top[r] == -__builtin_inff() ? 0.0f : top[r];
    };
    auto largest = [&](const f32x16 (&s)[U]) {
        float m[2] = {-__builtin_inff(), -__builtin_inff()};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 16; i += 2) m[i >> 1 & 1] = maximum3(m[i >> 1 & 1], s[u][i], s[u][i + 1]);
        return maximum3(m[0], m[1], m[1]);
    };
    auto weight = [&](float s, int r) { return __builtin_amdgcn_exp2f(__builtin_fmaf(s, to_log2, -base[r])); };

    f32x16 s[R][U];
    int buf = 0;
    for (int b0 = low; b0 <= t_hi; b0 += B, buf ^= 1) {
        wait_vmcnt<0>();
        __syncthreads();
        if (b0 + B <= t_hi) issue_k(b0 + B, buf ^ 1), issue_v(b0 + B, buf ^ 1);
        uint8_t *const k_lds = lds + buf * 2 * kTile, *const v_lds = k_lds + kTile;
        if (!whole(b0, t_lo, t_hi)) clean(v_lds);
        if (idle || b0 > w_hi || (window > 0 && b0 + B - 1 <= w_lo - window)) continue;
        scores(s, k_lds);
        u32x4 p[R][TYPE == kF32 ? 1 : U * 2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!whole(b0, w_lo, w_hi)) mask(r, s[r], b0);
            raise(r, largest(s[r]));
            float part[4] = {0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[r][u][i] = weight(s[r][u][i], r);
                    part[i & 3] += s[r][u][i];
                }
            sum[r] += (part[0] + part[1]) + (part[2] + part[3]);
            if constexpr (TYPE != kF32) {
#pragma unroll
                for (int j = 0; j < U * 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[r][j][e] = pack2<TYPE == kF16>(s[r][j / 2][(j & 1) * 8 + e * 2], s[r][j / 2][(j & 1) * 8 + e * 2 + 1]);
            }
        }
        if constexpr (TYPE == kF32) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float *row = (const float *)(v_lds + (u * 32 + (i >> 2) * 8 + g * 4 + (i & 3)) * G * 16);
#pragma unroll
                    for (int t = 0; t < DT; ++t)
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            out[r][t] = __builtin_amdgcn_mfma_f32_32x32x2f32(row[t * 32 + n], s[r][u][i], out[r][t], 0, 0, 0);
                }
        } else {
            products<U * 2 * DT, 2, R>([&](int i) { return value(v_lds, i); },
                                       [&](int i, u32x4 v) {
#pragma unroll
                                           for (int r = 0; r < R; ++r)
                                               out[r][i % DT] = mfma32<TYPE == kF16>(v, p[r][i / DT], out[r][i % DT]);
                                       });
        }
    }

    __syncthreads();
    const bool mend = *dirty != 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float total = sum_halves(sum[r]);
        if (token[r] < 0) continue;
        const int64_t row = wrow0 + r * 32 + n;
        const float inv = 1.0f / total;
        uint32_t even[2] = {0, 0};
        T *dst = (T *)a.out + ((first + token[r]) * a.n_heads + head * group + (int)(row % group)) * D;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const int d = t * 32 + i * 2 + g * 4;
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = out[r][t][i + e] * inv;
                if (mend) {
                    for (int b0 = low; b0 <= token[r]; b0 += B) {
                        if (whole(b0, t_lo, t_hi)) continue;
                        for (int j = b0; j < b0 + B && j <= token[r]; ++j) {
                            if (window > 0 && j <= token[r] - window) continue;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float v = (float)vp[(int64_t)j * a.v_stride + d + e];
                                if (!(fabsf(v) < __builtin_inff())) o[e] += v;
                            }
                        }
                    }
                }
                if constexpr (TYPE == kF32) {
                    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
                    *(f4 *)(dst + d) = f4{o[0], o[1], o[2], o[3]};
                } else {
                    // of two runs of four channels the half lanes take one's eight each: 16 bytes a store
                    const uint32_t w0 = pack2<TYPE == kF16>(o[0], o[1]), w1 = pack2<TYPE == kF16>(o[2], o[3]);
                    if (i % 8 == 0) {
                        even[0] = w0, even[1] = w1;
                    } else {
                        const auto x = __builtin_amdgcn_permlane32_swap(even[0], w0, false, false);
                        const auto y = __builtin_amdgcn_permlane32_swap(even[1], w1, false, false);
                        typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
                        *(u4 *)(dst + t * 32 + (i - 4) * 2 + g * 8) = u4{x[0], y[0], x[1], y[1]};
                    }
                }
            }
    }
}

template <int TYPE, int D>
hipError_t prompt(const PromptArgs &a, hipStream_t s) {
    constexpr int W = 4, R = 1;
    constexpr size_t lds = 4 * (size_t)block_of(TYPE, D) * D * sizeof(typename Elem<TYPE>::T) + 16;
    static_assert(lds <= 160 * 1024, "LDS");
    const int64_t group = a.n_heads / a.n_kv;
    const int64_t tiles = a.n_tokens * group / (W * R * 32) + a.n_seqs;
    prompt_kernel<TYPE, D, W, R><<<dim3((unsigned)(tiles * a.n_kv)), W * 64, lds, s>>>(a);
    return hipGetLastError();
}

template <int TYPE>
hipError_t prompt_dim(const PromptArgs &a, hipStream_t s) {
    switch (a.dim) {
        case 64: return prompt<TYPE, 64>(a, s);
        case 96: return prompt<TYPE, 96>(a, s);
        case 128: return prompt<TYPE, 128>(a, s);
        case 192: return prompt<TYPE, 192>(a, s);
        default: return prompt<TYPE, 256>(a, s);
    }
}

}  // namespace

hipError_t launch_prompt_attend(const PromptArgs &a, int type, hipStream_t s) {
    if (type == kF32) return prompt_dim<kF32>(a, s);
    if (type == kF16) return prompt_dim<kF16>(a, s);
    return prompt_dim<kBF16>(a, s);
}

}  // namespace qwg
