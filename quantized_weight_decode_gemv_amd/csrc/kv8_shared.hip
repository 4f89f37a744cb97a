// Attention behind a shared prefix of the 8-bit cache: the prefix's pass over the rows of all
// sequences at once. The sequences' own positions, and the meeting of both: kv8.hip.
#include <algorithm>
#include <type_traits>

#include "attend_device.h"
#include "kv8_device.h"
#include "mx_lds.h"

namespace qwg {

namespace {

// Four e4m3 codes as fp16 (HALF) or bf16, exact in both.
template <bool HALF>
__device__ __forceinline__ u32x2 widened(uint32_t w) {
    if constexpr (HALF)
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))};
    else
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
}

// What a page's positions share: its scale of the scores (log2 e and the call's scale in it; NaN
// where it is no page of the pool), log2 v as the products take it in and its inverse, what of v
// that leaves out.
struct Page {
    float scale, power, inverse, rest;
};

// Exponents of values that a split's products take in: at most so far below the largest.
constexpr int kPowers = 64;
// (beside a Page, where its head's keys and values begin in the pool: byte, or code, number)
constexpr int kPrefixPages = kMaxPages * (int)(sizeof(Page) + sizeof(int64_t));

// Eight wavefronts, a compute unit's registers: rows that share the conversion of what they see. (In
// fours, two workgroups to a compute unit, 64 sequences behind 32,000 positions, 8 heads of 128,
// took 58 us for 52.)
constexpr int kPrefixWaves = 8, kPrefixRows = kPrefixWaves * 32;

// LDS of a workgroup: two blocks of keys and values in 16 bits, of which one is made while the other is
// used, blocks on their way from memory, the split's pages, the exponents' range, a flag.
template <int D>
struct PrefixLds {
    static constexpr int kWide = 2 * kBlk * D * 2;
    static constexpr int kChunks = (4 * D + kPrefixWaves * 64 - 1) / (kPrefixWaves * 64);  // 16 bytes of K a thread, and of V
    static constexpr int kRaw = 2 * kChunks * kPrefixWaves * 1024;
    static constexpr int kAhead = 4;
    static constexpr int kBytes = 2 * kWide + kAhead * kRaw + ((kPrefixPages + 31) & ~15);
    static_assert(kBytes <= 160 * 1024, "LDS");
};

// One workgroup: one split of the prefix, one key/value head, W x 32 rows; a row is a (token of
// any sequence, head of the group) pair. 64 positions of keys and values at a time are made 16 bits
// wide by the workgroup together and lie in LDS for all wavefronts: each would spend as long on
// the conversion alone as on the products. The values' transposed rows go in the order in which the second product's lanes take
// positions: of sixteen, 0-3 and 8-11, then 4-7 and 12-15.
//
// S^T = K Q^T and O^T = V^T P^T as in attention over prompts: a lane's scores are the second
// product's operand as they stand. Keys and values are codes, exact in 16 bits; with k and v the
// scales of a position's page, q.k times k goes into the exponential and v with it: P = 2^(q.k k
// + log2 v - M), M the running maximum of q.k k + log2 v. So P is at most one (2^8 in between) whatever
// the pages' scales, what it loses by its rounding to fp16 (2^-11 of itself, 2^-25 of the largest) is
// small against the row's sum, and no product overflows. The softmax's total is the sum of P / v, in fp32.
// Where a page's v is below 2^-64 of the split's largest, P takes that in the exponent and the
// rest after the total.
//
// Bound by the conversion, the exponentials and the products in turn: the wavefronts of a unit meet at
// each block. 64 sequences behind 32,000 positions, 8 heads of 128, four queries' heads each, bf16:
// 51.5 us (34 GFLOP, 0.65 PFLOP/s; the attention kernel takes 80).
template <int TYPE, int D>
__global__ __launch_bounds__(kPrefixWaves * 64) void kv8_prefix_kernel(Kv8AttendArgs a) {
    typedef typename Elem<TYPE>::T T;
    constexpr int W = kPrefixWaves;
    constexpr bool KH = TYPE == kF16;        // keys in the queries' type; values and P in fp16
    constexpr int G = D / 8;                 // granules of a row of keys
    constexpr int S = D / 16;                // steps of the first product
    constexpr int DT = D / 32;               // channel tiles
    constexpr int kTile = kBlk * D * 2;      // bytes of a block's keys (or values)
    typedef PrefixLds<D> L;
    constexpr int N = L::kChunks;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int n = lane & 31, g = lane >> 5;
    const Kv8 &c = a.cache;
    const int group = a.n_heads / c.n_kv;
    const int rows = a.q_len * group;
    const int tiles = (rows + W * 32 - 1) / (W * 32);
    const int head = (int)blockIdx.x % c.n_kv, at = (int)blockIdx.x / c.n_kv;
    const int row0 = at % tiles * W * 32 + wave * 32, split = at / tiles;
    const int shift = __builtin_ctz(c.page);
    const int len0 = a.lens[0], cap = (int)a.width << shift;
    const int len = len0 < 0 || len0 > cap ? 0 : len0;  // (no such length: the join's NaN)
    const int begin = split * a.chunk, end = min(begin + a.chunk, len);
    if (begin >= end) return;

    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t *const raw = lds + 2 * L::kWide;
    Page *const pages = (Page *)(raw + L::kAhead * L::kRaw);
    int64_t *const places = (int64_t *)(pages + kMaxPages);
    int *const range = (int *)(places + kMaxPages);  // largest, smallest exponent
    int *const dirty = range + 2;
    if (threadIdx.x == 0) range[0] = 0, range[1] = 255, *dirty = 0;
    const float to_log2 = fabsf(a.scale) * 1.4426950408889634f;
    const int first_page = begin >> shift;
    for (int i = threadIdx.x; i << shift < a.chunk + kBlk; i += W * 64) {
        const int pos = (first_page + i) << shift;
        int id = pos < end ? a.table[first_page + i] : 0;  // past the end: any page does, its codes are masked
        const bool none = id < 0 || id >= c.n_pages;
        if (none) id = 0;
        places[i] = ((int64_t)id * c.n_kv + head) * ((int64_t)D << shift);
        pages[i].scale = none ? __builtin_nanf("") : 0.0f;
    }
    __syncthreads();

    // Blocks come by LDS DMA: chunk f of the keys is sixteen channels of position f / (D/16), of the
    // values sixteen positions (all in one page) of channel f / 4. A thread makes wide what
    // its own lane fetched.
    auto fetch = [&](int b0, int slot) {
        const uint32_t to = 2 * L::kWide + slot * L::kRaw + wave * 1024;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // (every wavefront fetches as much: the waits count)
            const int f = min(i * W * 64 + (int)threadIdx.x, 4 * D - 1);
            const int kpos = b0 + f / (D / 16), vpos = b0 + f % 4 * 16;
            const int64_t k0 = places[(kpos >> shift) - first_page], v0 = places[(vpos >> shift) - first_page];
            dma16(c.k + k0 + ((kpos & (c.page - 1)) * D + f % (D / 16) * 16), to + i * W * 1024);
            dma16(c.v + v0 + ((f / 4 << shift) + (vpos & (c.page - 1))), to + (N + i) * W * 1024);
        }
    };
    // A block behind the last is fetched like the others, from the last one's place.
    const int final_block = begin + (end - 1 - begin) / kBlk * kBlk;
#pragma unroll
    for (int i = 0; i < L::kAhead; ++i) fetch(min(begin + i * kBlk, final_block), i);

    for (int i = threadIdx.x; i << shift < a.chunk + kBlk; i += W * 64) {
        int v = 127;
        if ((first_page + i) << shift < end && pages[i].scale == 0) {
            const int64_t p = places[i] / ((int64_t)D << shift);
            v = c.v_scales[p];
            pages[i].scale = v == 255 ? __builtin_nanf("") : e8m0(c.k_scales[p]) * to_log2;
            if (v != 255) atomicMax(&range[0], v), atomicMin(&range[1], v);
        }
        pages[i].rest = v;
    }

    // the row, its queries' parts, the last position that it sees
    const bool live = row0 + n < rows;
    const int token = live ? (row0 + n) / group : 0;
    const int64_t out_row = (int64_t)token * a.n_heads + head * group + (row0 + n) % group;
    u32x4 q[S];
    {
        const T *p = (const T *)a.q + token * a.q_stride + (int64_t)(head * group + (row0 + n) % group) * D;
        const bool vec = ((uintptr_t)a.q | (uintptr_t)a.q_stride * sizeof(T)) % 16 == 0;
        const float sign = a.scale < 0 ? -1.0f : 1.0f;  // (the maximum is taken before the scale)
        auto load = [&](auto vec) {
            float v[S][8];
#pragma unroll
            for (int s = 0; s < S; ++s) load8<T, vec.value>(p + s * 16 + g * 8, v[s]);
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v0 = v[s][2 * e] * sign, v1 = v[s][2 * e + 1] * sign;
                    q[s][e] = pack2<KH>(v0, v1);
                }
        };
        if (vec) load(std::true_type{});
        else load(std::false_type{});
    }
    const int own = a.tails[token / a.tail_q_len] - a.tail_q_len + token % a.tail_q_len;
    const int last = len - 1 + min(own + 1, 0);
    // positions that every row of the workgroup sees
    int by_all = len;
    {
        const int r0 = at % tiles * W * 32, s0 = r0 / group / a.tail_q_len;
        const int s1 = min(r0 + W * 32 - 1, rows - 1) / group / a.tail_q_len;
        for (int s = s0 + lane; s <= s1; s += 64) by_all = min(by_all, len + min(a.tails[s] - a.tail_q_len + 1, 0));
#pragma unroll
        for (int o = 32; o; o >>= 1) by_all = min(by_all, __shfl_xor(by_all, o));
        by_all = __builtin_amdgcn_readfirstlane(by_all);
    }
    __syncthreads();
    const int largest = range[0], least = max(largest - kPowers, 0);
    const bool far = range[1] < least;
    for (int i = threadIdx.x; i << shift < a.chunk + kBlk; i += W * 64) {
        const int v = (int)pages[i].rest;
        pages[i].power = max(v, least) - largest;
        pages[i].inverse = __builtin_amdgcn_exp2f(largest - max(v, least));
        pages[i].rest = v < least ? __builtin_amdgcn_exp2f(v - least) : 1.0f;
    }

    auto put = [&](int b0, int slot, int buf) {
        uint8_t *const k_lds = lds + buf * L::kWide, *const v_lds = k_lds + kTile;
        const uint8_t *const from = raw + slot * L::kRaw + threadIdx.x * 16;
        const bool whole = b0 + kBlk <= by_all;
        bool found = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int f = i * W * 64 + threadIdx.x;
            if (4 * D % (W * 64) != 0 && f >= 4 * D) break;
            const int r = f / (D / 16), gr = f % (D / 16) * 2, ch = f / 4, piece = f % 4;
            u32x4 k = *(const u32x4 *)(from + i * W * 1024), v = *(const u32x4 *)(from + (N + i) * W * 1024);
            if (!whole) {
                // codes past the end are whatever the pool held; a NaN that some rows do not see
                // is left to the end
                const int keep = min(max(len - b0 - piece * 16, 0), 16);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int x = keep - w * 4;
                    v[w] &= x >= 4 ? ~0u : x <= 0 ? 0u : (1u << (8 * x)) - 1u;
                    const uint32_t bad = nan_bytes(v[w]) >> 7;
                    if (bad) v[w] &= ~(bad * 0xffu), found = true;
                }
            }
            const u32x2 k0 = widened<KH>(k[0]), k1 = widened<KH>(k[1]), k2 = widened<KH>(k[2]), k3 = widened<KH>(k[3]);
            const u32x2 v0 = widened<true>(v[0]), v1 = widened<true>(v[1]), v2 = widened<true>(v[2]), v3 = widened<true>(v[3]);
            const int kk = row_key<G>(r), vk = row_key<8>(ch);
            *(u32x4 *)(k_lds + (r * G + (gr ^ kk)) * 16) = u32x4{k0[0], k0[1], k1[0], k1[1]};
            *(u32x4 *)(k_lds + (r * G + ((gr + 1) ^ kk)) * 16) = u32x4{k2[0], k2[1], k3[0], k3[1]};
            *(u32x4 *)(v_lds + (ch * 8 + ((piece * 2) ^ vk)) * 16) = u32x4{v0[0], v0[1], v2[0], v2[1]};
            *(u32x4 *)(v_lds + (ch * 8 + ((piece * 2 + 1) ^ vk)) * 16) = u32x4{v1[0], v1[1], v3[0], v3[1]};
        }
        if (found) *dirty = 1;
    };

    float top = -__builtin_inff(), sum = 0;
    f32x16 out[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) out[t][i] = 0;
    int v_at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v_at[j] = (n * 8 + ((j * 2 + g) ^ row_key<8>(n))) * 16;

    // the oldest of the blocks under way has arrived when 2 N (kAhead - 1) younger DMAs may be left
    auto make = [&](int b0, int slot, int buf) {
        wait_vmcnt<2 * N * (L::kAhead - 1)>();
        put(b0, slot, buf);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // it has been read: its place is free
        fetch(min(b0 + L::kAhead * kBlk, final_block), slot);
    };
    __syncthreads();  // (the pages' powers)
    make(begin, 0, 0);
    int buf = 0, slot = 1;
    for (int b0 = begin; b0 < end; b0 += kBlk, slot = slot + 1 == L::kAhead ? 0 : slot + 1) {
        __syncthreads();  // the block is made, and nobody reads the one before any more
        const uint8_t *const k_lds = lds + buf * L::kWide, *const v_lds = k_lds + kTile;
        buf ^= 1;
        if (b0 + kBlk < end) make(b0 + kBlk, slot, buf);
        if (row0 >= rows) continue;
        f32x16 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[u][i] = 0;
        {
            const uint8_t *const row = k_lds + n * G * 16;
            const int key = row_key<G>(n);
            // both halves' operands of a step in turn: two chains of sums
            products<2 * S, 1, 1>(
                [&](int i) { return *(const u32x4 *)(row + i % 2 * 32 * G * 16 + ((i / 2 * 2 + g) ^ key) * 16); },
                [&](int i, u32x4 k) { s[i % 2] = mfma32<KH>(k, q[i / 2], s[i % 2]); });
        }
        const bool whole = b0 + kBlk <= by_all;
        const int hi = last - b0 - g * 4;
        auto seen = [&](int u, int i) { return u * 32 + (i >> 2) * 8 + (i & 3) <= hi; };
        if (!whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!seen(u, i)) s[u][i] = -__builtin_inff();
        }
        // sixteen positions at a time lie in one page: this lane's eight of them
        Page page[4];
        float m = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            page[j] = pages[((b0 + j * 16) >> shift) - first_page];
            const f32x16 &x = s[j / 2];
            const int i = (j & 1) * 8;
            const float t = maximum3(maximum3(maximum3(x[i], x[i + 1], x[i + 2]), x[i + 3], x[i + 4]),
                                     maximum3(x[i + 5], x[i + 6], x[i + 7]), x[i]);
            const float y = t == -__builtin_inff() ? t : __builtin_fmaf(t, page[j].scale, page[j].power);
            m = maximum3(m, y, y);
        }
        m = max_halves(m);
        if (__any(m > top + kSlack)) {  // (every number is more than -infinity)
            const float now = fmaxf(top, m);
            const float alpha = now == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top - now);
            top = now;
            sum *= alpha;
#pragma unroll
            for (int t = 0; t < DT; ++t) out[t] *= alpha;
        }
        const float base = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float x = __builtin_fmaf(s[i / 16][i % 16], page[i / 8].scale, page[i / 8].power - base);
            s[i / 16][i % 16] = __builtin_amdgcn_exp2f(x);
        }
        if (!whole) {  // (-infinity times a scale of zero, or of NaN, is none)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!seen(i / 16, i % 16)) s[i / 16][i % 16] = 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x16 &x = s[j / 2];
            const int i = (j & 1) * 8;
            const float part = ((x[i] + x[i + 1]) + (x[i + 2] + x[i + 3])) + ((x[i + 4] + x[i + 5]) + (x[i + 6] + x[i + 7]));
            sum = __builtin_fmaf(part, page[j].inverse, sum);
        }
        if (far) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i / 16][i % 16] *= page[i / 8].rest;
        }
        u32x4 w[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = pack2<true>(s[i / 8][i % 8 * 2], s[i / 8][i % 8 * 2 + 1]);
        products<4 * DT, 1, 1>([&](int i) { return *(const u32x4 *)(v_lds + v_at[i / DT] + i % DT * 32 * 8 * 16); },
                               [&](int i, u32x4 v) { out[i % DT] = mfma32<true>(v, w[i / DT], out[i % DT]); });
    }
    wait_vmcnt<0>();  // (no DMA outlives its workgroup's LDS)
    __syncthreads();
    const bool mend = *dirty != 0;
    const float total = sum_halves(sum);
    if (!live) return;
    const int64_t all = (int64_t)a.q_len * a.n_heads;
    float *part = a.partial + split * partial_floats(all, D);
    const float unit = e8m0(largest);  // (P's exponents count from the largest v)
    if (g == 0) part[all * D + out_row * 2] = top, part[all * D + out_row * 2 + 1] = total;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int d = t * 32 + i * 2 + g * 4;
            f32x4 o = f32x4{out[t][i], out[t][i + 1], out[t][i + 2], out[t][i + 3]} * unit;
            if (mend) {  // the NaNs of positions that some rows do not see
                for (int pos = max(begin, by_all & -kBlk); pos <= min(last, end - 1); ++pos) {
                    const uint8_t *codes = c.v + places[(pos >> shift) - first_page] + (pos & (c.page - 1));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((codes[(int64_t)(d + e) << shift] & 127) == 127) o[e] = __builtin_nanf("");
                }
            }
            *(f32x4 *)(part + out_row * D + d) = o;
        }
}

template <int TYPE, int D>
hipError_t prefix(const Kv8AttendArgs &a, hipStream_t s) {
    const int64_t rows = (int64_t)a.q_len * (a.n_heads / a.cache.n_kv), tiles = (rows + kPrefixRows - 1) / kPrefixRows;
    kv8_prefix_kernel<TYPE, D><<<(unsigned)(tiles * a.max_splits * a.cache.n_kv), kPrefixWaves * 64,
                                 PrefixLds<D>::kBytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Whether the prefix's pass takes kv8_prefix_kernel, and its splits. It does in 16 bits, up to 128
// channels, where rows and the positions that the prefix's pages may hold are many: a workgroup's
// start and end, and a split's sums on their way through memory, have to be small beside its blocks.
// Elsewhere attention's own kernel, whose wavefronts share a split's positions and not its rows, takes
// less (prefix's and own pass together, us, this and that: 256 rows of 256 channels, 4 key/value heads
// behind 20,000 positions, 83 and 73; fp32, 1000 rows of 64 behind 4000 35 and 34, of 128 73 and 52).
// Where the kernels cross (rows x heads x positions in 2^20, the switch being at 15): 256 rows, 8 heads
// of 128 behind 6000 (12) 34.0 and 31.7, behind 10,000 (20) 40.0 and 39.4, behind 16,000 (31) 46 and 51;
// 1000 rows of these behind 1500 (12) 53 and 51, 1920 (15) 51.7 and 54.2, 3000 (23) 56 and 63; of 4 heads
// of 64 behind 2000 (8) 24.6 and 24.6, 3900 (15) 27.4 and 30.9; 256 rows, 2 heads of 128 behind 30,000
// (15) 43.5 and 41.0: within 13% of the better one.
// The rows also have to fill three quarters of the tiles, which keeps the kernel from rows that it
// would be faster for: 260 to 380 rows, 8 heads of 128 behind 32,000 85-88 and 123-126, 520 143 and 203,
// 128 49 and 54; 320 rows, 4 heads of 64 behind 16,000 34 and 41, 264 34.0 and 34.7.
bool kv8_prefix_plan(Kv8AttendArgs &a, int type, int cus) {
    const int64_t rows = (int64_t)a.q_len * (a.n_heads / a.cache.n_kv), cap = a.width * a.cache.page;
    const int64_t tiles = (rows + kPrefixRows - 1) / kPrefixRows;
    if (type == kF32 || a.cache.dim > 128 || rows * a.cache.n_kv * cap < 15 << 20 || rows * 4 < tiles * kPrefixRows * 3)
        return false;
    // a workgroup to each compute unit
    int64_t chunk = (cap * a.cache.n_kv * tiles + cus - 1) / cus;
    chunk = std::min<int64_t>(std::max<int64_t>((chunk + kBlk - 1) / kBlk * kBlk, 256), kMaxChunk);
    a.chunk = (int)chunk;
    a.max_splits = (int)((cap + chunk - 1) / chunk);
    return true;
}

hipError_t launch_kv8_prefix(const Kv8AttendArgs &a, int type, hipStream_t s) {
    const bool half = type == kF16;
    switch (a.cache.dim) {
        case 64: return half ? prefix<kF16, 64>(a, s) : prefix<kBF16, 64>(a, s);
        case 96: return half ? prefix<kF16, 96>(a, s) : prefix<kBF16, 96>(a, s);
        default: return half ? prefix<kF16, 128>(a, s) : prefix<kBF16, 128>(a, s);
    }
}

}  // namespace qwg
