// Interfaces between the host boundary (mx_api.cpp) and the kernels of the
// microscaled weights (mx.hip, mx_gemm.hip, mx_matmul.hip) and of the 8-bit
// key/value cache (kv8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qwg {

constexpr int kMxBlock = 32;      // values per E8M0 scale
constexpr int kMxCodeBytes = 16;  // packed E2M1 codes of one block
constexpr int kMxMaxBatch = 16;   // rows of qwg_gemm_mxfp4

// element types of activations and results
enum { kF32 = 0, kF16 = 1, kBF16 = 2 };

struct MxGemmArgs {
    const uint8_t *codes;   // [n_out][n_in/2]
    const uint8_t *scales;  // [n_out][n_in/32]
    const void *x;          // [batch][n_in]
    void *y;                // [batch][n_out]
    int n_in, n_out, batch;
};

struct MxMatmulArgs {
    const uint8_t *a, *a_scales;  // [n_rows][n_in/2], [n_rows][n_in/32]
    const uint8_t *w, *w_scales;  // [n_out][n_in/2], [n_out][n_in/32]
    void *c;                      // [n_rows][n_out]
    int64_t n_rows, n_out;
    int n_in;
};

// One 8-bit cache: K pages [n_pages][n_kv][page][dim], V pages
// [n_pages][n_kv][dim][page] (e4m3 codes), scales [n_pages][n_kv] (E8M0).
struct Kv8 {
    uint8_t *k, *v, *k_scales, *v_scales;
    int64_t n_pages;
    int n_kv, dim, page;
};

struct Kv8AppendArgs {
    Kv8 cache;
    const void *k, *v;          // [n_tokens][n_kv][dim], token strides below
    int64_t k_stride, v_stride;  // elements
    int64_t n_tokens;
    const int32_t *starts;  // [n_seqs + 1], or null: n_tokens / n_seqs tokens each
    const int32_t *table;   // [n_seqs][width]
    const int32_t *lens;    // tokens held before the call
    int64_t width, n_seqs, max_new;
};

struct Kv8AttendArgs {
    Kv8 cache;
    const void *q;  // [n_seqs * q_len][n_heads][dim], token stride below
    void *out;      // [n_seqs * q_len][n_heads][dim]
    int64_t q_stride;
    const int32_t *table;  // [n_seqs][width]
    const int32_t *lens;   // tokens held, the queries' own among them
    int64_t width, n_seqs, window;
    int q_len, n_heads;
    float scale;
    int row_tiles;   // tiles of 16 rows per workgroup
    int chunk;       // positions per split (a multiple of 64)
    int max_splits;  // splits of a sequence that fills its table or window
    bool brief;      // more workgroups than fit at once, as far as known of 512 positions at most
    bool few;        // as far as known one split each, and no more workgroups, empty ones too, than compute units
    float *partial;  // [n_seqs][max_splits][q_len * n_heads][dim + 2], or null for one split
};

hipError_t launch_mxfp4_encode(uint8_t *codes, uint8_t *scales, const void *x, int type,
                               int64_t n_rows, int64_t n_in, int64_t x_stride, hipStream_t s);
hipError_t launch_mxfp4_dequant(const uint8_t *codes, const uint8_t *scales, void *dst, int type,
                                int64_t n, hipStream_t s);
hipError_t launch_mxfp4_gemm(const MxGemmArgs &a, int type, hipStream_t s);
hipError_t launch_mxfp4_matmul(const MxMatmulArgs &a, int type, hipStream_t s);
hipError_t launch_kv8_append(const Kv8AppendArgs &a, int type, hipStream_t s);
bool kv8_dim_supported(int dim);
// Sets what shapes the launch: row_tiles, chunk, max_splits, few and brief.
void kv8_attend_plan(Kv8AttendArgs &a, int64_t max_len, int cus);
int64_t kv8_attend_partial_bytes(const Kv8AttendArgs &a);
hipError_t launch_kv8_attend(const Kv8AttendArgs &a, int type, hipStream_t s);

}  // namespace qwg
