// C ABI of the MXFP4 and 8-bit cache calls (declared in include/qwg.h):
// argument validation and launch. Every check runs on the host before any HIP
// call, and no call allocates or keeps anything.
#include <hip/hip_runtime.h>

#include "../../include/qwg.h"
#include "mx_internal.h"

using namespace qwg;

namespace {

static_assert(QWG_F32 == kF32 && QWG_F16 == kF16 && QWG_BF16 == kBF16, "element types");
static_assert(QWG_MX_BLOCK == kMxBlock && QWG_MX_MAX_BATCH == kMxMaxBatch, "MXFP4 sizes");

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? QWG_OK : QWG_ERR_HIP; }

bool known_type(int type) { return type == QWG_F32 || type == QWG_F16 || type == QWG_BF16; }

uintptr_t size_of(int type) { return type == QWG_F32 ? 4 : 2; }

bool mx_width(int64_t n_in) {
    return n_in >= QWG_MX_BLOCK && n_in <= QWG_MAX_N_IN && n_in % QWG_MX_BLOCK == 0;
}

bool mx_count(int64_t n) { return n >= 1 && n <= QWG_MAX_N_OUT; }

// Outputs of qwg_matmul_mxfp4: a grid of large tiles (2^22 and the edges' at most) then
// stays below the 2^32 threads of a launch. In 16 bits they are 512 GB, more than the memory.
constexpr int64_t kMaxOutputs = (int64_t)1 << 38;

// Compute units of a current MI355X; the plan of a split needs no exact figure.
constexpr int kCus = 256;

int check_cache(const qwg_kv8 *c) {
    if (!c || !c->k_pages || !c->v_pages || !c->k_scales || !c->v_scales) return QWG_ERR_NULL;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->n_kv_heads < 1 || c->n_kv_heads > 1024 ||
        !kv8_dim_supported(c->head_dim))
        return QWG_ERR_SHAPE;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 &&
        c->page_tokens != 128)
        return QWG_ERR_SHAPE;
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return QWG_ERR_ALIGN;
    return QWG_OK;
}

bool cache_seqs(const qwg_kv8 *c, int64_t width, int64_t n_seqs) {
    return width >= 1 && width <= (1 << 30) / c->page_tokens && n_seqs >= 1 && n_seqs <= 65535;
}

Kv8 cache_of(const qwg_kv8 *c) {
    return Kv8{(uint8_t *)c->k_pages, (uint8_t *)c->v_pages, c->k_scales, c->v_scales,
               c->n_pages, c->n_kv_heads, c->head_dim, c->page_tokens};
}

int attend_shape(const qwg_kv8 *c, int64_t width, int64_t n_seqs, int q_len, int n_heads,
                 int64_t max_len) {
    if (!cache_seqs(c, width, n_seqs) || q_len < 1 || n_heads < 1 || n_heads % c->n_kv_heads ||
        (int64_t)q_len * n_heads > 65535 || max_len < 0)
        return QWG_ERR_SHAPE;
    return QWG_OK;
}

}  // namespace

extern "C" {

int qwg_encode_mxfp4(void *codes, void *scales, const void *x, int type, int64_t n_rows,
                     int64_t n_in, int64_t x_stride, void *stream) {
    if (!codes || !scales || !x) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    if (!mx_width(n_in) || !mx_count(n_rows) || x_stride < n_in) return QWG_ERR_SHAPE;
    if (!aligned(codes, 16) || !aligned(x, size_of(type))) return QWG_ERR_ALIGN;
    return hip_status(launch_mxfp4_encode((uint8_t *)codes, (uint8_t *)scales, x, type, n_rows,
                                          n_in, x_stride, (hipStream_t)stream));
}

int qwg_dequant_mxfp4(const void *codes, const void *scales, void *dst, int type, int64_t n,
                      void *stream) {
    if (!codes || !scales || !dst) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    if (n < QWG_MX_BLOCK || n % QWG_MX_BLOCK) return QWG_ERR_SHAPE;
    if (!aligned(codes, 16) || !aligned(dst, 16)) return QWG_ERR_ALIGN;
    return hip_status(launch_mxfp4_dequant((const uint8_t *)codes, (const uint8_t *)scales, dst,
                                           type, n, (hipStream_t)stream));
}

int qwg_gemm_mxfp4(void *y, const void *x, int type, const void *codes, const void *scales,
                   int64_t n_in, int64_t n_out, int batch, void *stream) {
    if (!y || !x || !codes || !scales) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    if (!mx_width(n_in) || !mx_count(n_out)) return QWG_ERR_SHAPE;
    if (batch < 1 || batch > QWG_MX_MAX_BATCH) return QWG_ERR_BATCH;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(y, size_of(type))) return QWG_ERR_ALIGN;
    const MxGemmArgs a = {(const uint8_t *)codes, (const uint8_t *)scales, x, y, (int)n_in,
                          (int)n_out, batch};
    return hip_status(launch_mxfp4_gemm(a, type, (hipStream_t)stream));
}

int qwg_gemv_mxfp4(void *y, const void *x, int type, const void *codes, const void *scales,
                   int64_t n_in, int64_t n_out, void *stream) {
    return qwg_gemm_mxfp4(y, x, type, codes, scales, n_in, n_out, 1, stream);
}

int qwg_matmul_mxfp4(void *c, int type, const void *a_codes, const void *a_scales,
                     const void *w_codes, const void *w_scales, int64_t n_rows, int64_t n_in,
                     int64_t n_out, void *stream) {
    if (!c || !a_codes || !a_scales || !w_codes || !w_scales) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    if (!mx_width(n_in) || !mx_count(n_out) || !mx_count(n_rows) || n_rows * n_out > kMaxOutputs)
        return QWG_ERR_SHAPE;
    if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(c, size_of(type)))
        return QWG_ERR_ALIGN;
    const MxMatmulArgs a = {(const uint8_t *)a_codes, (const uint8_t *)a_scales,
                            (const uint8_t *)w_codes, (const uint8_t *)w_scales, c, n_rows, n_out,
                            (int)n_in};
    return hip_status(launch_mxfp4_matmul(a, type, (hipStream_t)stream));
}

int qwg_kv8_append(const qwg_kv8 *cache, const void *k, const void *v, int type, int64_t k_stride,
                   int64_t v_stride, int64_t n_tokens, const int32_t *starts,
                   const int32_t *table, int64_t table_width, const int32_t *lens, int64_t n_seqs,
                   int64_t max_new, void *stream) {
    if (!cache || !k || !v || !table || !lens) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    const int rc = check_cache(cache);
    if (rc) return rc;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (!cache_seqs(cache, table_width, n_seqs) || n_tokens < 1 || n_tokens > INT32_MAX ||
        max_new < 1 || (!starts && n_tokens % n_seqs) ||
        (n_tokens > 1 && (k_stride < width || v_stride < width)))
        return QWG_ERR_SHAPE;
    if (!aligned(k, size_of(type)) || !aligned(v, size_of(type)) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(starts, 4))
        return QWG_ERR_ALIGN;
    const Kv8AppendArgs a = {cache_of(cache), k, v, k_stride, v_stride, n_tokens, starts, table,
                             lens, table_width, n_seqs, max_new};
    return hip_status(launch_kv8_append(a, type, (hipStream_t)stream));
}

int64_t qwg_kv8_attend_workspace(const qwg_kv8 *cache, int64_t table_width, int64_t n_seqs,
                                 int q_len, int n_heads, int64_t window, int64_t max_len) {
    int rc = check_cache(cache);
    if (!rc) rc = attend_shape(cache, table_width, n_seqs, q_len, n_heads, max_len);
    if (!rc && window < 0) rc = QWG_ERR_SHAPE;
    if (rc) return -rc;
    Kv8AttendArgs a = {};
    a.cache = cache_of(cache);
    a.width = table_width, a.n_seqs = n_seqs, a.q_len = q_len, a.n_heads = n_heads;
    a.window = window;
    kv8_attend_plan(a, max_len, kCus);
    return kv8_attend_partial_bytes(a);
}

int qwg_kv8_attend(const qwg_kv8 *cache, void *out, const void *q, int type, int64_t q_stride,
                   const int32_t *table, int64_t table_width, const int32_t *lens, int64_t n_seqs,
                   int q_len, int n_heads, float scale, int64_t window, int64_t max_len,
                   void *workspace, int64_t workspace_bytes, void *stream) {
    if (!cache || !out || !q || !table || !lens) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    int rc = check_cache(cache);
    if (!rc) rc = attend_shape(cache, table_width, n_seqs, q_len, n_heads, max_len);
    if (rc) return rc;
    if (window < 0 || (n_seqs * q_len > 1 && q_stride < (int64_t)n_heads * cache->head_dim))
        return QWG_ERR_SHAPE;
    if (!aligned(q, size_of(type)) || !aligned(out, size_of(type)) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(workspace, 16))
        return QWG_ERR_ALIGN;
    Kv8AttendArgs a = {};
    a.cache = cache_of(cache);
    a.q = q, a.out = out, a.q_stride = q_stride, a.table = table, a.lens = lens;
    a.width = table_width, a.n_seqs = n_seqs, a.window = window;
    a.q_len = q_len, a.n_heads = n_heads, a.scale = scale;
    kv8_attend_plan(a, max_len, kCus);
    const int64_t need = kv8_attend_partial_bytes(a);
    if (need > 0 && !workspace) return QWG_ERR_NULL;
    if (need > workspace_bytes) return QWG_ERR_SHAPE;
    a.partial = (float *)workspace;
    return hip_status(launch_kv8_attend(a, type, (hipStream_t)stream));
}

}  // extern "C"
