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

// (token, head) rows of qwg_prompt_attend, and its (sequence, key/value head) pairs: a grid of
// tiles of 32 rows then stays below the 2^32 threads of a launch.
constexpr int64_t kMaxPromptRows = (int64_t)1 << 28, kMaxPromptPairs = (int64_t)1 << 22;

// Elements between two of its tokens' keys: a block of 64 then spans less than 2^32 bytes.
constexpr int64_t kMaxPromptStride = 1 << 23;

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

// `rows` rows of `width` elements, `stride` apart, from `p`: where they lie.
struct Rows {
    const void *p;
    int64_t rows, width, stride;
    uintptr_t size;
};

// Whether two such blocks may share memory: rows at one distance interleave as the slices of
// a fused result do, others are told apart by their ends.
bool may_share(const Rows &a, const Rows &b) {
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uintptr_t a1 = a0 + ((uintptr_t)(a.rows - 1) * a.stride + a.width) * a.size;
    const uintptr_t b1 = b0 + ((uintptr_t)(b.rows - 1) * b.stride + b.width) * b.size;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return true;
    const uintptr_t pitch = (uintptr_t)a.stride * a.size;
    const uintptr_t ahead = b0 >= a0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
    return ahead < a.width * a.size || pitch - ahead < b.width * b.size;
}

// Whether `out` may not be written while `x` is read: x is all of out's rows (in_place: each is read by
// the one workgroup that writes it, before), or shares none of their memory.
bool clashes(const Rows &out, const Rows &x, bool in_place) {
    return may_share(out, x) && !(in_place && out.p == x.p && (out.rows == 1 || out.stride == x.stride));
}

// Rows of qwg_kv8_attend_shared: the prefix's tiles of 16 then fit the y of a grid.
constexpr int64_t kMaxSharedRows = 1 << 20;

int shared_shape(const qwg_kv8 *c, int64_t prefix_width, int64_t width, int64_t n_seqs, int q_len,
                 int n_heads) {
    const int rc = attend_shape(c, width, n_seqs, q_len, n_heads, 0);
    if (rc) return rc;
    if (!cache_seqs(c, prefix_width, 1) || n_seqs * q_len * n_heads > kMaxSharedRows)
        return QWG_ERR_SHAPE;
    return QWG_OK;
}

Kv8SharedArgs shared_of(const qwg_kv8 *cache, int type, int64_t prefix_width, int64_t width, int64_t n_seqs,
                        int q_len, int n_heads) {
    Kv8SharedArgs a = {};
    a.own.cache = cache_of(cache), a.own.width = width, a.own.n_seqs = n_seqs;
    a.own.q_len = q_len, a.own.n_heads = n_heads;
    a.prefix = a.own;
    a.prefix.parts = true;
    a.prefix.width = prefix_width, a.prefix.n_seqs = 1, a.prefix.q_len = (int)n_seqs * q_len;
    a.prefix.tail_q_len = q_len;
    kv8_shared_plan(a, type, kCus);
    return a;
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

int qwg_kv8_append_rotary(const qwg_kv8 *cache, void *q_out, int64_t q_out_stride, void *k_out,
                          int64_t k_out_stride, const void *q, int64_t q_stride, const void *k,
                          int64_t k_stride, const void *v, int64_t v_stride, int type, int n_heads,
                          const float *freqs, int rotary_dim, int interleaved,
                          const int32_t *prefix_len, int64_t n_tokens,
                          const int32_t *starts, const int32_t *table, int64_t table_width,
                          const int32_t *lens, int64_t n_seqs, int64_t max_new, void *stream) {
    if (!cache || !q_out || !q || !k || !v || !freqs || !table || !lens) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (n_heads < 1 || n_heads > 65535 || n_heads % cache->n_kv_heads || rotary_dim < 16 ||
        rotary_dim % 16 || rotary_dim > cache->head_dim)
        return QWG_ERR_SHAPE;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    const int64_t q_width = (int64_t)n_heads * cache->head_dim;
    if (!cache_seqs(cache, table_width, n_seqs) || n_tokens < 1 || n_tokens > INT32_MAX ||
        max_new < 1 || (!starts && n_tokens % n_seqs) ||
        (n_tokens > 1 && (k_stride < width || v_stride < width || q_stride < q_width ||
                          q_out_stride < q_width || (k_out && k_out_stride < width))))
        return QWG_ERR_SHAPE;
    const uintptr_t size = size_of(type);
    if (!aligned(k, size) || !aligned(v, size) || !aligned(q, size) || !aligned(q_out, size) ||
        !aligned(k_out, size) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4) ||
        !aligned(freqs, 4) || !aligned(prefix_len, 4))
        return QWG_ERR_ALIGN;
    // workgroups read and write in no order
    const Rows rk = {k, n_tokens, width, k_stride, size}, rv = {v, n_tokens, width, v_stride, size};
    const Rows rq = {q, n_tokens, q_width, q_stride, size};
    const Rows oq = {q_out, n_tokens, q_width, q_out_stride, size};
    const Rows ok = {k_out, n_tokens, width, k_out_stride, size};
    if (clashes(oq, rk, false) || clashes(oq, rv, false) || clashes(oq, rq, true) ||
        (k_out && (clashes(ok, rk, false) || clashes(ok, rv, false) || clashes(ok, rq, false) || clashes(ok, oq, false))))
        return QWG_ERR_OVERLAP;
    Kv8RotaryArgs a = {};
    static_cast<Kv8AppendArgs &>(a) = {cache_of(cache), k, v, k_stride, v_stride, n_tokens, starts,
                                       table, lens, table_width, n_seqs, max_new};
    a.q = q, a.q_out = q_out, a.k_out = k_out;
    a.q_stride = q_stride, a.q_out_stride = q_out_stride, a.k_out_stride = k_out_stride;
    a.freqs = freqs, a.before = prefix_len, a.n_heads = n_heads, a.rotary = rotary_dim, a.neighbours = interleaved != 0;
    return hip_status(launch_kv8_append_rotary(a, type, (hipStream_t)stream));
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

int64_t qwg_kv8_attend_shared_workspace(const qwg_kv8 *cache, int type, int64_t prefix_width,
                                        int64_t table_width, int64_t n_seqs, int q_len,
                                        int n_heads) {
    int rc = check_cache(cache);
    if (!rc && !known_type(type)) rc = QWG_ERR_TYPE;
    if (!rc) rc = shared_shape(cache, prefix_width, table_width, n_seqs, q_len, n_heads);
    if (rc) return -rc;
    return kv8_shared_partial_bytes(shared_of(cache, type, prefix_width, table_width, n_seqs, q_len, n_heads));
}

int qwg_kv8_attend_shared(const qwg_kv8 *cache, void *out, const void *q, int type, int64_t q_stride,
                          const int32_t *prefix, int64_t prefix_width, const int32_t *prefix_len,
                          const int32_t *table, int64_t table_width, const int32_t *lens,
                          int64_t n_seqs, int q_len, int n_heads, float scale, void *workspace,
                          int64_t workspace_bytes, void *stream) {
    if (!cache || !out || !q || !prefix || !prefix_len || !table || !lens || !workspace)
        return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    int rc = check_cache(cache);
    if (!rc) rc = shared_shape(cache, prefix_width, table_width, n_seqs, q_len, n_heads);
    if (rc) return rc;
    if (n_seqs * q_len > 1 && q_stride < (int64_t)n_heads * cache->head_dim) return QWG_ERR_SHAPE;
    if (!aligned(q, size_of(type)) || !aligned(out, size_of(type)) || !aligned(prefix, 4) ||
        !aligned(prefix_len, 4) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(workspace, 16))
        return QWG_ERR_ALIGN;
    const int64_t n = n_seqs * q_len, q_width = (int64_t)n_heads * cache->head_dim;
    const uintptr_t size = size_of(type);
    if (clashes({out, n, q_width, q_width, size}, {q, n, q_width, q_stride, size}, true)) return QWG_ERR_OVERLAP;
    Kv8SharedArgs a = shared_of(cache, type, prefix_width, table_width, n_seqs, q_len, n_heads);
    if (kv8_shared_partial_bytes(a) > workspace_bytes) return QWG_ERR_SHAPE;
    for (Kv8AttendArgs *p : {&a.prefix, &a.own}) p->q = q, p->out = out, p->q_stride = q_stride, p->scale = scale;
    a.prefix.table = prefix, a.prefix.lens = prefix_len, a.prefix.tails = lens;
    a.own.table = table, a.own.lens = lens;
    a.prefix.partial = (float *)workspace;
    return hip_status(launch_kv8_attend_shared(a, type, (hipStream_t)stream));
}

int qwg_prompt_attend(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, int type, int64_t n_tokens,
                      const int32_t *starts, int64_t n_seqs, int64_t max_len, int n_heads,
                      int n_kv_heads, int head_dim, float scale, int64_t window, void *stream) {
    if (!out || !q || !k || !v) return QWG_ERR_NULL;
    if (!known_type(type)) return QWG_ERR_TYPE;
    if (!kv8_dim_supported(head_dim) || n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < 1 ||
        n_heads > 65535 || n_heads % n_kv_heads)
        return QWG_ERR_SHAPE;
    const int64_t width = (int64_t)n_kv_heads * head_dim, q_width = (int64_t)n_heads * head_dim;
    if (n_seqs < 1 || n_seqs > kMaxPromptPairs || n_seqs * n_kv_heads > kMaxPromptPairs ||
        n_tokens < 1 || n_tokens > kMaxPromptRows || n_tokens * n_heads > kMaxPromptRows ||
        max_len < 0 || window < 0 || (!starts && n_tokens % n_seqs) ||
        (n_tokens > 1 && (q_stride < q_width || k_stride < width || v_stride < width ||
                          k_stride > kMaxPromptStride || v_stride > kMaxPromptStride)))
        return QWG_ERR_SHAPE;
    const uintptr_t size = size_of(type);
    if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(out, size) ||
        !aligned(starts, 4))
        return QWG_ERR_ALIGN;
    const Rows ro = {out, n_tokens, q_width, q_width, size};
    if (clashes(ro, {k, n_tokens, width, k_stride, size}, false) || clashes(ro, {v, n_tokens, width, v_stride, size}, false) ||
        clashes(ro, {q, n_tokens, q_width, q_stride, size}, true))
        return QWG_ERR_OVERLAP;
    PromptArgs a = {q, k, v, out, q_stride, k_stride, v_stride, starts, n_tokens, n_seqs, window,
                    n_heads, n_kv_heads, head_dim, scale, false};
    if (n_tokens == 1) a.q_stride = q_width, a.k_stride = a.v_stride = width;
    a.vec = aligned(q, 16) && aligned(k, 16) && aligned(v, 16) &&
            (a.q_stride | a.k_stride | a.v_stride) * size % 16 == 0;
    return hip_status(launch_prompt_attend(a, type, (hipStream_t)stream));
}

}  // extern "C"
