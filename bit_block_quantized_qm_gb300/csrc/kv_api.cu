// The C ABI of the 4-bit key/value cache (declared in include/qm.h): argument
// checks, then launches on the caller's stream.  Page tables, lengths and row
// offsets are device memory that the host does not read: the kernels check
// them and set the device error word (QM_ERR_RANGE from qm_device_status).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "qm.h"
#include "qm_checks.h"
#include "qm_internal.h"

namespace {

using qm::check_pointer;
using qm::from_cuda;
using qm::mul_ok;
using qm::overlaps;

constexpr int64_t kMaxLen = int64_t(1) << 30;
static_assert(qm::kAttnZeroed == QM_ATTN_WORKSPACE_ZEROED, "the header's number");

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    const void* p;
    int64_t n;
};
// Whether `a` shares bytes with one of the others.
bool meets(const Range& a, std::initializer_list<Range> others) {
    for (const Range& b : others)
        if (a.p && b.p && overlaps(a.p, a.n, b.p, b.n)) return true;
    return false;
}
Range table_of(const qm_kv_cache* c) { return {c->page_table, int64_t(c->n_seqs) * c->table_stride * 4}; }
Range lengths_of(const qm_kv_cache* c) { return {c->lengths, int64_t(c->n_seqs) * 4}; }
Range starts_of(const qm_kv_cache* c, const int32_t* q_starts) { return {q_starts, (int64_t(c->n_seqs) + 1) * 4}; }

// A cache's sizes and pointers; fills the kernels' view and the pool's bytes.
int check_cache(const qm_kv_cache* c, qm::KvView* view, int64_t* pool_bytes) {
    if (!c) return QM_ERR_NULL;
    if (c->n_seqs < 0 || c->n_kv_heads < 1 || c->n_kv_heads > 65535 / 2 || c->head_dim < 32 || c->head_dim > 256 ||
        c->head_dim % 32 || c->page_tokens < 16 || c->page_tokens > 65536 ||
        (c->page_tokens & (c->page_tokens - 1)) || c->n_pages < 0 || c->n_pages > 0x7FFFFFFF || c->table_stride < 0 ||
        c->table_stride > 0x7FFFFFFF || c->n_seqs > 65535 || c->max_len < 0 || c->max_len > kMaxLen || c->reserved)
        return QM_ERR_SHAPE;
    if (c->max_len > c->table_stride * c->page_tokens) return QM_ERR_SHAPE;
    const int64_t page = int64_t(c->page_tokens) / 16 * 9 * c->head_dim;
    if (!mul_ok(c->n_pages, page * c->n_kv_heads, pool_bytes)) return QM_ERR_SHAPE;
    if (c->n_seqs > 0) {
        if (!c->lengths) return QM_ERR_NULL;
        if (c->max_len > 0 && (!c->k_pages || !c->v_pages || !c->page_table)) return QM_ERR_NULL;
    }
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->page_table, 4) || !aligned(c->lengths, 4))
        return QM_ERR_ALIGN;
    if (overlaps(c->k_pages, *pool_bytes, c->v_pages, *pool_bytes)) return QM_ERR_ALIAS;
    int shift = 4;
    while ((1 << shift) < c->page_tokens) ++shift;
    *view = {static_cast<uint8_t*>(c->k_pages), static_cast<uint8_t*>(c->v_pages), c->page_table, c->lengths,
             c->table_stride, c->max_len, static_cast<int>(c->n_pages), c->n_seqs, c->n_kv_heads, c->head_dim, shift, nullptr, 0};
    return QM_OK;
}

// The current device, and what the kernels need to know of it.
int on_device(qm::DeviceInfo* dev, qm::KvView* view) {
    if (qm::current_device_info(dev) != cudaSuccess) return QM_ERR_CUDA;
    view->sms = dev->sm_count;
    return from_cuda(qm::kv_error_word(dev->device, &view->err));
}

int check_cache_pointers(const qm_kv_cache* c, int device) {
    int rc = check_pointer(c->lengths, device);
    if (c->max_len > 0) {
        if (rc == QM_OK) rc = check_pointer(c->page_table, device);
        if (rc == QM_OK) rc = check_pointer(c->k_pages, device);
        if (rc == QM_OK) rc = check_pointer(c->v_pages, device);
    }
    return rc;
}

// The rows of a call.  Without q_starts every sequence has n_tokens / n_seqs.
int check_rows(const qm_kv_cache* c, int64_t n_tokens, int64_t max_q, const int32_t* q_starts, qm::KvRows* rows) {
    if (n_tokens < 0 || n_tokens > 0x7FFFFFFF || max_q < 0) return QM_ERR_SHAPE;
    if (!aligned(q_starts, 4)) return QM_ERR_ALIGN;
    int64_t uniform = 0;
    if (!q_starts && n_tokens > 0) {
        if (c->n_seqs == 0 || n_tokens % c->n_seqs) return QM_ERR_SHAPE;
        uniform = n_tokens / c->n_seqs;
        max_q = uniform;
    }
    if (max_q > n_tokens) max_q = n_tokens;
    if (max_q < 1 && n_tokens > 0) max_q = 1;  // (no kernel is made for sequences of no rows at all)
    *rows = {q_starts, static_cast<int>(uniform), static_cast<int>(n_tokens), static_cast<int>(max_q)};
    return QM_OK;
}

// Bytes from the first element of a [n][..] tensor with rows of `row` elements
// `stride` apart to its last; 0 for no rows.
int span(int64_t n, int64_t stride, int64_t row, int64_t item, int64_t* bytes) {
    if (stride < row || stride % 4) return QM_ERR_SHAPE;
    int64_t e;
    if (!mul_ok(n > 0 ? n - 1 : 0, stride, &e) || e > INT64_MAX / 8 - row) return QM_ERR_SHAPE;
    *bytes = n > 0 ? (e + row) * item : 0;
    return QM_OK;
}

int attn_sizes(const qm_kv_cache* c, int64_t n_heads) {
    return n_heads < 1 || n_heads > 0x7FFFFFFF / 256 || n_heads % c->n_kv_heads ? QM_ERR_SHAPE : QM_OK;
}

// The sizes that a workspace is asked for.  The rows' layout does not matter
// there: as if there were offsets.
int check_workspace(const qm_kv_cache* c, int64_t n_heads, int64_t n_tokens, int64_t max_q, qm::KvView* view,
                    qm::KvRows* rows) {
    int64_t pool;
    int rc = check_cache(c, view, &pool);
    if (rc == QM_OK) rc = attn_sizes(c, n_heads);
    if (rc == QM_OK) rc = check_rows(c, n_tokens, max_q, c->lengths, rows);
    return rc;
}

}  // namespace

extern "C" {

int qm_kv_append_q4_0(const qm_kv_cache* cache, const void* k, const void* v, int dtype, int64_t n_tokens,
                      int64_t k_stride, int64_t v_stride, const int32_t* q_starts, void* stream) {
    qm::KvView view;
    qm::KvRows rows;
    int64_t pool;
    int rc = check_cache(cache, &view, &pool);
    if (rc == QM_OK) rc = check_rows(cache, n_tokens, n_tokens, q_starts, &rows);
    if (rc != QM_OK) return rc;
    if (dtype != QM_F32 && dtype != QM_BF16) return QM_ERR_SHAPE;
    const int64_t row = int64_t(view.heads) * view.dim, item = dtype == QM_F32 ? 4 : 2;
    int64_t kb, vb;
    if ((rc = span(n_tokens, k_stride, row, item, &kb)) != QM_OK || (rc = span(n_tokens, v_stride, row, item, &vb)) != QM_OK)
        return rc;
    if (n_tokens == 0 || view.n_seqs == 0) return QM_OK;
    if (!k || !v) return QM_ERR_NULL;
    if (!aligned(k, 4 * item) || !aligned(v, 4 * item)) return QM_ERR_ALIGN;
    for (const void* p : {cache->k_pages, cache->v_pages})
        if (meets({p, pool}, {{k, kb}, {v, vb}, table_of(cache), lengths_of(cache), starts_of(cache, q_starts)}))
            return QM_ERR_ALIAS;
    qm::DeviceInfo dev;
    if (on_device(&dev, &view) != QM_OK) return QM_ERR_CUDA;
    rc = check_cache_pointers(cache, dev.device);
    if (rc == QM_OK) rc = check_pointer(k, dev.device);
    if (rc == QM_OK) rc = check_pointer(v, dev.device);
    if (rc == QM_OK && q_starts) rc = check_pointer(q_starts, dev.device);
    if (rc != QM_OK) return rc;
    return from_cuda(qm::launch_kv_append(view, rows, k, v, dtype == QM_F32 ? qm::KvType::kF32 : qm::KvType::kBF16,
                                          k_stride, v_stride, static_cast<cudaStream_t>(stream)));
}

int qm_kv_read_q4_0(const qm_kv_cache* cache, float* k, float* v, int64_t n_tokens, const int32_t* q_starts,
                    void* stream) {
    qm::KvView view;
    qm::KvRows rows;
    int64_t pool;
    int rc = check_cache(cache, &view, &pool);
    if (rc == QM_OK) rc = check_rows(cache, n_tokens, n_tokens, q_starts, &rows);
    if (rc != QM_OK) return rc;
    if (n_tokens == 0 || view.n_seqs == 0) return QM_OK;
    int64_t bytes;
    if (!mul_ok(n_tokens, int64_t(view.heads) * view.dim * 4, &bytes)) return QM_ERR_SHAPE;
    if (!k || !v) return QM_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16)) return QM_ERR_ALIGN;
    if (overlaps(k, bytes, v, bytes)) return QM_ERR_ALIAS;
    for (const float* p : {k, v})
        if (meets({p, bytes}, {{cache->k_pages, pool}, {cache->v_pages, pool}, table_of(cache), lengths_of(cache),
                               starts_of(cache, q_starts)}))
            return QM_ERR_ALIAS;
    qm::DeviceInfo dev;
    if (on_device(&dev, &view) != QM_OK) return QM_ERR_CUDA;
    rc = check_cache_pointers(cache, dev.device);
    if (rc == QM_OK) rc = check_pointer(k, dev.device);
    if (rc == QM_OK) rc = check_pointer(v, dev.device);
    if (rc == QM_OK && q_starts) rc = check_pointer(q_starts, dev.device);
    if (rc != QM_OK) return rc;
    return from_cuda(qm::launch_kv_read(view, rows, k, v, static_cast<cudaStream_t>(stream)));
}

int64_t qm_attn_workspace(const qm_kv_cache* cache, int64_t n_heads, int64_t n_tokens, int64_t max_q, int weights) {
    qm::KvView view;
    qm::KvRows rows;
    const int rc = check_workspace(cache, n_heads, n_tokens, max_q, &view, &rows);
    if (rc != QM_OK) return rc;
    return qm::attn_workspace_most(view, static_cast<int>(n_heads), rows.n_tokens, rows.max_q, weights != 0);
}

int64_t qm_attn_workspace_exact(const qm_kv_cache* cache, int64_t n_heads, int64_t n_tokens, int64_t max_q, int weights) {
    qm::KvView view;
    qm::KvRows rows;
    const int rc = check_workspace(cache, n_heads, n_tokens, max_q, &view, &rows);
    if (rc != QM_OK) return rc;
    return qm::attn_workspace_bytes(view, static_cast<int>(n_heads), rows.n_tokens, rows.max_q, weights != 0);
}

int qm_attn_q4_0(const qm_kv_cache* cache, const qm_attn_args* a, void* stream) {
    qm::KvView view;
    qm::KvRows rows;
    int64_t pool;
    int rc = check_cache(cache, &view, &pool);
    if (rc != QM_OK) return rc;
    if (!a) return QM_ERR_NULL;
    if (a->reserved || (a->dtype != QM_F32 && a->dtype != QM_BF16) || a->window < 0 || a->sinks < 0 ||
        !std::isfinite(a->scale))
        return QM_ERR_SHAPE;
    if ((rc = attn_sizes(cache, a->n_heads)) != QM_OK) return rc;
    if ((rc = check_rows(cache, a->n_tokens, a->max_q, a->q_starts, &rows)) != QM_OK) return rc;
    if (a->n_tokens * a->n_heads > 0x7FFFFFFF) return QM_ERR_SHAPE;  // rows and heads are numbered in an int
    const int64_t row = int64_t(a->n_heads) * view.dim, item = a->dtype == QM_F32 ? 4 : 2;
    int64_t qb, ob, lb, wb = 0;
    if ((rc = span(a->n_tokens, a->q_stride, row, item, &qb)) != QM_OK ||
        (rc = span(a->n_tokens, a->out_stride, row, item, &ob)) != QM_OK)
        return rc;
    lb = a->lse ? a->n_tokens * a->n_heads * 4 : 0;
    if (a->weights) {
        if (a->weights_stride < view.max_len || a->weights_stride < 0) return QM_ERR_SHAPE;
        if (!mul_ok(int64_t(view.n_seqs) * view.heads * 4, a->weights_stride, &wb)) return QM_ERR_SHAPE;
    }
    if (a->n_tokens == 0 || view.n_seqs == 0) return QM_OK;
    const int64_t need =
        qm::attn_workspace_bytes(view, static_cast<int>(a->n_heads), rows.n_tokens, rows.max_q, a->weights != nullptr);
    if (a->workspace_bytes < need) return QM_ERR_WORKSPACE;
    if (!a->q || !a->out || (need > 0 && !a->workspace)) return QM_ERR_NULL;
    if (!aligned(a->q, 4 * item) || !aligned(a->out, 4 * item) || !aligned(a->lse, 4) || !aligned(a->weights, 4) ||
        !aligned(a->workspace, 16))
        return QM_ERR_ALIGN;
    const Range outs[4] = {{a->out, ob}, {a->lse, lb}, {a->weights, wb}, {a->workspace, need}};
    for (int i = 0; i < 4; ++i) {
        if (meets(outs[i], {{a->q, qb}, {cache->k_pages, pool}, {cache->v_pages, pool}, table_of(cache), lengths_of(cache),
                            starts_of(cache, a->q_starts)}))
            return QM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], {outs[j]})) return QM_ERR_ALIAS;
    }
    qm::DeviceInfo dev;
    if (on_device(&dev, &view) != QM_OK) return QM_ERR_CUDA;
    rc = check_cache_pointers(cache, dev.device);
    const void* more[5] = {a->q, a->out, a->lse, a->weights, a->q_starts};
    for (const void* p : more)
        if (rc == QM_OK && p) rc = check_pointer(p, dev.device);
    if (rc == QM_OK && need > 0) rc = check_pointer(a->workspace, dev.device);
    if (rc != QM_OK) return rc;
    // A window as long as the cache hides nothing.
    const int window = a->window == 0 || a->window >= view.max_len ? 0 : static_cast<int>(a->window);
    qm::AttnCall call = {a->q, a->out, a->lse, a->weights, a->q_stride, a->out_stride, a->weights_stride,
                         static_cast<int>(a->n_heads), window,
                         static_cast<int>(a->sinks < view.max_len ? a->sinks : view.max_len), a->scale,
                         a->dtype == QM_F32 ? qm::KvType::kF32 : qm::KvType::kBF16,
                         static_cast<uint8_t*>(a->workspace)};
    return from_cuda(qm::launch_attn(view, rows, call, static_cast<cudaStream_t>(stream)));
}

int qm_kv_evict_q4_0(const qm_kv_cache* from, const qm_kv_cache* to, const float* weights, int64_t weights_stride,
                     int64_t budget, int64_t sinks, int64_t recent, int32_t* kept, float* weights_out,
                     int64_t out_stride, void* stream) {
    qm::KvView src, dst;
    int64_t src_pool, dst_pool;
    int rc = check_cache(from, &src, &src_pool);
    if (rc == QM_OK) rc = check_cache(to, &dst, &dst_pool);
    if (rc != QM_OK) return rc;
    if (src.n_seqs != dst.n_seqs || src.heads != dst.heads || src.dim != dst.dim) return QM_ERR_SHAPE;
    if (budget < 0 || budget > kMaxLen || sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
        return QM_ERR_SHAPE;
    const int64_t most = budget < src.max_len ? budget : src.max_len;  // tokens a sequence can keep
    if (dst.max_len < most) return QM_ERR_SHAPE;
    if (weights_stride < src.max_len || out_stride < budget) return QM_ERR_SHAPE;
    const int64_t lists = int64_t(src.n_seqs) * src.heads;
    int64_t wb, ob, kb;
    if (!mul_ok(lists * 4, weights_stride, &wb) || !mul_ok(lists * 4, out_stride, &ob) || !mul_ok(lists * 4, budget, &kb))
        return QM_ERR_SHAPE;
    if (src.n_seqs == 0) return QM_OK;
    if ((src.max_len > 0 && !weights) || (budget > 0 && (!kept || !weights_out))) return QM_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(kept, 4) || !aligned(weights_out, 4)) return QM_ERR_ALIGN;
    // In place: the same pages in the same order.  Otherwise the two caches
    // may share pools (on different pages), but then not half a cache.
    const bool in_place = src.k == dst.k && src.v == dst.v && src.table == dst.table;
    if (in_place && src.table && (src.page_shift != dst.page_shift || src.n_pages != dst.n_pages ||
                     src.table_stride != dst.table_stride))
        return QM_ERR_SHAPE;
    if (!in_place && (src.table == dst.table || overlaps(src.k, src_pool, dst.v, dst_pool) ||
                      overlaps(src.v, src_pool, dst.k, dst_pool)))
        return QM_ERR_ALIAS;
    if (weights_out != weights && overlaps(weights, wb, weights_out, ob)) return QM_ERR_ALIAS;
    if (weights && weights_out == weights && out_stride != weights_stride) return QM_ERR_ALIAS;
    if (overlaps(kept, kb, weights, wb) || overlaps(kept, kb, weights_out, ob)) return QM_ERR_ALIAS;
    // Two arrays of lengths that share some entries would change under the kernels that read them.
    if (from->lengths != to->lengths && meets(lengths_of(to), {lengths_of(from)})) return QM_ERR_ALIAS;
    // What is written (the pools, the lengths, the lists) shares nothing with what else is read or written.
    const Range ranks[3] = {{kept, kb}, {weights_out, ob}, {weights, wb}};
    for (const Range& x : ranks)
        if (meets(x, {{src.k, src_pool}, {src.v, src_pool}, {dst.k, dst_pool}, {dst.v, dst_pool}, lengths_of(to)}))
            return QM_ERR_ALIAS;
    for (int i = 0; i < 2; ++i)
        if (meets(ranks[i], {table_of(from), table_of(to), lengths_of(from)})) return QM_ERR_ALIAS;
    if (meets(lengths_of(to), {{src.k, src_pool}, {src.v, src_pool}, {dst.k, dst_pool}, {dst.v, dst_pool}, table_of(from),
                               table_of(to)}))
        return QM_ERR_ALIAS;
    for (const void* p : {dst.k, dst.v})
        if (meets({p, dst_pool}, {table_of(from), table_of(to), lengths_of(from)})) return QM_ERR_ALIAS;
    qm::DeviceInfo dev;
    if (on_device(&dev, &src) != QM_OK) return QM_ERR_CUDA;
    rc = check_cache_pointers(from, dev.device);
    if (rc == QM_OK) rc = check_cache_pointers(to, dev.device);
    const void* more[3] = {weights, kept, weights_out};
    for (const void* p : more)
        if (rc == QM_OK && p) rc = check_pointer(p, dev.device);
    if (rc != QM_OK) return rc;
    const qm::EvictCall e = {weights, weights_out, kept, to->lengths, weights_stride, out_stride,
                             static_cast<int>(budget), static_cast<int>(sinks), static_cast<int>(recent)};
    return from_cuda(qm::launch_kv_evict(src, dst, e, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
