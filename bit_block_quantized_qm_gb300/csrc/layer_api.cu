// The C ABI of a layer's norm, routing and experts (declared in include/qm.h):
// argument checks, then launches on the caller's stream.
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

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    const void* p;
    int64_t n;
};
bool meets(const Range& a, std::initializer_list<Range> others) {
    for (const Range& b : others)
        if (a.p && b.p && overlaps(a.p, a.n, b.p, b.n)) return true;
    return false;
}

// Bytes from the first element of n rows of `row` elements, `stride` apart, to the last.
int span(int64_t n, int64_t stride, int64_t row, int64_t item, int64_t* bytes) {
    if (n > 1 && stride < row) return QM_ERR_SHAPE;
    int64_t e;
    if (!mul_ok(n > 1 ? n - 1 : 0, n > 1 ? stride : 0, &e) || e > INT64_MAX / 8 - row) return QM_ERR_SHAPE;
    *bytes = n > 0 ? (e + row) * item : 0;
    return QM_OK;
}

bool known_type(int dtype) { return dtype == QM_F32 || dtype == QM_BF16; }
int item_of(int dtype) { return dtype == QM_F32 ? 4 : 2; }
qm::KvType type_of(int dtype) { return dtype == QM_F32 ? qm::KvType::kF32 : qm::KvType::kBF16; }

int check_pointers(int device, std::initializer_list<const void*> pointers) {
    for (const void* p : pointers) {
        const int rc = p ? check_pointer(p, device) : QM_OK;
        if (rc != QM_OK) return rc;
    }
    return QM_OK;
}

// Sizes, alignments and pointers of the experts; the bytes of each matrix tensor.
int check_experts(const qm_experts* e, qm::ExpertsView* view, int64_t bytes[3]) {
    if (!e) return QM_ERR_NULL;
    for (int64_t n : {e->hidden, e->inner})
        if (n < 32 || n > 65536 || n % 32) return QM_ERR_SHAPE;
    if (e->n_experts < 1 || e->n_experts > 1024 || e->activation < QM_ACT_NONE || e->activation > QM_ACT_GELU ||
        e->reserved[0] || e->reserved[1])
        return QM_ERR_SHAPE;
    if (!e->w_up || !e->w_down) return QM_ERR_NULL;
    const int64_t matrix = e->hidden * e->inner / 32 * 18;
    const int64_t strides[3] = {e->w_gate ? e->gate_stride : matrix, e->up_stride, e->down_stride};
    for (int i = 0; i < 3; ++i) {
        if (e->n_experts > 1 && (strides[i] < matrix || strides[i] % 16 || strides[i] >= int64_t(1) << 40))
            return QM_ERR_SHAPE;
        if (!mul_ok(e->n_experts - 1, e->n_experts > 1 ? strides[i] : 0, &bytes[i]) || bytes[i] > INT64_MAX / 2)
            return QM_ERR_SHAPE;
        bytes[i] += matrix;
    }
    if (!e->w_gate) bytes[0] = 0;
    if (!aligned(e->w_gate, 16) || !aligned(e->w_up, 16) || !aligned(e->w_down, 16)) return QM_ERR_ALIGN;
    const bool one = e->n_experts == 1;  // (whose strides do not matter)
    *view = {static_cast<const uint8_t*>(e->w_gate), static_cast<const uint8_t*>(e->w_up),
             static_cast<const uint8_t*>(e->w_down), one ? matrix : e->gate_stride, one ? matrix : e->up_stride,
             one ? matrix : e->down_stride, static_cast<int>(e->hidden), static_cast<int>(e->inner), e->n_experts,
             e->activation};
    return QM_OK;
}

int check_pairs(int64_t n_tokens, int32_t top_k) {
    if (n_tokens < 0 || top_k < 1 || top_k > 1024 || n_tokens >= (int64_t(1) << 24) ||
        n_tokens * top_k >= (int64_t(1) << 24))
        return QM_ERR_SHAPE;
    return QM_OK;
}

}  // namespace

extern "C" {

int qm_add_rmsnorm(const qm_rmsnorm_args* a, void* stream) {
    if (!a) return QM_ERR_NULL;
    if (a->reserved || !known_type(a->dtype) || a->n_rows < 0 || a->n_rows > 0x7FFFFFFF || a->width < 1 ||
        a->width > (1 << 20) || !(a->eps >= 0.f) || !std::isfinite(a->eps) || !std::isfinite(a->weight_offset) ||
        (a->q8 && a->width % 32))
        return QM_ERR_SHAPE;
    const int64_t item = item_of(a->dtype);
    int64_t xb, rb = 0, ob = 0, sb = 0;
    int rc = span(a->n_rows, a->x_stride, a->width, item, &xb);
    if (rc == QM_OK && a->residual) rc = span(a->n_rows, a->residual_stride, a->width, item, &rb);
    if (rc == QM_OK && a->out) rc = span(a->n_rows, a->out_stride, a->width, item, &ob);
    if (rc == QM_OK && a->sum) rc = span(a->n_rows, a->sum_stride, a->width, item, &sb);
    if (rc != QM_OK) return rc;
    const int64_t qb = a->q8 ? a->n_rows * (a->width / 32 * 34) : 0, wb = a->width * 4;
    if (a->n_rows == 0 || (!a->out && !a->sum && !a->q8)) return QM_OK;
    if (!a->x) return QM_ERR_NULL;
    if (!aligned(a->x, item) || !aligned(a->residual, item) || !aligned(a->out, item) || !aligned(a->sum, item) ||
        !aligned(a->weight, 4) || !aligned(a->q8, 2))
        return QM_ERR_ALIGN;
    const Range x = {a->x, xb}, res = {a->residual, rb}, w = {a->weight, wb}, out = {a->out, ob}, sum = {a->sum, sb},
                q8 = {a->q8, qb};
    if (meets(out, {x, res, w, sum, q8}) || meets(q8, {x, res, w, sum}) || meets(sum, {w})) return QM_ERR_ALIAS;
    // The sum may take the place of what it is the sum of, row by row.
    const bool one = a->n_rows == 1;
    if (meets(sum, {x}) && (a->sum != a->x || (!one && a->sum_stride != a->x_stride))) return QM_ERR_ALIAS;
    if (meets(sum, {res}) && (a->sum != a->residual || (!one && a->sum_stride != a->residual_stride))) return QM_ERR_ALIAS;
    qm::DeviceInfo dev;
    if (qm::current_device_info(&dev) != cudaSuccess) return QM_ERR_CUDA;
    rc = check_pointers(dev.device, {a->x, a->residual, a->weight, a->out, a->sum, a->q8});
    if (rc != QM_OK) return rc;
    const qm::NormCall call = {a->x, a->residual, a->weight, a->out, a->sum, static_cast<uint8_t*>(a->q8), a->n_rows,
                               a->x_stride, a->residual_stride, a->out_stride, a->sum_stride, static_cast<int>(a->width),
                               a->eps, a->weight_offset, type_of(a->dtype)};
    return from_cuda(qm::launch_add_rmsnorm(call, dev, static_cast<cudaStream_t>(stream)));
}

int qm_route_experts(const qm_route_args* a, void* stream) {
    if (!a) return QM_ERR_NULL;
    if (a->reserved || !known_type(a->dtype) || a->n_tokens < 0 || a->n_tokens > 0x7FFFFFFF || a->n_experts < 1 ||
        a->n_experts > 1024 || a->n_groups < 1 || a->n_groups > 64 || a->n_experts % a->n_groups || a->top_groups < 1 ||
        a->top_groups > a->n_groups || a->group_top < 1 || a->group_top > 2 || a->top_k < 1 || a->top_k > 32 ||
        a->top_k > a->n_experts / a->n_groups * a->top_groups || a->scoring < QM_SCORE_SOFTMAX ||
        a->scoring > QM_SCORE_SIGMOID || a->renormalize < 0 || a->renormalize > 1 || !std::isfinite(a->scale))
        return QM_ERR_SHAPE;
    const int64_t item = item_of(a->dtype);
    int64_t lb;
    int rc = span(a->n_tokens, a->logits_stride, a->n_experts, item, &lb);
    if (rc != QM_OK) return rc;
    if (a->n_tokens == 0) return QM_OK;
    if (!a->logits || !a->ids || !a->weights) return QM_ERR_NULL;
    if (!aligned(a->logits, item) || !aligned(a->bias, 4) || !aligned(a->ids, 4) || !aligned(a->weights, 4))
        return QM_ERR_ALIGN;
    const int64_t kb = a->n_tokens * a->top_k * 4;
    const Range logits = {a->logits, lb}, bias = {a->bias, int64_t(a->n_experts) * 4}, ids = {a->ids, kb},
                weights = {a->weights, kb};
    if (meets(ids, {logits, bias, weights}) || meets(weights, {logits, bias})) return QM_ERR_ALIAS;
    qm::DeviceInfo dev;
    if (qm::current_device_info(&dev) != cudaSuccess) return QM_ERR_CUDA;
    rc = check_pointers(dev.device, {a->logits, a->bias, a->ids, a->weights});
    if (rc != QM_OK) return rc;
    const qm::RouteCall call = {a->logits, a->bias, a->ids, a->weights, a->n_tokens, a->logits_stride, a->n_experts,
                                a->top_k, a->n_groups, a->top_groups, a->group_top, a->scoring == QM_SCORE_SIGMOID,
                                a->renormalize != 0, a->scale, type_of(a->dtype)};
    return from_cuda(qm::launch_route_experts(call, static_cast<cudaStream_t>(stream)));
}

int64_t qm_experts_workspace(const qm_experts* experts, int64_t n_tokens, int32_t top_k) {
    qm::ExpertsView view;
    int64_t bytes[3];
    int rc = check_experts(experts, &view, bytes);
    if (rc == QM_OK) rc = check_pairs(n_tokens, top_k);
    return rc != QM_OK ? rc : n_tokens == 0 ? 0 : qm::experts_workspace(view, n_tokens, top_k);
}

int qm_experts_q4_0(const qm_experts* experts, const qm_experts_args* a, void* stream) {
    qm::ExpertsView view;
    int64_t wb[3];
    int rc = check_experts(experts, &view, wb);
    if (rc != QM_OK) return rc;
    if (!a) return QM_ERR_NULL;
    if (a->reserved[0] || a->reserved[1] || !known_type(a->dtype)) return QM_ERR_SHAPE;
    if ((rc = check_pairs(a->n_tokens, a->top_k)) != QM_OK) return rc;
    const int64_t item = item_of(a->dtype), kb = a->n_tokens * a->top_k * 4;
    int64_t xb, ob;
    if ((a->n_tokens > 1 && (a->x_stride % 4 || a->out_stride % 4)) ||
        (rc = span(a->n_tokens, a->x_stride, view.hidden, item, &xb)) != QM_OK ||
        (rc = span(a->n_tokens, a->out_stride, view.hidden, item, &ob)) != QM_OK)
        return QM_ERR_SHAPE;
    if (a->n_tokens == 0) return QM_OK;
    const int64_t need = qm::experts_workspace(view, a->n_tokens, a->top_k);
    if (a->workspace_bytes < need) return QM_ERR_WORKSPACE;
    if (!a->x || !a->out || !a->ids || !a->weights || !a->workspace) return QM_ERR_NULL;
    if (!aligned(a->x, 4 * item) || !aligned(a->out, 4 * item) || !aligned(a->ids, 4) || !aligned(a->weights, 4) ||
        !aligned(a->workspace, 16))
        return QM_ERR_ALIGN;
    const Range out = {a->out, ob}, ws = {a->workspace, need};
    const Range ins[6] = {{a->x, xb}, {a->ids, kb}, {a->weights, kb}, {view.gate, wb[0]}, {view.up, wb[1]}, {view.down, wb[2]}};
    for (const Range& in : ins)
        if (meets(in, {out, ws})) return QM_ERR_ALIAS;
    if (meets(out, {ws})) return QM_ERR_ALIAS;
    qm::DeviceInfo dev;
    if (qm::current_device_info(&dev) != cudaSuccess) return QM_ERR_CUDA;
    rc = check_pointers(dev.device, {a->x, a->out, a->ids, a->weights, a->workspace, view.gate, view.up, view.down});
    if (rc != QM_OK) return rc;
    qm::ExpertsCall call = {a->x, a->out, a->ids, a->weights, static_cast<uint8_t*>(a->workspace), a->x_stride,
                            a->out_stride, static_cast<int>(a->n_tokens), a->top_k, type_of(a->dtype), nullptr};
    if (qm::kv_error_word(dev.device, &call.err) != cudaSuccess) return QM_ERR_CUDA;
    return from_cuda(qm::launch_experts(view, call, dev, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
