// The feed-forward block of a decoder with experts (qm_experts_q4_0): the pairs of
// tokens and experts in the experts' order, the products, and their weighted sum.
#include <cuda_bf16.h>

#include "qm_device.cuh"

namespace qm {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// Where the parts of the workspace are.
struct Parts {
    int64_t starts, order, inner, part, bytes;
};
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
Parts layout(const ExpertsView& e, int64_t n_tokens, int64_t top_k) {
    const int64_t pairs = n_tokens * top_k;
    Parts p;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t a = at;
        at += up256(bytes);
        return a;
    };
    p.starts = take((e.n + 1) * 4);
    p.order = take(pairs * 4);
    p.inner = take(pairs * e.inner * 4);
    p.part = take(pairs * e.hidden * 4);
    p.bytes = at;
    return p;
}

// The pairs of expert blockIdx.x in ascending order, order[starts[e] ..
// starts[e + 1]), by one CTA that goes over all ids: it counts those of lower
// experts too, so that no CTA waits for another.  Every thread has a range of
// consecutive ids.
__global__ void __launch_bounds__(1024) experts_order(const int32_t* ids, int pairs, int n, int32_t* starts, int32_t* order,
                                                      unsigned int* err) {
    __shared__ int sums[2][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int e = blockIdx.x;
    const int each = (pairs + blockDim.x - 1) / blockDim.x;
    const int lo = min(pairs, static_cast<int>(threadIdx.x) * each), hi = min(pairs, lo + each);
    int below = 0, mine = 0;
    bool range = false;
    for (int i = lo; i < hi; ++i) {
        const int id = ids[i];
        below += id >= 0 && id < e;
        mine += id == e;
        range |= id >= n;
    }
    if (range && e == 0) atomicOr(err, kErrRange);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = mine;  // of this warp's lanes up to this one
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    below = __reduce_add_sync(kAll, below);
    if (lane == 31) sums[0][warp] = upto;
    if (lane == 0) sums[1][warp] = below;
    __syncthreads();
    const int before_all = __reduce_add_sync(kAll, sums[1][lane]);
    const int before = __reduce_add_sync(kAll, lane < warp ? sums[0][lane] : 0);
    int at = before_all + before + upto - mine;
    if (mine)
        for (int i = lo; i < hi; ++i)
            if (ids[i] == e) order[at++] = i;
    if (threadIdx.x == 0) starts[e] = before_all;
    if (threadIdx.x == blockDim.x - 1 && e == n - 1) starts[n] = before_all + before + upto;
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float activate(float a, int kind) {
    if (kind == 1) return a / (1.f + expf(-a));
    if (kind == 2) return 0.5f * a * (1.f + tanhf(0.7978845608028654f * (a + 0.044715f * a * a * a)));
    return a;
}

// A warp's dot product of a row of K / 32 blocks with K values.
template <typename T>
__device__ __forceinline__ float row_dot(const uint8_t* blocks, const T* x, int K, int lane) {
    float s = 0.f;
    for (int b = 0; b < K / 32; ++b) {
        const uint8_t* blk = blocks + 18 * b;
        const float d = f16_bits_to_float(*reinterpret_cast<const uint16_t*>(blk));
        const uint32_t byte = blk[2 + (lane & 15)];
        const int q = static_cast<int>(lane < 16 ? byte & 15u : byte >> 4) - 8;
        s = fmaf(load1(x + 32 * b + lane), static_cast<float>(q) * d, s);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kAll, s, d);
    return s;
}

__device__ __forceinline__ int expert_of(const int32_t* starts, int n, int p) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid + 1] <= p) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// inner[p][i] = act(gate) * up of sorted pair p = blockIdx.y; a warp per i.
template <typename T>
__global__ void __launch_bounds__(256) experts_up_rows(const ExpertsView e, const ExpertsCall c, const int32_t* starts,
                                                       const int32_t* order, float* inner) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, p = blockIdx.x;
    if (p >= starts[e.n]) return;
    const int ex = expert_of(starts, e.n, p);
    const T* x = static_cast<const T*>(c.x) + static_cast<int64_t>(order[p] / c.top_k) * c.x_stride;
    const int64_t row_bytes = e.hidden / 32 * 18;
    for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < e.inner; i += gridDim.y * 8) {
        const float u = row_dot(e.up + ex * e.up_stride + i * row_bytes, x, e.hidden, lane);
        float h;
        if (e.gate) h = activate(row_dot(e.gate + ex * e.gate_stride + i * row_bytes, x, e.hidden, lane), e.activation) * u;
        else h = activate(u, e.activation);
        if (lane == 0) inner[static_cast<int64_t>(p) * e.inner + i] = h;
    }
}

// part[pair][i], the pair's place among all pairs.
__global__ void __launch_bounds__(256) experts_down_rows(const ExpertsView e, const int32_t* starts, const int32_t* order,
                                                         const float* inner, float* part) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, p = blockIdx.x;
    if (p >= starts[e.n]) return;
    const int ex = expert_of(starts, e.n, p);
    const int64_t row_bytes = e.inner / 32 * 18;
    for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < e.hidden; i += gridDim.y * 8) {
        const float y = row_dot(e.down + ex * e.down_stride + i * row_bytes, inner + static_cast<int64_t>(p) * e.inner,
                                e.inner, lane);
        if (lane == 0) part[static_cast<int64_t>(order[p]) * e.hidden + i] = y;
    }
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// out[t] = the weighted sum of the token's pairs, in their order.
template <typename T>
__global__ void __launch_bounds__(128) experts_combine(const ExpertsCall c, int hidden, int n, const float* part) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int at = (blockIdx.x * 128 + threadIdx.x) * 4;
    if (at >= hidden) return;
    for (int t = blockIdx.y; t < c.n_tokens; t += gridDim.y) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < c.top_k; ++j) {
            const int64_t pair = static_cast<int64_t>(t) * c.top_k + j;
            const int id = c.ids[pair];
            if (id < 0 || id >= n) continue;
            const float w = c.weights[pair];
            const float4 y = *reinterpret_cast<const float4*>(part + pair * hidden + at);
            s.x = fmaf(w, y.x, s.x), s.y = fmaf(w, y.y, s.y), s.z = fmaf(w, y.z, s.z), s.w = fmaf(w, y.w, s.w);
        }
        store4(static_cast<T*>(c.out) + t * c.out_stride + at, s);
    }
}

template <typename T>
cudaError_t launch_type(const ExpertsView& e, const ExpertsCall& c, cudaStream_t stream) {
    const Parts at = layout(e, c.n_tokens, c.top_k);
    const int pairs = c.n_tokens * c.top_k;
    int32_t* starts = reinterpret_cast<int32_t*>(c.ws + at.starts);
    int32_t* order = reinterpret_cast<int32_t*>(c.ws + at.order);
    float* inner = reinterpret_cast<float*>(c.ws + at.inner);
    float* part = reinterpret_cast<float*>(c.ws + at.part);
    cudaError_t err = launch_pdl(experts_order, dim3(e.n), dim3(1024), 0, stream, c.ids, pairs, e.n, starts, order, c.err);
    if (err == cudaSuccess) {
        note_launch();
        err = launch_pdl(experts_up_rows<T>, dim3(pairs, 16), dim3(256), 0, stream, e, c, starts, order, inner);
    }
    if (err == cudaSuccess) {
        note_launch();
        err = launch_pdl(experts_down_rows, dim3(pairs, 16), dim3(256), 0, stream, e, starts, order, inner, part);
    }
    if (err == cudaSuccess) {
        note_launch();
        err = launch_pdl(experts_combine<T>, dim3((e.hidden + 511) / 512, c.n_tokens < 4096 ? c.n_tokens : 4096), dim3(128), 0,
                         stream, c, e.hidden, e.n, part);
    }
    if (err == cudaSuccess) note_launch();
    return err;
}

}  // namespace

int64_t experts_workspace(const ExpertsView& e, int64_t n_tokens, int64_t top_k) { return layout(e, n_tokens, top_k).bytes; }

cudaError_t launch_experts(const ExpertsView& e, const ExpertsCall& c, const DeviceInfo&, cudaStream_t stream) {
    return c.type == KvType::kF32 ? launch_type<float>(e, c, stream) : launch_type<__nv_bfloat16>(e, c, stream);
}

}  // namespace qm
