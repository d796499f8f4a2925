// The norm that adds the residual (qm_add_rmsnorm).
//
// Bound: memory, each input read once and each output written once (8192 rows of 4096
// bf16 with a residual and both outputs, 268 MB: 42 us, 6.4 TB/s; f32: 80 us, 6.7 TB/s);
// few rows: the latency of one load, one reduction over the CTA and one store (600 rows:
// 4 us).  A row belongs to one CTA, whose threads keep their 8 (or 16, 32) elements of it
// in registers between the sum of squares and the outputs (but for 19 words of a thread with 32 f32 elements,
// beside its weights and the next row's; those come back from L1).  Statistics and products are f32;
// outputs are rounded once.  The row's Q8_0 blocks are made from the f32 values by
// four lanes a block, as quantize_q8_0 does.
#include <cuda_bf16.h>

#include "qm_device.cuh"

namespace qm {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void load8(const float* p, float v[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// 8 elements as they are loaded.
struct F32x8 {
    float4 a, b;
};
template <typename T>
struct RawOf {
    using type = F32x8;
};
template <>
struct RawOf<__nv_bfloat16> {
    using type = uint4;
};
__device__ __forceinline__ void unpack8(const F32x8& r, float v[8]) {
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w, v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void unpack8(const uint4& w, float v[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float v[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float v[8]) {
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
}

// Sum over the CTA, on every thread; `part` has a word per warp.
__device__ __forceinline__ float cta_sum(float v, float* part) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < static_cast<unsigned>(warps) ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

__device__ __forceinline__ float row_factor(const NormCall& c, float squares) {
    return 1.f / sqrtf(squares / static_cast<float>(c.width) + c.eps);
}

// 8 elements of a row, those of lanes 4 b .. 4 b + 3 a block: its Q8_0 bytes.  All
// lanes of the warp take part; `in`: this thread's elements exist.
__device__ __forceinline__ void store_q8(uint8_t* row, int at, const float v[8], bool in) {
    float amax = 0.f;
    if (in)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
    amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
    if (!in) return;
    const float d = __fdiv_rn(amax, 127.f), r = __frcp_rn(d);
    uint8_t* block = row + at / 32 * 34;
    if (at % 32 == 0) *reinterpret_cast<uint16_t*>(block) = static_cast<uint16_t>(f16_bits_rn(d));
    uint16_t* q = reinterpret_cast<uint16_t*>(block + 2 + at % 32);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        q[e] = static_cast<uint16_t>(q8_quant_byte(v[2 * e], d, r) | q8_quant_byte(v[2 * e + 1], d, r) << 8);
}

// Rows of up to 8 * VEC elements a thread, 16-byte aligned.  A CTA takes every gridDim.x-th
// row: it keeps the weights, and asks for the next row's elements before it waits for the sum
// over the one at hand.
template <int VEC, typename T>
__global__ void __launch_bounds__(512) rmsnorm_rows(const NormCall c) {
    __shared__ float part[2][32];
    grid_launch_dependents();
    const int stride = blockDim.x * 8;
    float w[VEC][8], v[VEC][8];
    using Raw = typename RawOf<T>::type;
    Raw x_raw[VEC], r_raw[VEC];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int at = i * stride + threadIdx.x * 8;
            if (at >= c.width) continue;
            x_raw[i] = *reinterpret_cast<const Raw*>(static_cast<const T*>(c.x) + r * c.x_stride + at);
            if (c.residual) r_raw[i] = *reinterpret_cast<const Raw*>(static_cast<const T*>(c.residual) + r * c.residual_stride + at);
        }
    };
    grid_dependency_wait();
    fetch(blockIdx.x);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int at = i * stride + threadIdx.x * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
        if (!c.weight || at >= c.width) continue;
        load8(c.weight + at, w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] += c.weight_offset;
    }
    int buf = 0;
#pragma unroll 1
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x, buf ^= 1) {
        float squares = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if (i * stride + static_cast<int>(threadIdx.x) * 8 >= c.width) continue;
            unpack8(x_raw[i], v[i]);
            if (c.residual) {
                float y[8];
                unpack8(r_raw[i], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] += y[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) squares = fmaf(v[i][e], v[i][e], squares);
        }
        if (r + gridDim.x < c.rows) fetch(r + gridDim.x);
        if (c.sum) {
            T* sum = static_cast<T*>(c.sum) + r * c.sum_stride;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int at = i * stride + threadIdx.x * 8;
                if (at < c.width) store8(sum + at, v[i]);
            }
        }
        const float f = row_factor(c, cta_sum(squares, part[buf]));
        T* out = static_cast<T*>(c.out) + r * c.out_stride;
        uint8_t* q8 = c.q8 + r * (c.width / 32 * 34);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int at = i * stride + threadIdx.x * 8;
            const bool in = at < c.width;
            if (in) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * f * w[i][e];
                if (c.out) store8(out + at, v[i]);
            }
            if (c.q8) store_q8(q8, at, v[i], in);
        }
    }
}

// Rows of up to E * 1024 elements of any width and alignment, element by element: a CTA each, a warp for
// 32 E elements next to each other (4096 bf16 rows of 4097 with a residual: 45 us against 57 when they are
// read twice; of 16383: 191 against 202, f32 244 against 312).
template <int E, typename T>
__global__ void __launch_bounds__(1024) rmsnorm_held(const NormCall c) {
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(c.x) + r * c.x_stride;
    const int first = (threadIdx.x >> 5) * (32 * E) + (threadIdx.x & 31);
    float v[E], w[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int at = first + 32 * i;
        v[i] = at < c.width ? load1(x + at) : 0.f;
    }
    if (c.residual) {
        const T* res = static_cast<const T*>(c.residual) + r * c.residual_stride;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int at = first + 32 * i;
            if (at < c.width) v[i] += load1(res + at);
        }
    }
    float squares = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int at = first + 32 * i;
        squares = fmaf(v[i], v[i], squares);
        w[i] = c.weight && at < c.width ? c.weight_offset + c.weight[at] : 1.f;
    }
    if (c.sum) {
        T* sum = static_cast<T*>(c.sum) + r * c.sum_stride;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int at = first + 32 * i;
            if (at < c.width) store1(sum + at, v[i]);
        }
    }
    const float f = row_factor(c, cta_sum(squares, part));
    if (!c.out) return;
    T* out = static_cast<T*>(c.out) + r * c.out_stride;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int at = first + 32 * i;
        if (at < c.width) store1(out + at, v[i] * f * w[i]);
    }
}

// Rows of any width and alignment: read twice.  An element is read and written by one
// thread, after its last read, so `sum` may be x or the residual.
template <typename T>
__global__ void __launch_bounds__(512) rmsnorm_any(const NormCall c) {
    __shared__ float part[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(c.x) + r * c.x_stride;
    const T* res = static_cast<const T*>(c.residual) + r * c.residual_stride;
    auto s_at = [&](int at) { return c.residual ? load1(x + at) + load1(res + at) : load1(x + at); };
    float squares = 0.f;
    for (int at = threadIdx.x; at < c.width; at += blockDim.x) {
        const float s = s_at(at);
        squares = fmaf(s, s, squares);
    }
    const float f = row_factor(c, cta_sum(squares, part));
    T* out = static_cast<T*>(c.out) + r * c.out_stride;
    T* sum = static_cast<T*>(c.sum) + r * c.sum_stride;
    uint8_t* q8 = c.q8 + r * (c.width / 32 * 34);
    // (With q8 the width is a multiple of 32: a warp's elements are one block or none.)
    for (int at = threadIdx.x; at < c.width; at += blockDim.x) {
        const float s = s_at(at);
        const float y = s * f * (c.weight ? c.weight_offset + c.weight[at] : 1.f);
        if (c.sum) store1(sum + at, s);
        if (c.out) store1(out + at, y);
        if (c.q8) {
            float amax = fabsf(y);
            if (isnan(amax)) amax = 0.f;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, d));
            const float d = __fdiv_rn(amax, 127.f);
            uint8_t* block = q8 + at / 32 * 34;
            const uint32_t q = q8_quant_byte(y, d, __frcp_rn(d)), q_next = __shfl_down_sync(kAll, q, 1);
            if ((at & 1) == 0) *reinterpret_cast<uint16_t*>(block + 2 + at % 32) = static_cast<uint16_t>(q | q_next << 8);
            if (at % 32 == 0) *reinterpret_cast<uint16_t*>(block) = static_cast<uint16_t>(f16_bits_rn(d));
        }
    }
}

template <typename T>
cudaError_t launch_type(const NormCall& c, const DeviceInfo& dev, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(c.rows));
    auto fits = [](const void* p, int64_t stride) {
        return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * sizeof(T)) % 16 == 0;
    };
    const bool one = c.rows == 1;  // (whose strides do not matter)
    const bool fast = c.width % 8 == 0 && c.width <= 512 * 32 && fits(c.x, one ? 0 : c.x_stride) &&
                      (!c.residual || fits(c.residual, one ? 0 : c.residual_stride)) &&
                      (!c.out || fits(c.out, one ? 0 : c.out_stride)) && (!c.sum || fits(c.sum, one ? 0 : c.sum_stride)) &&
                      fits(c.weight, 0);
    note_launch();
    if (!fast && !c.q8 && c.width <= 16 * 1024) {
        const int e = c.width <= 8 * 1024 ? 8 : 16;
        const dim3 block((c.width + 32 * e - 1) / (32 * e) * 32);
        return e == 8 ? launch_pdl(rmsnorm_held<8, T>, grid, block, 0, stream, c)
                      : launch_pdl(rmsnorm_held<16, T>, grid, block, 0, stream, c);
    }
    if (!fast) return launch_pdl(rmsnorm_any<T>, grid, dim3(512), 0, stream, c);
    // Few rows: many threads each, for the latency.  Many rows: fewer threads with more loads on their
    // way (8192 bf16 rows of 4096: 42 us against 49 with 512 threads), and as many CTAs as the SMs hold
    // at once, which keep the weights (42 against 46 with a CTA a row; 60000 rows of 128: 17 against 61).
    // f32 rows of 64 threads or more are better off with a CTA each, whose weights are the smaller part
    // (8192 rows of 4096: 80 us against 85; 40000 of 512: 52 against 55; 60000 of 128: 61 against 23).
    const int most = c.rows <= 2 * dev.sm_count ? 512 : 128;
    const int vec = c.width <= most * 8 ? 1 : c.width <= most * 16 ? 2 : 4;
    const int threads = (c.width + vec * 256 - 1) / (vec * 256) * 32;
    const int64_t resident = sizeof(T) == 4 && threads >= 64
                                 ? c.rows
                                 : static_cast<int64_t>(dev.sm_count) * (1536 / (threads < 64 ? 64 : threads));
    const dim3 block(threads), rows(static_cast<unsigned>(c.rows < resident ? c.rows : resident));
    if (vec == 1) return launch_pdl(rmsnorm_rows<1, T>, rows, block, 0, stream, c);
    if (vec == 2) return launch_pdl(rmsnorm_rows<2, T>, rows, block, 0, stream, c);
    return launch_pdl(rmsnorm_rows<4, T>, rows, block, 0, stream, c);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormCall& c, const DeviceInfo& dev, cudaStream_t stream) {
    return c.type == KvType::kF32 ? launch_type<float>(c, dev, stream) : launch_type<__nv_bfloat16>(c, dev, stream);
}

}  // namespace qm
