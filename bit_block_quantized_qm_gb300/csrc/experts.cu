// The feed-forward block of a decoder with experts (qm_experts_q4_0): the pairs of
// tokens and experts in the experts' order, the products, and their weighted sum.
#include <type_traits>

#include "experts.cuh"
#include "tcgen05.cuh"

namespace qm {

namespace {

constexpr int kCounters = 16 * kExpertCtas;  // of shared tiles (and their warps), for each of the two products
constexpr int kSetupThreads = 512;

// Where the parts of the workspace are.
struct Parts {
    int64_t starts, order, place, counters, x_pieces, x_unit, inner, i_pieces, i_unit, part, split, bytes;
    int split_cols;
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
    p.split_cols = static_cast<int>(pairs < kExpertTokens ? (pairs + 15) / 16 * 16 : kExpertTokens);
    p.starts = take((e.n + 1) * 4);
    p.order = take(pairs * 4);
    p.place = take(pairs * 4);
    p.counters = take(2 * kCounters * 4);
    p.x_pieces = take(pairs * piece_pitch(e.hidden) * 4);
    p.x_unit = take(pairs * 4);
    p.inner = take(pairs * e.inner * 4);
    p.i_pieces = take(pairs * piece_pitch(e.inner) * 4);
    p.i_unit = take(pairs * 4);
    p.part = take(pairs * e.hidden * 4);
    p.split = take(int64_t(2 * kExpertCtas) * 256 * p.split_cols * 4);
    p.bytes = at;
    return p;
}

// How many of the pairs 0 .. pairs - 1 have experts below e, and how many e in the ranges of
// the warps before this one: every warp goes over a range of consecutive ids, 32 at a time.
struct Ranks {
    int lo, hi;      // this warp's range
    int below, all;  // pairs of lower experts; pairs of e
    int before;      // pairs of e in lower warps' ranges
    bool range;      // an id of its lane's is no expert's
};
__device__ __forceinline__ Ranks rank_pairs(int e, const int32_t* ids, int pairs, int n) {
    constexpr int kWarps = kSetupThreads / 32;
    __shared__ int sums[2][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Ranks r;
    const int each = (pairs + kSetupThreads - 1) / kSetupThreads * 32;
    r.lo = min(pairs, warp * each), r.hi = min(pairs, r.lo + each);
    int below = 0, mine = 0;
    r.range = false;
#pragma unroll 8
    for (int i = r.lo + lane; i < r.hi; i += 32) {
        const int id = ids[i];
        below += id >= 0 && id < e;
        mine += id == e;
        r.range |= id >= n;
    }
    below = __reduce_add_sync(kAll, below);
    mine = __reduce_add_sync(kAll, mine);
    if (lane == 0) sums[0][warp] = mine, sums[1][warp] = below;
    __syncthreads();
    const int m = lane < kWarps ? sums[0][lane] : 0;
    r.below = __reduce_add_sync(kAll, lane < kWarps ? sums[1][lane] : 0);
    r.all = __reduce_add_sync(kAll, m);
    r.before = __reduce_add_sync(kAll, lane < warp ? m : 0);
    return r;
}

// The pairs of expert e in ascending order, order[starts[e] .. starts[e + 1]), and the place of
// each of them there (-1 of a pair without an expert), by one CTA that goes over all ids: it
// counts those of lower experts too, so that no CTA waits for another.
__device__ __forceinline__ void order_pairs(int e, const int32_t* ids, int pairs, int n, int32_t* starts, int32_t* order,
                                            int32_t* place, unsigned int* err) {
    const Ranks r = rank_pairs(e, ids, pairs, n);
    if (r.range && e == 0) atomicOr(err, kErrRange);
    const int lane = threadIdx.x & 31;
    int at = r.below + r.before;
#pragma unroll 4
    for (int i0 = r.lo; i0 < r.hi; i0 += 32) {
        const int i = i0 + lane, id = i < r.hi ? ids[i] : -2;
        const unsigned here = __ballot_sync(kAll, id == e);
        if (id == e) {
            const int p = at + __popc(here & ((1u << lane) - 1u));
            order[p] = i;
            place[i] = p;
        } else if (e == 0 && i < r.hi && (id < 0 || id >= n)) {
            place[i] = -1;
        }
        at += __popc(here);
    }
    if (threadIdx.x == 0) starts[e] = r.below;
    if (threadIdx.x == 0 && e == n - 1) starts[n] = r.below + r.all;
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The sum of a row of weights with a row of numbers, element by element: for sums that
// came out infinite or NaN.
template <typename T>
__device__ __noinline__ float exact_dot(const uint8_t* blocks, int K, const T* x) {
    float s = 0.f;
    for (int b = 0; b < K / 32; ++b) {
        const uint8_t* blk = blocks + 18 * b;
        const float d = f16_bits_to_float(*reinterpret_cast<const uint16_t*>(blk));
        for (int j = 0; j < 32; ++j) {
            const uint32_t byte = blk[2 + (j & 15)];
            const float q = magic_minus8((j < 16 ? byte & 15u : byte >> 4) | kMagicBits);
            s = fmaf(load1(x + 32 * b + j), q * d, s);
        }
    }
    return s;
}
__device__ __forceinline__ bool finite4(float4 v) { return fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, v.w * 0.f))) == 0.f; }

// The expert of sorted row p.
__device__ __forceinline__ int expert_of(const int32_t* starts, int n, int p) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid + 1] <= p) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Inner activations of sorted row p that are not finite, four from `at` on: again, from x.
template <typename T>
__device__ __forceinline__ float4 inner_again(const ExpertsView& e, const ExpertsCall& c, const int32_t* starts,
                                           const int32_t* order, int p, int at, float4 v) {
    const int ex = expert_of(starts, e.n, p);
    const T* x = static_cast<const T*>(c.x) + static_cast<int64_t>(order[p] / c.top_k) * c.x_stride;
    const int64_t row_bytes = e.hidden / 32 * 18;
    float* vs = &v.x;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        if (isfinite(vs[i])) continue;
        const float u = exact_dot(e.up + ex * e.up_stride + (at + i) * row_bytes, e.hidden, x);
        if (e.gate)
            vs[i] = activate<true>(exact_dot(e.gate + ex * e.gate_stride + (at + i) * row_bytes, e.hidden, x), e.activation) * u;
        else vs[i] = activate<true>(u, e.activation);
    }
    return v;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) { return load_q4(p); }

// A row as f16 pieces, times the power of two that takes its largest value to 2^13 ..
// 2^14; a thread has 8 elements of a block, those that a word's quants are for, in the
// order in which they unpack.  The products keep 2^-38 of the largest value.
// With `mend` not null, a row with elements that are not finite is handed to it first.
struct NoMend {
    static constexpr bool kThere = false;
    __device__ __forceinline__ void operator()(int) const {}
};
template <bool LO, int THREADS, typename T, typename F>
__device__ __forceinline__ void split_row(const T* x, int K, __half* hi, __half* lo, float* unit, F&& mend) {
    __shared__ float part[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto from = [&](int c) { return x + 32 * (c >> 2) + 4 * (c & 3); };
    const int chunks = K / 8;
    constexpr int kHeld = 4;  // chunks of a thread that stay in registers
    float4 a[kHeld], b[kHeld];
    auto largest = [](float4 v) { return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))); };
    float amax;
#pragma unroll 1
    for (int round = 0;; ++round) {
        amax = 0.f;
        bool fine = true;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int c = threadIdx.x + i * THREADS;
            a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < chunks) a[i] = load4(from(c)), b[i] = load4(from(c) + 16);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            amax = fmaxf(amax, fmaxf(largest(a[i]), largest(b[i])));
            if (std::decay_t<F>::kThere) fine = fine && finite4(a[i]) && finite4(b[i]);
        }
        for (int c = threadIdx.x + kHeld * THREADS; c < chunks; c += THREADS) {
            const float4 u = load4(from(c)), v = load4(from(c) + 16);
            amax = fmaxf(amax, fmaxf(largest(u), largest(v)));
            if (std::decay_t<F>::kThere) fine = fine && finite4(u) && finite4(v);
        }
        if (!std::decay_t<F>::kThere || round == 1 || !__syncthreads_or(!fine)) break;
#pragma unroll 1
        for (int q = threadIdx.x; q < K / 4; q += THREADS) mend(4 * q);
        __syncthreads();  // (what a thread mends, another may read)
    }
    amax = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(amax)));
    if (lane == 0) part[warp] = amax;
    __syncthreads();
    amax = __uint_as_float(__reduce_max_sync(kAll, lane < THREADS / 32 ? __float_as_uint(part[lane]) : 0u));
    const int up = min(126, 13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127));
    const float f = pow2(up);
    if (threadIdx.x == 0) *unit = pow2(-up);
    auto store = [&](int c, float4 a, float4 b) {
        const float v[8] = {a.x, a.z, a.y, a.w, b.x, b.z, b.y, b.w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v0 = v[2 * e] * f, v1 = v[2 * e + 1] * f;
            const __half2 x2 = __floats2half2_rn(v0, v1);
            h[e] = word(x2);
            const float2 back = __half22float2(x2);
            if (LO) l[e] = word(__floats2half2_rn(v0 - back.x, v1 - back.y));
        }
        *reinterpret_cast<uint4*>(hi + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
        if (LO) *reinterpret_cast<uint4*>(lo + 8 * c) = make_uint4(l[0], l[1], l[2], l[3]);
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int c = threadIdx.x + i * THREADS;
        if (c < chunks) store(c, a[i], b[i]);
    }
    for (int c = threadIdx.x + kHeld * THREADS; c < chunks; c += THREADS) store(c, load4(from(c)), load4(from(c) + 16));
}

// CTAs 0 .. n - 1: the pairs in the experts' order.  With `rows`, the CTAs after them: a
// pair's token row each, as pieces at the pair's sorted place, which the CTA counts itself.
template <typename T>
__global__ void __launch_bounds__(kSetupThreads)
    experts_setup(const ExpertsCall c, int n, int K, int32_t* starts, int32_t* order, int32_t* place,
                  unsigned* counters, __half* hi, __half* lo, float* unit) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int pairs = c.n_tokens * c.top_k;
    if (static_cast<int>(blockIdx.x) < n) {
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < 2 * kCounters; i += kSetupThreads) counters[i] = 0;
        order_pairs(blockIdx.x, c.ids, pairs, n, starts, order, place, c.err);
        return;
    }
    const int pair = blockIdx.x - n, e = c.ids[pair];
    if (e < 0 || e >= n) return;
    __shared__ int own;
    const Ranks r = rank_pairs(e, c.ids, pairs, n);
    if (r.lo <= pair && pair < r.hi) {
        const int lane = threadIdx.x & 31;
        int p = 0;
        for (int i = r.lo + lane; i < pair; i += 32) p += c.ids[i] == e;
        p = __reduce_add_sync(kAll, p);
        if (lane == 0) own = r.below + r.before + p;
    }
    __syncthreads();
    const int64_t p = own, pitch = piece_pitch(K);
    const T* x = static_cast<const T*>(c.x) + static_cast<int64_t>(pair / c.top_k) * c.x_stride;
    split_row<sizeof(T) == 4, kSetupThreads>(x, K, hi + p * pitch, lo + p * pitch, unit + p, NoMend{});
}

// The pairs' tokens as pieces, a sorted row each.
template <typename T>
__global__ void __launch_bounds__(128)
    experts_split(const ExpertsCall c, int K, const int32_t* starts, const int32_t* order, int n, __half* hi, __half* lo, float* unit) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t p = blockIdx.x, pitch = piece_pitch(K);
    if (p >= starts[n]) return;
    const T* x = static_cast<const T*>(c.x) + static_cast<int64_t>(order[p] / c.top_k) * c.x_stride;
    split_row<sizeof(T) == 4, 128>(x, K, hi + p * pitch, lo + p * pitch, unit + p, NoMend{});
}

template <typename T>
struct Mend {
    static constexpr bool kThere = true;
    const ExpertsView& e;
    const ExpertsCall& c;
    const int32_t *starts, *order;
    float* row;
    int p;
    __device__ __forceinline__ void operator()(int at) const {
        float4 v = *reinterpret_cast<const float4*>(row + at);
        if (!finite4(v)) *reinterpret_cast<float4*>(row + at) = inner_again<T>(e, c, starts, order, p, at, v);
    }
};

// The inner activations as pieces, those that are not finite taken again first.  bf16 calls: one piece, 11 bits,
// whose rounding (2^-11, as that of the weights where rows are many) is an eighth of the output's own; a second
// piece would be another product.
template <int THREADS, typename T>
__global__ void __launch_bounds__(THREADS)
    experts_inner(const ExpertsView e, const ExpertsCall c, float* inner, const int32_t* starts, const int32_t* order, __half* hi,
                  __half* lo, float* unit) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t p = blockIdx.x, pitch = piece_pitch(e.inner);
    if (p >= starts[e.n]) return;
    float* row = inner + p * e.inner;
    const Mend<T> mend{e, c, starts, order, row, static_cast<int>(p)};
    split_row<sizeof(T) == 4, THREADS>(row, e.inner, hi + p * pitch, lo + p * pitch, unit + p, mend);
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Outputs of sorted row p's expert that are not finite, four from `at` on: again, from the inner
// activations.
__device__ __forceinline__ float4 down_again(const ExpertsView& e, const int32_t* starts, const float* inner, int p, int at,
                                          float4 v) {
    const uint8_t* w = e.down + expert_of(starts, e.n, p) * e.down_stride;
    float* vs = &v.x;
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
        if (!isfinite(vs[i]))
            vs[i] = exact_dot(w + static_cast<int64_t>(at + i) * (e.inner / 32 * 18), e.inner, inner + static_cast<int64_t>(p) * e.inner);
    return v;
}

// out[t] = the weighted sum of the token's pairs, in their order.
template <typename T>
__global__ void __launch_bounds__(128)
    experts_combine(const ExpertsView e, const ExpertsCall c, const int32_t* starts, const int32_t* place, const float* inner,
                    const float* part) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int at = (blockIdx.x * 128 + threadIdx.x) * 4;
    if (at >= e.hidden) return;
    for (int t = blockIdx.y; t < c.n_tokens; t += gridDim.y) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAtOnce = 8;  // pairs whose loads are on their way together
#pragma unroll 1
        for (int j0 = 0; j0 < c.top_k; j0 += kAtOnce) {
            const int64_t pair = static_cast<int64_t>(t) * c.top_k + j0;
            const int n = min(kAtOnce, c.top_k - j0);
            int p[kAtOnce];
            float w[kAtOnce];
            float4 y[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) p[j] = j < n ? place[pair + j] : -1, w[j] = j < n ? c.weights[pair + j] : 0.f;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (p[j] >= 0) y[j] = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(p[j]) * e.hidden + at);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (p[j] < 0) continue;
                if (!finite4(y[j])) y[j] = down_again(e, starts, inner, p[j], at, y[j]);
                s.x = fmaf(w[j], y[j].x, s.x), s.y = fmaf(w[j], y[j].y, s.y), s.z = fmaf(w[j], y[j].z, s.z), s.w = fmaf(w[j], y[j].w, s.w);
            }
        }
        store4(static_cast<T*>(c.out) + t * c.out_stride + at, s);
    }
}

template <typename T>
cudaError_t launch_type(const ExpertsView& e, const ExpertsCall& c, const DeviceInfo& dev, cudaStream_t stream) {
    const Parts at = layout(e, c.n_tokens, c.top_k);
    const int pairs = c.n_tokens * c.top_k;
    auto words = [&](int64_t offset) { return reinterpret_cast<int32_t*>(c.ws + offset); };
    auto floats = [&](int64_t offset) { return reinterpret_cast<float*>(c.ws + offset); };
    auto halves = [&](int64_t offset) { return reinterpret_cast<__half*>(c.ws + offset); };
    int32_t *starts = words(at.starts), *order = words(at.order), *place = words(at.place);
    unsigned* counters = reinterpret_cast<unsigned*>(words(at.counters));
    float *inner = floats(at.inner), *part = floats(at.part);
    __half *x_hi = halves(at.x_pieces), *x_lo = x_hi + pairs * piece_pitch(e.hidden);
    __half *i_hi = halves(at.i_pieces), *i_lo = i_hi + pairs * piece_pitch(e.inner);

    // Up to this many pairs a row's CTA counts its own place, which saves a launch (one token: 65 us against 67, 35
    // against 37); the counting takes (pairs / 512) ids a thread in every CTA (1024 pairs: 126 us against 121).
    constexpr int kOwnPlace = 256;
    const bool own_place = pairs <= kOwnPlace;
    cudaError_t err = launch_pdl(experts_setup<T>, dim3(e.n + (own_place ? pairs : 0)), dim3(kSetupThreads), 0, stream, c, e.n,
                                 e.hidden, starts, order, place, counters, x_hi, x_lo, floats(at.x_unit));
    if (err != cudaSuccess) return err;
    note_launch();
    if (!own_place) {
        err = launch_pdl(experts_split<T>, dim3(pairs), dim3(128), 0, stream, c, e.hidden, starts, order, e.n, x_hi, x_lo,
                         floats(at.x_unit));
        if (err != cudaSuccess) return err;
        note_launch();
    }
    const uint8_t* const gate = e.gate ? e.gate : e.up;
    ExpertsMm m = {starts, floats(at.x_unit), inner, floats(at.split), counters, c.err, {e.gate ? nullptr : e.up, e.up},
                   {e.gate ? e.gate_stride : e.up_stride, e.up_stride}, e.n, e.hidden, e.inner, e.activation, at.split_cols,
                   0x64006400u, false, {gate, e.up}};
    // Few rows an expert: experts_few.cu (16 experts of 4096 x 4096, 8 rows each: bf16 127 us against 143, f32
    // 191 against 221; 12 rows each: 152 against 141, 244 against 219).
    const bool few = pairs <= 8 * static_cast<int64_t>(e.n);
    auto products = [&](bool down, const __half* hi, const __half* lo) {
        return few ? launch_experts_few(m, e, c.type, hi, lo, dev, stream)
                   : launch_experts_mm(m, e, down, c.type, hi, lo, pairs, dev, stream);
    };
    if ((err = products(false, x_hi, x_lo)) != cudaSuccess) return err;
    // Few rows take many threads each, for the latency (192 rows of 4096: 219 us in all against 221), and so do long
    // ones, which stay in registers between their maximum and their pieces (8192 rows of 14336: 133 us against
    // 146); many short ones few (64 experts with 48 rows of 1408 each: 163 us in all against 173).
    const bool wide = pairs <= 512;
    err = wide || e.inner > 4096 ? launch_pdl(experts_inner<512, T>, dim3(pairs), dim3(512), 0, stream, e, c, inner, starts, order, i_hi, i_lo,
                            floats(at.i_unit))
               : launch_pdl(experts_inner<128, T>, dim3(pairs), dim3(128), 0, stream, e, c, inner, starts, order, i_hi, i_lo,
                            floats(at.i_unit));
    if (err != cudaSuccess) return err;
    note_launch();
    m = {starts, floats(at.i_unit), part, floats(at.split), counters + kCounters, c.err, {e.down, e.down},
         {e.down_stride, e.down_stride}, e.n, e.inner, e.hidden, QM_ACT_NONE, at.split_cols, 0x64006400u, true, {e.down, e.down}};
    if ((err = products(true, i_hi, i_lo)) != cudaSuccess) return err;
    err = launch_pdl(experts_combine<T>, dim3((e.hidden + 511) / 512, c.n_tokens < 4096 ? c.n_tokens : 4096), dim3(128), 0,
                     stream, e, c, starts, place, inner, part);
    if (err == cudaSuccess) note_launch();
    return err;
}

}  // namespace

int64_t experts_workspace(const ExpertsView& e, int64_t n_tokens, int64_t top_k) { return layout(e, n_tokens, top_k).bytes; }

cudaError_t launch_experts(const ExpertsView& e, const ExpertsCall& c, const DeviceInfo& dev, cudaStream_t stream) {
    return c.type == KvType::kF32 ? launch_type<float>(e, c, dev, stream) : launch_type<__nv_bfloat16>(e, c, dev, stream);
}

}  // namespace qm
