// Each token's experts (qm_route_experts): scores, groups, the top_k largest
// choices, their weights.
//
// A warp per token; lane l holds the experts l, l + 32, ...  A choice becomes a
// 32-bit key whose unsigned order is the choices' order, so that one step of the
// selection is two warp-wide integer reductions: the largest key, and the lowest
// expert that has it.  Scores are computed in f32.  Where selected choices lie closer
// than the scores' error, those that could change places (a lane each) are put in order
// by f64 choices (64-bit keys); where groups at the border do, the whole row is done
// again in f64.  So the ids are those of the formula and not of a rounding; without a
// bias the logits themselves are compared, which is exact.  (f64 is slow here: a row
// done again takes some 10 us, and one in a thousand asks for it; with the few of them
// in order by themselves 4096 tokens, 256 experts in 8 groups take 18 us against 34.)
#include <cuda_bf16.h>

#include <cfloat>

#include "qm_device.cuh"

namespace qm {

namespace {

constexpr int kWarps = 4;  // tokens of a CTA
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float logit(const float* p) { return *p; }
__device__ __forceinline__ float logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Unsigned keys in the numbers' order; -0 as +0, NaN below all numbers, and 0 for
// an expert that is out.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (isnan(v)) return 1u;
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
    if (isnan(v)) return 1u;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ bool apart(uint32_t above, uint32_t below, float near) {
    const float a = value_of(above);
    return a - value_of(below) > near + 0x1p-22f * fabsf(a);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// The largest key of the warp and the lowest expert that has it.
template <int PER, typename K>
__device__ __forceinline__ void largest(const K (&key)[PER], int lane, K* top, int* which) {
    K mine = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (key[i] > mine) {
            mine = key[i];
            at = i;
        }
    const K m = warp_max(mine);
    const unsigned e = mine == m ? static_cast<unsigned>(32 * at + lane) : kAll;
    *top = m;
    *which = static_cast<int>(__reduce_min_sync(kAll, e));
}

// Sum of a group's one or two largest choices, and the second, on every lane.
template <typename F>
__device__ __forceinline__ F warp_top(F a, F b, bool both, F* second) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const F a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
        const F lo = a < a2 ? a : a2;
        a = a < a2 ? a2 : a;
        b = b < b2 ? b2 : b;
        b = b < lo ? lo : b;
    }
    *second = b;
    return both ? a + b : a;
}

// Clears the keys of the experts whose groups do not count among the top_groups
// largest.  True if one of those may be as large as one that stays, in f32: a group's sum a + b
// is off by `near` for its scores and by 2^-24 (|a| + |b| + |a + b|) for the roundings of choices
// and sum, where a and b may be far larger than a + b.
template <int PER, typename F, typename K>
__device__ __forceinline__ bool drop_groups(const RouteCall& c, const F (&choice)[PER], K (&key)[PER], int lane, float near) {
    const int size = c.experts / c.groups;
    constexpr F kLow = -INFINITY;
    const bool both = c.group_top == 2 && size > 1;
    F mine[2] = {kLow, kLow};                // groups `lane` and lane + 32
    [[maybe_unused]] F second[2] = {0, 0};  // and their second choices, where those count
    for (int g = 0; g < c.groups; ++g) {
        F a = kLow, b = kLow;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = 32 * i + lane;
            if (e >= g * size && e < (g + 1) * size) {
                const F v = isnan(choice[i]) ? kLow : choice[i];
                if (v > a) {
                    b = a;
                    a = v;
                } else if (v > b) {
                    b = v;
                }
            }
        }
        F b_top;
        const F s = warp_top(a, b, both, &b_top);
        if (lane == (g & 31)) {
            mine[g >> 5] = s;
            if (sizeof(F) == 4 && both) second[g >> 5] = b_top;
        }
    }
    K gkey[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) gkey[i] = 32 * i + lane < c.groups ? key_of(mine[i]) : 0;
    uint64_t stays = 0;
    for (int n = 0; n < c.top_groups; ++n) {
        K top;
        int g;
        largest(gkey, lane, &top, &g);
        stays |= uint64_t(1) << g;
        if (lane == (g & 31)) gkey[g >> 5] = 0;
    }
    bool close = false;
    if constexpr (sizeof(F) == 4) {
        // The most that a group that is out may be, and the least of one that stays.  (A sum past f32's range is the
        // end of that range at least.  One that counts a masked expert is -infinity, or NaN, in any precision:
        // out, it is above no other.)
        uint32_t most = 0, least = 0;  // keys, of `least` the complement
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = 32 * i + lane;
            if (g >= c.groups) continue;
            const float at = fminf(fmaxf(mine[i], -FLT_MAX), FLT_MAX);  // (NaN: the lowest)
            // (|a| <= |a + b| + |b|; and 2^-24 of the sum for the rounding of at +- by)
            const float by = isfinite(mine[i]) ? near + 0x1.01p-23f * (2.f * fabsf(mine[i]) + fabsf(second[i])) : 0.f;
            if ((stays >> g) & 1u) least = max(least, ~key_of(at - by));
            else if ((both ? second[i] : mine[i]) != kLow) most = max(most, key_of(at + by));
        }
        close = c.top_groups < c.groups && warp_max(most) >= ~warp_max(least);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 32 * i + lane;
        if (e < c.experts && !((stays >> (e / size)) & 1u)) key[i] = 0;
    }
    return close;
}

// The row's experts, largest choice first: lane j gets the j-th.  With `near` not negative
// (32-bit keys) the next lanes get the ones after the last that could change places with one
// of them, *n is how many lanes have one, and *ordered says whether all of the first top_k
// are more than `near` and 2^-22 of themselves apart from each other and from the rest.  (Of
// two of different size the larger counts: an expert masked by a bias of -infinity is far
// from all others.)
template <int PER, typename K>
__device__ __forceinline__ int select(const RouteCall& c, K (&key)[PER], int lane, float near, bool* ordered, int* n) {
    int id = 0;
    K last = 0;
    for (int j = 0; j <= 32; ++j) {
        if (j >= c.top_k && near < 0.f) break;
        K top;
        int e;
        largest(key, lane, &top, &e);
        if constexpr (sizeof(K) == 4) {
            if (near >= 0.f) {
                const bool far = j == 0 || !top || apart(last, top, near);
                if (!far) *ordered = false;
                if (j >= c.top_k && far) break;
            }
        }
        *n = j + 1;
        if (j == 32) break;
        if (lane == j) id = e;
        last = top;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == 32 * i + lane) key[i] = 0;
    }
    return id;
}

// The same experts in the order of their f64 choices: lanes 0 .. n - 1 have one each.
template <int PER, typename T>
__device__ __noinline__ int order_f64(const RouteCall& c, const T* row, int lane, int id, int n, float mx) {
    double score;
    const double x = static_cast<double>(logit(row + id));
    if (c.sigmoid) {
        score = 1.0 / (1.0 + exp(-x));
    } else {
        double sum = 0.0;
#pragma unroll 1
        for (int i = 0; i < PER; ++i) {
            const int e = 32 * i + lane;
            if (e < c.experts) sum += exp(static_cast<double>(logit(row + e)) - mx);
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        score = mx == -INFINITY ? 0.0 : exp(x - mx) / sum;  // (a row of nothing but -infinity: the bias alone)
    }
    uint64_t key = lane < n ? key_of(score + static_cast<double>(c.bias[id])) : 0;
    int sorted = 0;
    for (int j = 0; j < c.top_k; ++j) {
        const uint64_t top = warp_max(key);
        const int e = static_cast<int>(__reduce_min_sync(kAll, key == top && lane < n ? static_cast<unsigned>(id) : kAll));
        if (lane == j) sorted = e;
        if (id == e && lane < n) key = 0;
    }
    return sorted;
}

// A row's experts from f64 choices.
template <int PER, typename T>
__device__ __noinline__ int select_f64(const RouteCall& c, const T* row, int lane) {
    double choice[PER];
    double mx = -INFINITY, sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 32 * i + lane;
        choice[i] = e < c.experts ? static_cast<double>(logit(row + e)) : -INFINITY;
        mx = fmax(mx, choice[i]);
    }
    if (!c.sigmoid) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mx = fmax(mx, __shfl_xor_sync(kAll, mx, d));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const double x = choice[i];
        if (c.sigmoid) choice[i] = 1.0 / (1.0 + exp(-x));
        else choice[i] = x == -INFINITY ? 0.0 : exp(x - mx);
        sum += choice[i];
    }
    if (!c.sigmoid) {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        const double r = sum > 0.0 ? 1.0 / sum : 1.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) choice[i] *= r;
    }
    uint64_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 32 * i + lane;
        if (c.bias && e < c.experts) choice[i] += static_cast<double>(c.bias[e]);
        key[i] = 0;
        if (e < c.experts) key[i] = key_of(c.bias ? choice[i] : static_cast<double>(logit(row + e)));
    }
    if (c.groups > 1) drop_groups(c, choice, key, lane, 0.f);
    int n;
    return select(c, key, lane, -1.f, nullptr, &n);
}

// The weights of row t's experts (lane j's is the j-th), their scores divided by the sum in f64.  (It writes
// them itself, so that its caller keeps nothing across the call.)
template <typename T>
__device__ __noinline__ void small_weights(const RouteCall& c, int64_t t, int lane, int id, float mx) {
    const T* row = static_cast<const T*>(c.logits) + t * c.stride;
    double s = 0.0;
    if (lane < c.top_k) {
        const double x = static_cast<double>(logit(row + id));
        if (c.sigmoid) s = 1.0 / (1.0 + exp(-x));
        else s = x == -INFINITY ? 0.0 : exp(x - mx);  // (the sum of all scores cancels)
    }
    double sum = s;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    if (lane < c.top_k) {
        c.ids[t * c.top_k + lane] = id;
        c.weights[t * c.top_k + lane] = (sum == 0.0 ? 0.f : static_cast<float>(s / sum)) * c.scale;
    }
}

// CTAs of an SM, for the registers that this leaves (up to 64 experts 32: 4096 tokens with a bias 8.1 us, 9.3 with 40).
template <int PER>
constexpr int kCtasOf = PER <= 2 ? 16 : PER <= 4 ? 10 : PER <= 8 ? 8 : PER <= 16 ? 5 : 3;

template <int PER, typename T>
__global__ void __launch_bounds__(kWarps * 32, kCtasOf<PER>) route_kernel(const RouteCall c) {
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    grid_dependency_wait();
    if (t >= c.n_tokens) return;
    const T* row = static_cast<const T*>(c.logits) + t * c.stride;
    float l[PER], s[PER];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 32 * i + lane;
        l[i] = e < c.experts ? logit(row + e) : -INFINITY;
        mx = fmaxf(mx, l[i]);
    }
    bool bad = false;  // NaN or +infinity: the whole row's softmax is NaN
    if (c.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = 1.f / (1.f + expf(-l[i]));
    } else {
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            s[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - mx);
            sum += s[i];
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        bad = isnan(sum);
        const float r = sum > 0.f ? 1.f / sum : 1.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) s[i] = bad ? NAN : s[i] * r;
    }
    float choice[PER];
    uint32_t key[PER];
    float s_top = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 32 * i + lane;
        choice[i] = s[i];
        if (c.bias && e < c.experts) choice[i] += c.bias[e];
        key[i] = e < c.experts ? key_of(c.bias ? choice[i] : l[i]) : 0;
        if (e < c.experts) s_top = fmaxf(s_top, s[i]);
    }
    bool ordered = true;
    float near = 0.f;
    if (c.bias || c.groups > 1) {
        s_top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(s_top)));
        // Twice what a choice may be off by: a score s = exp(d) / sum by (|d| + 8) 2^-23 of
        // itself (d's rounding, exp's 2 units, the sum's PER + 5 roundings of terms that are
        // mostly small, the products), where s |d| is s_top / e at most; a sigmoid by 4 units.
        // The bias adds a rounding of the choice (2^-24 of it).  A group's sum of two is off by
        // `near` at most, and the roundings (drop_groups).
        // Scores near the end of f32's range are off by 2^-128 at most.
        near = 0x1p-22f * (c.sigmoid ? 4.f * s_top : (9.f + PER) * s_top) + 0x1p-126f;
    }
    bool again = false;
    if (c.groups > 1) again = drop_groups(c, choice, key, lane, near);
    // Logits are compared as they are.
    int n;
    int id = select(c, key, lane, c.bias && !again ? near : -1.f, &ordered, &n);
    if (!bad && (again || (!ordered && n > 32))) id = select_f64<PER>(c, row, lane);
    else if (!bad && !ordered) id = order_f64<PER>(c, row, lane, id, n, mx);
    // The chosen scores, one per lane.
    float w = 0.f;
    for (int j = 0; j < c.top_k; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i == (e >> 5)) v = s[i];
        v = __shfl_sync(kAll, v, e & 31);
        if (lane == j) w = v;
    }
    if (c.renormalize) {
        float sum = w;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        // (Scores near the end of f32's range have few bits there, or none: they lose 2^-128 at most, and
        // weights so 2^-102.)
        if (sum < 0x1p-26f) return small_weights<T>(c, t, lane, id, mx);
        w /= sum;
    }
    if (lane < c.top_k) {
        c.ids[t * c.top_k + lane] = id;
        c.weights[t * c.top_k + lane] = w * c.scale;
    }
}

template <typename T>
cudaError_t launch_type(const RouteCall& c, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((c.n_tokens + kWarps - 1) / kWarps)), block(kWarps * 32);
    const int per = (c.experts + 31) / 32;
    note_launch();
    if (per <= 1) return launch_pdl(route_kernel<1, T>, grid, block, 0, stream, c);
    if (per <= 2) return launch_pdl(route_kernel<2, T>, grid, block, 0, stream, c);
    if (per <= 4) return launch_pdl(route_kernel<4, T>, grid, block, 0, stream, c);
    if (per <= 8) return launch_pdl(route_kernel<8, T>, grid, block, 0, stream, c);
    if (per <= 16) return launch_pdl(route_kernel<16, T>, grid, block, 0, stream, c);
    return launch_pdl(route_kernel<32, T>, grid, block, 0, stream, c);
}

}  // namespace

cudaError_t launch_route_experts(const RouteCall& c, cudaStream_t stream) {
    return c.type == KvType::kF32 ? launch_type<float>(c, stream) : launch_type<__nv_bfloat16>(c, stream);
}

}  // namespace qm
