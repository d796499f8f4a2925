// The paged Q4_0 key/value cache: quantizing rows into it, reading them back,
// and cutting it back to the tokens that collected the most attention.
#include <algorithm>

#include "kv_cache.cuh"

namespace qm {

// The error word of every kernel of the cache (KvView::err): one word, so that
// qm_device_status has one more to read, not one for each file.
__device__ unsigned int g_kv_error = 0;

namespace {

constexpr int kThreads = 256;

// Eight elements as they lie in memory (bf16: 8-byte aligned), and as floats.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float x[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        a = reinterpret_cast<const uint2*>(p)[0], b = reinterpret_cast<const uint2*>(p)[1];
    }
    __device__ __forceinline__ void get(float x[8]) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
};

// Q4_0 quantization of a block of 32 by 4 lanes of 8 elements each (i: the lane's
// number in the block): m = the first element of largest magnitude, d = m / -8,
// r = 1 / d (both correctly rounded f32 divisions), q = min(15, floor(x r + 8.5))
// with the product and the sum each rounded to f32; the stored scale is d
// narrowed to binary16.  With m mapped to q = 0 the other sign gets only 7 steps:
// taking the signed maximum gives the larger side the extra one.  NaN elements
// do not raise the maximum; q = 8 (the value 0) where x r is NaN or d is 0.
// Returns the eight quants as bytes; *scale = d's bits.
__device__ __forceinline__ uint2 quantize_q4_lane(const float x[8], int i, uint32_t* scale) {
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        hi = fmaxf(fmaxf(hi, x[e]), x[e + 1]);
        lo = fminf(fminf(lo, x[e]), x[e + 1]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    }
    float m = hi > -lo ? hi : lo;
    if (__any_sync(0xFFFFFFFFu, hi == -lo && hi > 0.f)) {  // both signs: the first one counts
        uint32_t at = 0x7FFFFFFFu;  // smallest 2 * index + sign
#pragma unroll
        for (int e = 7; e >= 0; --e)
            if (fabsf(x[e]) == hi) at = 2u * (8 * i + e) + (__float_as_uint(x[e]) >> 31);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) at = min(at, __shfl_xor_sync(0xFFFFFFFFu, at, o));
        if (hi == -lo && !(at & 1u)) m = hi;
    }
    const float d = __fdiv_rn(m, -8.f);
    const float r = d == 0.f ? 0.f : __frcp_rn(d);
    *scale = f16_bits_rn(d);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float t = __fadd_rn(__fmul_rn(x[e], r), 8.5f);
        t = t == t ? fminf(fmaxf(t, 0.f), 15.5f) : 8.5f;
        // Adding 2^23 toward zero leaves floor(t) in the low bits.
        w[e >> 2] |= (__float_as_uint(__fadd_rz(t, 8388608.f)) & 15u) << (8 * (e & 3));
    }
    return make_uint2(w[0], w[1]);
}

// How the rows of a call go to warps: eight blocks at a time, i.e. one kv head of
// kTokens consecutive rows; a warp takes `heads_each` heads of them, of keys or of
// values, one after another.  Lane 4 s + i has elements 8 i .. 8 i + 7 of block
// s % NB of row s / NB.
template <int NB>
struct RowWork {
    static constexpr int kTokens = 8 / NB;
    int row, blk, i, h_first, h_end, pos;
    bool is_v, in;         // `in`: this lane has a row with a place in the cache
    int64_t cell0, h_step;  // byte offset of its cell of head 0, and from head to head
    __device__ RowWork(const KvView& c, const KvRows& r, int heads_each, unsigned int* err) {
        const int lane = threadIdx.x & 31;
        const int parts = (c.heads + heads_each - 1) / heads_each;
        const unsigned unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
        const unsigned group = unit / (2 * parts);
        const int rest = static_cast<int>(unit - group * 2 * parts);
        is_v = rest >= parts;
        h_first = (is_v ? rest - parts : rest) * heads_each;
        h_end = min(c.heads, h_first + heads_each);
        const int s = lane >> 2;
        i = lane & 3;
        blk = s % NB;
        const int64_t at = static_cast<int64_t>(group) * kTokens + s / NB;
        in = s / NB < kTokens && at < r.n_tokens;
        row = in ? static_cast<int>(at) : 0;
        pos = 0;
        cell0 = h_step = 0;
        if (!in) return;
        const int b = kv_seq_of_row(r, c.n_seqs, row);
        in = b >= 0;
        if (!in) return;
        int first, count;
        kv_rows(r, b, &first, &count, err);
        pos = kv_length(c, b, err) - count + (row - first);
        if (row - first >= count || pos < 0) {
            atomicOr(err, kErrRange);
            in = false;
            return;
        }
        cell0 = kv_cell(c, b, 0, pos, err);
        in = cell0 >= 0;
        h_step = static_cast<int64_t>(1 << (c.page_shift - 4)) * cell_bytes(32 * NB);
    }
};

// Memory-bound: 4 (or 2) bytes read and 9/16 written per element; about 100
// instructions per 8 elements of a lane.  Measured: 8 ragged prompts of up to 4096
// rows, 8 kv heads, D = 128, bf16: 42 us, 3.5 TB/s; with the read back 89 us.
// Warps to switch between matter more than loads in flight: 6 CTAs per SM with
// 32 bytes a lane ahead 89 us, 4 with 64 bytes 94, 8 (which spills) 102.
template <int NB, typename T>
__global__ void __launch_bounds__(kThreads, 6)
    kv_append_kernel(KvView c, KvRows r, const T* k, const T* v, int64_t k_stride, int64_t v_stride, int heads_each) {
    grid_launch_dependents();
    grid_dependency_wait();
    const RowWork<NB> w(c, r, heads_each, c.err);
    const T* src = (w.is_v ? v + w.row * v_stride : k + w.row * k_stride) + 32 * w.blk + 8 * w.i;
    uint8_t* pool = w.is_v ? c.v : c.k;
    const int slot = w.pos & 15;
    constexpr int kAhead = 4 / sizeof(T);  // heads whose elements are on their way: 32 bytes a lane
    Eight<T> ahead[kAhead] = {};
#pragma unroll
    for (int x = 0; x < kAhead; ++x)
        if (w.in && w.h_first + x < w.h_end) ahead[x].load(src + (w.h_first + x) * (32 * NB));
#pragma unroll 1
    for (int h = w.h_first; h < w.h_end; ++h) {
        float y[8];
        ahead[0].get(y);
#pragma unroll
        for (int x = 0; x + 1 < kAhead; ++x) ahead[x] = ahead[x + 1];
        if (w.in && h + kAhead < w.h_end) ahead[kAhead - 1].load(src + (h + kAhead) * (32 * NB));
        uint32_t scale;
        uint2 q = quantize_q4_lane(y, w.i, &scale);
        // Lanes 0, 1 of a block have the low nibbles of bytes 0 .. 7, 8 .. 15, lanes 2, 3 the high ones.
        q.x |= __shfl_down_sync(0xFFFFFFFFu, q.x, 2) << 4;
        q.y |= __shfl_down_sync(0xFFFFFFFFu, q.y, 2) << 4;
        if (w.in) {
            uint8_t* cell = pool + w.cell0 + h * w.h_step;
            if (w.i < 2) *reinterpret_cast<uint2*>(cell + w.blk * 256 + slot * 16 + 8 * w.i) = q;
            if (w.i == 2)
                *reinterpret_cast<uint16_t*>(cell + cell_scales(32 * NB) + (slot * NB + w.blk) * 2) =
                    static_cast<uint16_t>(scale);
        }
    }
}

// The inverse: f32 values of the call's rows, contiguous [n_tokens][heads][dim].
// The same rows: 50 us, 4.8 TB/s, where the library's dequants of the same mix of
// bytes reach 0.9 of HBM: a lane's two 16-byte stores lie together, so each store
// instruction of a warp fills half of every sector that it touches.
template <int NB>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(KvView c, KvRows r, float* k, float* v, int heads_each) {
    grid_launch_dependents();
    grid_dependency_wait();
    const RowWork<NB> w(c, r, heads_each, c.err);
    if (!w.in) return;
    const uint8_t* pool = w.is_v ? c.v : c.k;
    const int slot = w.pos & 15;
    float* dst = (w.is_v ? v : k) + (static_cast<int64_t>(w.row) * c.heads) * (32 * NB) + 32 * w.blk + 8 * w.i;
#pragma unroll 4
    for (int h = w.h_first; h < w.h_end; ++h) {
        const uint8_t* cell = pool + w.cell0 + h * w.h_step;
        const uint2 q = *reinterpret_cast<const uint2*>(cell + w.blk * 256 + slot * 16 + 8 * (w.i & 1));
        const float d = f16_bits_to_float(
            *reinterpret_cast<const uint16_t*>(cell + cell_scales(32 * NB) + (slot * NB + w.blk) * 2));
        const uint32_t n[2] = {w.i < 2 ? q.x : q.x >> 4, w.i < 2 ? q.y : q.y >> 4};
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = magic_minus8(((n[e >> 2] >> (8 * (e & 3))) & 15u) | kMagicBits) * d;
        float4* to = reinterpret_cast<float4*>(dst + h * (32 * NB));
        to[0] = make_float4(y[0], y[1], y[2], y[3]);
        to[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
}

// Warps of RowWork, and how many heads each takes: one where that is what fills
// the GPU, else up to eight.
template <int NB>
unsigned row_warps(const KvView& c, const KvRows& r, int* heads_each) {
    const int64_t groups = (static_cast<int64_t>(r.n_tokens) + RowWork<NB>::kTokens - 1) / RowWork<NB>::kTokens;
    int each = 1;
    while (each < 8 && each < c.heads && groups * 2 * c.heads / (2 * each) >= c.sms * 64) each *= 2;
    *heads_each = each;
    return static_cast<unsigned>(groups * 2 * ((c.heads + each - 1) / each));
}

// ---- eviction --------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kEach = 8;  // consecutive tokens of a thread in the last pass

// Unsigned order of a score: larger score, larger key; NaN below everything.
__device__ __forceinline__ uint32_t score_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum of v over the threads before this one; *total: over all of them.
__device__ __forceinline__ int sel_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sums of the scan before have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const int before = warp ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0;
    return before + x - v;
}

// One CTA per (sequence, kv head): finds the smallest kept key by a radix select
// (three passes of 11, 11 and 10 bits: the first digit takes the exponent and
// two bits more, so ordinary scores do not all count in one bin), then
// writes the kept tokens in ascending order, 8192 at a time.  16 sequences of up to
// 8192 scores, 8 kv heads: 15 us, five passes over scores that stay in L1 or L2, with
// 128 of 152 SMs in use.
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(KvView c, EvictCall e, int set_lengths) {
    grid_launch_dependents();
    grid_dependency_wait();
    __shared__ int hist[2048];
    __shared__ int warp_sums[32];
    __shared__ int s_bin, s_need;
    const int h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x;
    const int L = kv_length(c, b, c.err);
    const float* w = e.weights + (static_cast<int64_t>(b) * c.heads + h) * e.weights_stride;
    float* wo = e.weights_out + (static_cast<int64_t>(b) * c.heads + h) * e.out_stride;
    int32_t* kept = e.kept + (static_cast<int64_t>(b) * c.heads + h) * e.budget;
    const int n_keep = min(L, e.budget);
    if (set_lengths && h == 0 && tid == 0) e.lengths_out[b] = n_keep;
    const int lo = min(e.sinks, L);            // tokens below lo and from hi on stay
    const int hi = max(lo, L - e.recent);
    const int need0 = n_keep - lo - (L - hi);  // of the tokens between
    const bool all = L <= e.budget;
    uint32_t prefix = 0, known = 0;  // the digits found so far, and their mask
    int need = need0;
    if (!all && need > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            hist[tid] = 0;
            hist[tid + 1024] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                const uint32_t key = score_key(w[j]);
                if ((key & known) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
            }
            __syncthreads();
            // Bins from the top: this thread's are bins - 1 - 2 tid and the one below.
            const int top = bins - 1 - 2 * tid;
            const int n1 = top >= 0 ? hist[top] : 0, n2 = top >= 1 ? hist[top - 1] : 0;
            int total;
            const int before = sel_scan(n1 + n2, warp_sums, &total);
            if (before < need && need <= before + n1) s_bin = top, s_need = need - before;
            if (before + n1 < need && need <= before + n1 + n2) s_bin = top - 1, s_need = need - before - n1;
            __syncthreads();
            prefix |= static_cast<uint32_t>(s_bin) << shift;
            known |= static_cast<uint32_t>(bins - 1) << shift;
            need = s_need;
        }
    }
    // Keys above `prefix` are kept, and the first `need` equal to it.
    int base_keep = 0, base_tie = 0;
#pragma unroll 1
    for (int j0 = 0; j0 < L; j0 += kSelThreads * kEach) {
        const int j = j0 + tid * kEach;
        float score[kEach];
        uint32_t keep = 0, tie = 0;  // a bit per token
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            score[x] = j + x < L ? w[j + x] : 0.f;
            if (j + x < L) {
                if (all || j + x < lo || j + x >= hi) keep |= 1u << x;
                else if (need0 > 0) {
                    const uint32_t key = score_key(score[x]);
                    if (key > prefix) keep |= 1u << x;
                    if (key == prefix) tie |= 1u << x;
                }
            }
        }
        int total;
        int rank = base_tie + sel_scan(__popc(tie), warp_sums, &total);
        base_tie += total;
#pragma unroll
        for (int x = 0; x < kEach; ++x)
            if ((tie >> x) & 1u) {
                if (rank < need) keep |= 1u << x;
                ++rank;
            }
        // (In place, weights_out == weights: a place is never above its token's, and
        // every score of this round has been read before the scans' barriers.)
        int at = base_keep + sel_scan(__popc(keep), warp_sums, &total);
        base_keep += total;
#pragma unroll
        for (int x = 0; x < kEach; ++x)
            if ((keep >> x) & 1u) {
                kept[at] = j + x;
                wo[at] = score[x];
                ++at;
            }
    }
    for (int i = n_keep + tid; i < e.budget; i += kSelThreads) {
        kept[i] = -1;
        wo[i] = 0.f;
    }
}

// Copies the kept tokens' quants and scales, of keys and values, to the first
// places of dst: a token per thread, all its pieces (16-byte quant rows, 256 bytes
// contiguous over 16 tokens) in flight together.  With in_place one CTA walks all
// of a head's tokens: a kept token never moves up, so reading a round before
// writing it is enough.  4096 of up to 8192 tokens for each of 16 sequences: 28 us,
// 149 MB, 5.3 TB/s.
template <int NB>
__global__ void __launch_bounds__(kThreads)
    kv_move_kernel(KvView src, KvView dst, const int32_t* kept_all, int budget, int in_place) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int h = blockIdx.y, b = blockIdx.z;
    const int32_t* kept = kept_all + (static_cast<int64_t>(b) * src.heads + h) * budget;
    const int n_keep = min(kv_length(src, b, src.err), budget);
    const int end = in_place ? n_keep : min(n_keep, static_cast<int>(blockIdx.x + 1) * kThreads);
    for (int at0 = in_place ? 0 : blockIdx.x * kThreads; at0 < end; at0 += kThreads) {
        const int at = at0 + threadIdx.x;
        uint4 q[2][NB];
        uint16_t sc[2][NB];
        int64_t to = -1;
        if (at < end) {
            const int token = kept[at];
            if (token < 0) atomicOr(src.err, kErrRange);  // (a length that changed meanwhile)
            const int64_t from = token < 0 ? -1 : kv_cell(src, b, h, token, src.err);
            to = kv_cell(dst, b, h, at, src.err);
            if (from < 0) to = -1;
            if (to >= 0) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const uint8_t* cell = (p ? src.v : src.k) + from;
                    const uint16_t* s = reinterpret_cast<const uint16_t*>(cell + cell_scales(32 * NB)) + (token & 15) * NB;
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        q[p][x] = *reinterpret_cast<const uint4*>(cell + x * 256 + (token & 15) * 16);
                        sc[p][x] = s[x];
                    }
                }
            }
        }
        if (in_place) __syncthreads();
        if (to >= 0) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint8_t* cell = (p ? dst.v : dst.k) + to;
                uint16_t* s = reinterpret_cast<uint16_t*>(cell + cell_scales(32 * NB)) + (at & 15) * NB;
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    *reinterpret_cast<uint4*>(cell + x * 256 + (at & 15) * 16) = q[p][x];
                    s[x] = sc[p][x];
                }
            }
        }
        if (in_place) __syncthreads();
    }
}

__global__ void kv_lengths_kernel(KvView src, int32_t* out, int budget) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < src.n_seqs) out[b] = min(kv_length(src, b, src.err), budget);
}

}  // namespace

namespace {

// F<NB> for the blocks of a head, 1 .. 8.
template <template <int> class F, typename... Args>
cudaError_t by_blocks(int dim, Args&&... args) {
    switch (dim / 32) {
        case 1: return F<1>::run(args...);
        case 2: return F<2>::run(args...);
        case 3: return F<3>::run(args...);
        case 4: return F<4>::run(args...);
        case 5: return F<5>::run(args...);
        case 6: return F<6>::run(args...);
        case 7: return F<7>::run(args...);
        default: return F<8>::run(args...);
    }
}

template <int NB>
struct Append {
    static cudaError_t run(const KvView& c, const KvRows& r, const void* k, const void* v, KvType type, int64_t k_stride,
                           int64_t v_stride, cudaStream_t stream) {
        int each;
        const unsigned warps = row_warps<NB>(c, r, &each);
        const dim3 grid((warps + kThreads / 32 - 1) / (kThreads / 32));
        note_launch();
        if (type == KvType::kF32)
            return launch_pdl(kv_append_kernel<NB, float>, grid, dim3(kThreads), 0, stream, c, r,
                              static_cast<const float*>(k), static_cast<const float*>(v), k_stride, v_stride, each);
        return launch_pdl(kv_append_kernel<NB, __nv_bfloat16>, grid, dim3(kThreads), 0, stream, c, r,
                          static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), k_stride, v_stride,
                          each);
    }
};

template <int NB>
struct Read {
    static cudaError_t run(const KvView& c, const KvRows& r, float* k, float* v, cudaStream_t stream) {
        int each;
        const unsigned warps = row_warps<NB>(c, r, &each);
        note_launch();
        return launch_pdl(kv_read_kernel<NB>, dim3((warps + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), 0,
                          stream, c, r, k, v, each);
    }
};

template <int NB>
struct Move {
    static cudaError_t run(const KvView& src, const KvView& dst, const EvictCall& e, unsigned chunks, int in_place,
                           cudaStream_t stream) {
        note_launch();
        return launch_pdl(kv_move_kernel<NB>, dim3(chunks, src.heads, src.n_seqs), dim3(kThreads), 0, stream, src, dst,
                          static_cast<const int32_t*>(e.kept), e.budget, in_place);
    }
};

}  // namespace

cudaError_t launch_kv_append(const KvView& c, const KvRows& r, const void* k, const void* v, KvType type,
                             int64_t k_stride, int64_t v_stride, cudaStream_t stream) {
    return by_blocks<Append>(c.dim, c, r, k, v, type, k_stride, v_stride, stream);
}

cudaError_t launch_kv_read(const KvView& c, const KvRows& r, float* k, float* v, cudaStream_t stream) {
    return by_blocks<Read>(c.dim, c, r, k, v, stream);
}

cudaError_t launch_kv_evict(const KvView& src, const KvView& dst, const EvictCall& e, cudaStream_t stream) {
    // The lengths are read until the last cell has moved: where the new ones go to
    // the same array they are written by a kernel of their own.
    const bool same_lengths = src.lengths == e.lengths_out;
    note_launch();
    cudaError_t err = launch_pdl(kv_select_kernel, dim3(src.heads, src.n_seqs), dim3(kSelThreads), 0, stream, src, e,
                                 same_lengths ? 0 : 1);
    if (err != cudaSuccess) return err;
    const bool in_place = src.table == dst.table && src.k == dst.k;
    const int64_t most = std::min<int64_t>(e.budget, src.max_len);
    if (most > 0) {
        const int64_t chunks = in_place ? 1 : (most + kThreads - 1) / kThreads;
        err = by_blocks<Move>(src.dim, src, dst, e, static_cast<unsigned>(chunks), in_place ? 1 : 0, stream);
        if (err != cudaSuccess) return err;
    }
    if (!same_lengths) return cudaSuccess;
    note_launch();
    return launch_pdl(kv_lengths_kernel, dim3((src.n_seqs + 127) / 128), dim3(128), 0, stream, src, e.lengths_out,
                      e.budget);
}

cudaError_t kv_error_word(int device, unsigned int** word) {
    static unsigned int* words[64];
    unsigned int* w = device < 64 ? __atomic_load_n(&words[device], __ATOMIC_ACQUIRE) : nullptr;
    if (!w) {
        void* p;
        const cudaError_t err = cudaGetSymbolAddress(&p, g_kv_error);
        if (err != cudaSuccess) return err;
        w = static_cast<unsigned int*>(p);
        if (device < 64) __atomic_store_n(&words[device], w, __ATOMIC_RELEASE);
    }
    *word = w;
    return cudaSuccess;
}

cudaError_t kv_read_device_error(unsigned int* bits, bool clear) {
    unsigned int v = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(v));
    if (err != cudaSuccess) return err;
    *bits |= v;
    if (clear && v) {
        const unsigned int zero = 0;
        err = cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(zero));
    }
    return err;
}

}  // namespace qm
