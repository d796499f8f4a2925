// The paged Q4_0 key/value cache: quantizing rows into it, reading them back,
// and cutting it back to the tokens that collected the most attention.
#include <algorithm>

#include "kv_cache.cuh"

namespace qm {

__device__ unsigned int g_kv_error = 0;

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

// Q4_0 quantization of a block of 32 by 8 lanes of 4 elements each: m = the
// first element of largest magnitude, d = m / -8, r = 1 / d (both correctly
// rounded f32 divisions), q = min(15, floor(x r + 8.5)) with the product and
// the sum each rounded to f32; the stored scale is d narrowed to binary16.
// With m mapped to q = 0 the other sign gets only 7 steps: taking the signed
// maximum gives the larger side the extra one.  NaN elements do not raise the
// maximum; q = 8 (the value 0) where x r is NaN or d is 0.
// Returns the four quants as bytes (element 4 i + e in byte e); *scale = d's bits.
__device__ __forceinline__ uint32_t quantize_q4_lane(float4 x4, int i, uint32_t* scale) {
    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    // Sign of the first element of that magnitude: the smallest 2 * index + sign.
    uint32_t at = 0x7FFFFFFFu;
#pragma unroll
    for (int e = 3; e >= 0; --e)
        if (fabsf(x[e]) == amax) at = 2u * (4 * i + e) + (__float_as_uint(x[e]) >> 31);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) at = min(at, __shfl_xor_sync(0xFFFFFFFFu, at, o));
    const float m = (at & 1u) ? -amax : amax;
    const float d = __fdiv_rn(m, -8.f);
    const float r = d == 0.f ? 0.f : __frcp_rn(d);
    *scale = f16_bits_rn(d);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float t = floorf(__fadd_rn(__fmul_rn(x[e], r), 8.5f));
        const uint32_t q = isnan(t) ? 8u : static_cast<uint32_t>(fminf(fmaxf(t, 0.f), 15.f));
        w |= q << (8 * e);
    }
    return w;
}

// One lane per 4 elements of a key or value row, 8 lanes per block; the lanes
// of a warp run over the blocks of a row, then the kv heads, then K and V.
// Memory-bound: 4 (or 2) bytes read and 9/16 written per element.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(KvView c, KvRows r, const T* k, const T* v, int64_t k_stride, int64_t v_stride, int64_t n4) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const bool in = t < n4;  // n4 is a multiple of 8: whole blocks
    const int per_row = c.heads * c.dim / 4;  // lanes of one token's K (or V)
    const int64_t tt = in ? t : 0;
    const int row = static_cast<int>(tt / (2 * per_row));
    int rest = static_cast<int>(tt - static_cast<int64_t>(row) * 2 * per_row);
    const bool is_v = rest >= per_row;
    if (is_v) rest -= per_row;
    const T* src = (is_v ? v + row * v_stride : k + row * k_stride) + 4 * rest;
    const float4 x = in ? load4(src) : make_float4(0.f, 0.f, 0.f, 0.f);
    uint32_t scale;
    const int i = threadIdx.x & 7;
    uint32_t w = quantize_q4_lane(x, i, &scale);
    w |= __shfl_down_sync(0xFFFFFFFFu, w, 4) << 4;  // lanes 0..3 of a block: low nibbles, 4..7: high
    if (!in) return;
    const int b = kv_seq_of_row(r, c.n_seqs, row);
    if (b < 0) return;
    int first, count;
    kv_rows(r, b, &first, &count, &g_kv_error);
    const int pos = kv_length(c, b, &g_kv_error) - count + (row - first);
    if (row - first >= count || pos < 0) {
        atomicOr(&g_kv_error, kErrRange);
        return;
    }
    const int h = rest * 4 / c.dim;
    const int blk = (rest * 4 - h * c.dim) >> 5;
    const int64_t off = kv_cell(c, b, h, pos, &g_kv_error);
    if (off < 0) return;
    uint8_t* cell = (is_v ? c.v : c.k) + off;
    const int slot = pos & 15;
    if (i < 4) *reinterpret_cast<uint32_t*>(cell + blk * 256 + slot * 16 + 4 * i) = w;
    if (i == 4)
        *reinterpret_cast<uint16_t*>(cell + cell_scales(c.dim) + (slot * (c.dim >> 5) + blk) * 2) =
            static_cast<uint16_t>(scale);
}

// The inverse: f32 values of the call's rows, contiguous [n_tokens][heads][dim].
__global__ void __launch_bounds__(kThreads)
    kv_read_kernel(KvView c, KvRows r, float* k, float* v, int64_t n4) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= n4) return;
    const int per_row = c.heads * c.dim / 4;
    const int row = static_cast<int>(t / (2 * per_row));
    int rest = static_cast<int>(t - static_cast<int64_t>(row) * 2 * per_row);
    const bool is_v = rest >= per_row;
    if (is_v) rest -= per_row;
    const int b = kv_seq_of_row(r, c.n_seqs, row);
    if (b < 0) return;
    int first, count;
    kv_rows(r, b, &first, &count, &g_kv_error);
    const int pos = kv_length(c, b, &g_kv_error) - count + (row - first);
    const int h = rest * 4 / c.dim;
    const int blk = (rest * 4 - h * c.dim) >> 5;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    int64_t off = -1;
    if (row - first < count && pos >= 0) off = kv_cell(c, b, h, pos, &g_kv_error);
    else atomicOr(&g_kv_error, kErrRange);
    if (off >= 0) {
        const uint8_t* cell = (is_v ? c.v : c.k) + off;
        const int slot = pos & 15;
        const int i = rest & 7;
        uint32_t w = *reinterpret_cast<const uint32_t*>(cell + blk * 256 + slot * 16 + 4 * (i & 3));
        if (i >= 4) w >>= 4;
        const float d = f16_bits_to_float(*reinterpret_cast<const uint16_t*>(
            cell + cell_scales(c.dim) + (slot * (c.dim >> 5) + blk) * 2));
        x.x = magic_minus8((w & 15u) | kMagicBits) * d;
        x.y = magic_minus8(((w >> 8) & 15u) | kMagicBits) * d;
        x.z = magic_minus8(((w >> 16) & 15u) | kMagicBits) * d;
        x.w = magic_minus8(((w >> 24) & 15u) | kMagicBits) * d;
    }
    float* dst = (is_v ? v : k) + static_cast<int64_t>(row) * per_row * 4 + 4 * rest;
    *reinterpret_cast<float4*>(dst) = x;
}

// ---- eviction --------------------------------------------------------------

constexpr int kSelThreads = 1024;

// Unsigned order of a score: larger score, larger key; NaN below everything.
__device__ __forceinline__ uint32_t score_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, kv head): finds the smallest kept key by a radix
// select (four passes of 8 bits over the scores), then writes the kept tokens
// in ascending order with a block-wide scan per 1024 tokens.
__global__ void __launch_bounds__(kSelThreads)
    kv_select_kernel(KvView c, EvictCall e) {
    grid_launch_dependents();
    grid_dependency_wait();
    __shared__ unsigned hist[256];
    __shared__ unsigned warp_n[2][32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = kv_length(c, b, &g_kv_error);
    const float* w = e.weights + (static_cast<int64_t>(b) * c.heads + h) * e.weights_stride;
    float* wo = e.weights_out + (static_cast<int64_t>(b) * c.heads + h) * e.out_stride;
    int32_t* kept = e.kept + (static_cast<int64_t>(b) * c.heads + h) * e.budget;
    const int n_keep = min(L, e.budget);
    const int lo = min(e.sinks, L);             // tokens below lo and from hi on stay
    const int hi = max(lo, L - e.recent);
    const int need0 = n_keep - lo - (L - hi);   // of the tokens between
    uint32_t prefix = 0;
    int need = need0;
    const bool all = L <= e.budget;
    if (!all && need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                const uint32_t key = score_key(w[j]);
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                int left = need;
                int bin = 255;
                while (bin > 0 && static_cast<int>(hist[bin]) < left) left -= hist[bin--];
                s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
                s_need = left;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
    }
    // Keys above `prefix` are kept, and the first `need` equal to it.
    int base_keep = 0, base_tie = 0;
    for (int j0 = 0; j0 < L; j0 += kSelThreads) {
        const int j = j0 + tid;
        float score = 0.f;
        bool keep = false, tie = false;
        if (j < L) {
            score = w[j];
            if (all || j < lo || j >= hi) keep = true;
            else if (need0 > 0) {
                const uint32_t key = score_key(score);
                keep = key > prefix;
                tie = key == prefix;
            }
        }
        const unsigned tb = __ballot_sync(0xFFFFFFFFu, tie);
        if (lane == 0) warp_n[0][warp] = __popc(tb);
        __syncthreads();
        int before = base_tie, total_tie = 0;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) before += warp_n[0][i];
            total_tie += warp_n[0][i];
        }
        if (tie && before + __popc(tb & ((1u << lane) - 1u)) < need) keep = true;
        const unsigned kb = __ballot_sync(0xFFFFFFFFu, keep);
        if (lane == 0) warp_n[1][warp] = __popc(kb);
        __syncthreads();
        int at = base_keep, total_keep = 0;
        for (int i = 0; i < 32; ++i) {
            if (i < warp) at += warp_n[1][i];
            total_keep += warp_n[1][i];
        }
        at += __popc(kb & ((1u << lane) - 1u));
        // In place (weights_out == weights): at <= j, and every thread of the
        // CTA has read its score of this chunk before the barriers above.
        if (keep && at < n_keep) {
            kept[at] = j;
            wo[at] = score;
        }
        base_keep += total_keep;
        base_tie += total_tie;
        __syncthreads();
    }
    for (int i = n_keep + tid; i < e.budget; i += kSelThreads) {
        kept[i] = -1;
        wo[i] = 0.f;
    }
}

// Copies the kept tokens' quants and scales to the first places of dst.
// Thread: one 16-byte quant row of a token (or its scales); a CTA takes
// `cells` destination cells.  With in_place one CTA walks all of them: a kept
// token never moves up, so reading a batch before writing it is enough.
__global__ void __launch_bounds__(kThreads)
    kv_move_kernel(KvView src, KvView dst, const int32_t* kept_all, int budget, int cells, int in_place) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int h = blockIdx.y % src.heads;
    const bool is_v = blockIdx.y >= static_cast<unsigned>(src.heads);
    const int b = blockIdx.z;
    const int32_t* kept = kept_all + (static_cast<int64_t>(b) * src.heads + h) * budget;
    const int n_keep = min(kv_length(src, b, &g_kv_error), budget);
    const int pieces = src.dim / 32 + 1;  // quant rows of a token, then its scales
    const int per_cell = kCellTokens * pieces;
    const uint8_t* from = is_v ? src.v : src.k;
    uint8_t* to = is_v ? dst.v : dst.k;
    const int n_cells = (n_keep + kCellTokens - 1) / kCellTokens;
    const int end = in_place ? n_cells : min(n_cells, static_cast<int>(blockIdx.x + 1) * cells);
    const int step = kThreads / kCellTokens;  // (cell, piece) pairs per pass
    const int first = in_place ? 0 : blockIdx.x * cells;
    for (int p0 = first * pieces; p0 < end * pieces; p0 += step) {
        const int p = p0 + threadIdx.x / kCellTokens;
        const int cell = p / pieces, piece = p - cell * pieces;
        const int slot = threadIdx.x & 15;
        const int at = cell * kCellTokens + slot;
        uint4 x = make_uint4(0, 0, 0, 0);
        const uint8_t* s = nullptr;
        uint8_t* d = nullptr;
        if (cell < end && at < n_keep) {
            const int token = kept[at];
            const int64_t so = kv_cell(src, b, h, token, &g_kv_error);
            const int64_t dd = kv_cell(dst, b, h, at, &g_kv_error);
            if (so >= 0 && dd >= 0) {
                s = from + so;
                d = to + dd;
                if (piece < src.dim / 32) {
                    x = *reinterpret_cast<const uint4*>(s + piece * 256 + (token & 15) * 16);
                } else {
                    const int nb = src.dim / 32;
                    const uint16_t* sc = reinterpret_cast<const uint16_t*>(s + cell_scales(src.dim)) + (token & 15) * nb;
                    uint16_t hsc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    for (int i = 0; i < nb; ++i) hsc[i] = sc[i];
                    x = make_uint4(hsc[0] | (hsc[1] << 16), hsc[2] | (hsc[3] << 16), hsc[4] | (hsc[5] << 16),
                                   hsc[6] | (hsc[7] << 16));
                }
            }
        }
        if (in_place) __syncthreads();
        if (d) {
            if (piece < src.dim / 32) {
                *reinterpret_cast<uint4*>(d + piece * 256 + slot * 16) = x;
            } else {
                const int nb = src.dim / 32;
                uint16_t* sc = reinterpret_cast<uint16_t*>(d + cell_scales(src.dim)) + slot * nb;
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                for (int i = 0; i < nb; ++i) sc[i] = static_cast<uint16_t>(xs[i >> 1] >> (16 * (i & 1)));
            }
        }
        if (in_place) __syncthreads();
    }
}

__global__ void kv_lengths_kernel(KvView src, int32_t* out, int budget) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < src.n_seqs) out[b] = min(kv_length(src, b, &g_kv_error), budget);
}

}  // namespace

cudaError_t launch_kv_append(const KvView& c, const KvRows& r, const void* k, const void* v, KvType type,
                             int64_t k_stride, int64_t v_stride, cudaStream_t stream) {
    const int64_t n4 = static_cast<int64_t>(r.n_tokens) * 2 * c.heads * (c.dim / 4);
    const dim3 grid(static_cast<unsigned>((n4 + kThreads - 1) / kThreads));
    note_launch();
    if (type == KvType::kF32)
        return launch_pdl(kv_append_kernel<float>, grid, dim3(kThreads), 0, stream, c, r, static_cast<const float*>(k),
                          static_cast<const float*>(v), k_stride, v_stride, n4);
    return launch_pdl(kv_append_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, c, r,
                      static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), k_stride, v_stride,
                      n4);
}

cudaError_t launch_kv_read(const KvView& c, const KvRows& r, float* k, float* v, cudaStream_t stream) {
    const int64_t n4 = static_cast<int64_t>(r.n_tokens) * 2 * c.heads * (c.dim / 4);
    note_launch();
    return launch_pdl(kv_read_kernel, dim3(static_cast<unsigned>((n4 + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                      stream, c, r, k, v, n4);
}

cudaError_t launch_kv_evict(const KvView& src, const KvView& dst, const EvictCall& e, cudaStream_t stream,
                            const DeviceInfo& /*dev*/) {
    note_launch();
    cudaError_t err = launch_pdl(kv_select_kernel, dim3(src.heads, src.n_seqs), dim3(kSelThreads), 0, stream, src, e);
    if (err != cudaSuccess) return err;
    const bool in_place = src.table == dst.table && src.k == dst.k;
    const int64_t most = std::min<int64_t>(e.budget, src.max_len);
    const int cells = 8;
    const int64_t chunks = in_place ? 1 : (most + cells * kCellTokens - 1) / (cells * kCellTokens);
    if (most > 0) {
        note_launch();
        err = launch_pdl(kv_move_kernel, dim3(static_cast<unsigned>(chunks), 2 * src.heads, src.n_seqs), dim3(kThreads),
                         0, stream, src, dst, e.kept, e.budget, cells, in_place ? 1 : 0);
        if (err != cudaSuccess) return err;
    }
    note_launch();
    return launch_pdl(kv_lengths_kernel, dim3((src.n_seqs + 127) / 128), dim3(128), 0, stream, src, e.lengths_out,
                      e.budget);
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
