// Attention over the paged Q4_0 key/value cache, for any head dimension and
// any number of rows: the plain kernels.
#include <algorithm>

#include "kv_cache.cuh"

namespace qm {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
// Of the workspace's first 4 KB, zero between calls, the step kernel has all but
// the last 16 bytes; there is the number of the rows to be done again.
constexpr int64_t kRedoCount = kAttnZeroed - 16;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Value of dim 32 blk + lane of the token in `slot` of a cell.
__device__ __forceinline__ float cell_value(const uint8_t* cell, int dim, int slot, int blk, int lane) {
    const uint32_t byte = cell[blk * 256 + slot * 16 + (lane & 15)];
    const uint32_t q = lane < 16 ? (byte & 15u) : (byte >> 4);
    const float d = f16_bits_to_float(
        *reinterpret_cast<const uint16_t*>(cell + cell_scales(dim) + (slot * (dim >> 5) + blk) * 2));
    return magic_minus8(q | kMagicBits) * d;
}

// One row and query head (item = row * heads + head) by the `parts` warps of a
// CTA that call this with part = 0 .. parts - 1, or by one warp; lane l holds dims
// 32 i + l.  The softmax runs in one pass over the tokens with a running maximum
// and sum, in f32, four tokens at a time so that their loads overlap; the warps'
// sums meet in shared memory.
template <int NB, typename T, int kParts>
__device__ __forceinline__ void attn_plain_row(const KvView& c, const KvRows& r, const AttnCall& a, float* lse,
                                               int64_t item, int part) {
    const int lane = threadIdx.x & 31;
    const int row = static_cast<int>(item / a.heads), head = static_cast<int>(item % a.heads);
    const int b = kv_seq_of_row(r, c.n_seqs, row);
    if (b < 0) return;
    int first, count;
    kv_rows(r, b, &first, &count, c.err);
    if (row - first >= count) return;
    const int pos = kv_length(c, b, c.err) - count + (row - first);
    const int h = head / (a.heads / c.heads);
    const T* q = static_cast<const T*>(a.q) + row * a.q_stride + static_cast<int64_t>(head) * c.dim;
    float qv[NB], o[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        qv[i] = load1(q + 32 * i + lane) * (a.scale * kLog2e);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    // The tokens seen: 0 .. n_first - 1 and lo .. pos, numbered in a row.
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int n_first = a.window > 0 ? min(min(a.sinks, lo), pos + 1) : 0;
    const int n = n_first + max(0, pos - lo + 1);
    for (int x0 = 4 * part; x0 < n; x0 += 4 * kParts) {
        float s[4], v[4][NB];
        float top = m;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x = min(x0 + u, n - 1);
            const int j = x < n_first ? x : lo + (x - n_first);
            const int64_t off = kv_cell(c, b, h, j, c.err);
            s[u] = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                s[u] = off < 0 ? 0.f : fmaf(qv[i], cell_value(c.k + off, c.dim, j & 15, i, lane), s[u]);
                v[u][i] = off < 0 ? 0.f : cell_value(c.v + off, c.dim, j & 15, i, lane);
            }
        }
#pragma unroll
        for (int y = 16; y; y >>= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xFFFFFFFFu, s[u], y);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (x0 + u >= n) s[u] = -INFINITY;
            top = fmaxf(top, s[u]);
        }
        const float base = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(m - base);
        m = top;
        l *= keep;
#pragma unroll
        for (int i = 0; i < NB; ++i) o[i] *= keep;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float p = exp2f(s[u] - base);
            l += p;
            if (x0 + u < n) {
#pragma unroll
                for (int i = 0; i < NB; ++i) o[i] = fmaf(p, v[u][i], o[i]);
            }
        }
    }
    if constexpr (kParts > 1) {
        __shared__ float s_o[kParts][NB * 32], s_m[kParts], s_l[kParts];
#pragma unroll
        for (int i = 0; i < NB; ++i) s_o[part][32 * i + lane] = o[i];
        if (lane == 0) s_m[part] = m, s_l[part] = l;
        __syncthreads();
        m = -INFINITY;
        for (int y = 0; y < kParts; ++y) m = fmaxf(m, s_m[y]);
        const float base = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) o[i] = 0.f;
        for (int y = 0; y < kParts; ++y) {
            const float f = exp2f(s_m[y] - base);
            l = fmaf(f, s_l[y], l);
#pragma unroll
            for (int i = 0; i < NB; ++i) o[i] = fmaf(f, s_o[y][32 * i + lane], o[i]);
        }
        __syncthreads();
        if (part) return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + static_cast<int64_t>(head) * c.dim;
#pragma unroll
    for (int i = 0; i < NB; ++i) store1(out + 32 * i + lane, o[i] * inv);
    if (lane == 0) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (a.lse) a.lse[item] = lse2 * kLn2;
        if (lse) lse[item] = lse2;
    }
}

template <int NB, typename T>
__global__ void __launch_bounds__(kWarps * 32) attn_plain_kernel(KvView c, KvRows r, AttnCall a, float* lse) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (item < static_cast<int64_t>(r.n_tokens) * a.heads) attn_plain_row<NB, T, 1>(c, r, a, lse, item, 0);
}

// The rows that the prompt kernel listed in `redo` (redo_n[0] of them, but no more
// than there are rows; redo_n[1] counts CTAs), a CTA each; the last CTA to finish leaves the list empty for
// the next call.
constexpr int kRedoWarps = 8;
template <int NB, typename T>
__global__ void __launch_bounds__(kRedoWarps * 32)
    attn_redo_kernel(KvView c, KvRows r, AttnCall a, float* lse, unsigned* redo_n, const unsigned* redo) {
    grid_launch_dependents();
    grid_dependency_wait();
    const unsigned n = min(__ldcg(redo_n), static_cast<unsigned>(static_cast<int64_t>(r.n_tokens) * a.heads));
    for (unsigned i = blockIdx.x; i < n; i += gridDim.x)
        attn_plain_row<NB, T, kRedoWarps>(c, r, a, lse, __ldcg(redo + i), threadIdx.x >> 5);
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(redo_n + 1, 1u) == gridDim.x - 1) redo_n[0] = redo_n[1] = 0;
    }
}

// weights[b][h][j] += sum over the sequence's rows that see token j and the
// group's query heads of exp(scale q . k_j - lse).  One warp per token, so
// the sum has one owner and a fixed order.
template <int NB, typename T>
__global__ void __launch_bounds__(kWarps * 32) attn_weights_plain_kernel(KvView c, KvRows r, AttnCall a, const float* lse) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int j = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int h = blockIdx.y, b = blockIdx.z;
    const int L = kv_length(c, b, c.err);
    if (j >= L) return;
    int first, count;
    kv_rows(r, b, &first, &count, c.err);
    const int64_t off = kv_cell(c, b, h, j, c.err);
    if (off < 0) return;
    float k[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) k[i] = cell_value(c.k + off, c.dim, j & 15, i, lane) * (a.scale * kLog2e);
    const int group = a.heads / c.heads;
    float acc = 0.f;
    for (int i = max(0, j - (L - count)); i < count; ++i) {  // rows at positions >= j
        const int pos = L - count + i;
        if (a.window > 0 && j <= pos - a.window && j >= a.sinks) break;
        for (int g = 0; g < group; ++g) {
            const int head = h * group + g;
            const T* q = static_cast<const T*>(a.q) + (first + i) * a.q_stride + static_cast<int64_t>(head) * c.dim;
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < NB; ++x) s = fmaf(load1(q + 32 * x + lane), k[x], s);
#pragma unroll
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
            acc += exp2f(s - lse[static_cast<int64_t>(first + i) * a.heads + head]);
        }
    }
    if (lane == 0) {
        float* w = a.weights + (static_cast<int64_t>(b) * c.heads + h) * a.weights_stride + j;
        *w += acc;
    }
}

// The workspace of calls that the step kernel does not take: 4 KB that are zero
// between calls; the rows to be done again; with weights, logarithms to base 2
// and (head dimensions of the prompt kernel) the queries' tiles and units.
struct Room {
    int64_t redo = kAttnZeroed, lse = 0, units = 0, images = 0, bytes = 0, per_head = 0;
};
Room room_of(const KvView& c, int heads, int64_t n_tokens, bool weights) {
    Room m;
    const bool tiles = attn_prompt_takes(c);
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    m.lse = m.redo + (tiles ? up(n_tokens * heads * 4) : 0);
    m.units = m.lse + (weights ? up(n_tokens * heads * 4) : 0);
    m.per_head = query_tiles_per_head(n_tokens, heads / c.heads, c.n_seqs);
    m.images = m.units + (weights && tiles ? up(c.heads * m.per_head * 128 * 4) : 0);
    m.bytes = m.images + (weights && tiles ? c.heads * m.per_head * 128 * 4 * c.dim : 0);
    if (!tiles && !weights) m.bytes = 0;
    return m;
}

template <int NB, typename T>
cudaError_t launch_plain(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    const Room m = room_of(c, a.heads, r.n_tokens, a.weights != nullptr);
    float* lse = a.weights ? reinterpret_cast<float*>(a.ws + m.lse) : nullptr;  // to base 2
    cudaError_t err;
    if (attn_prompt_takes(c)) {
        unsigned* redo_n = reinterpret_cast<unsigned*>(a.ws + kRedoCount);
        unsigned* redo = reinterpret_cast<unsigned*>(a.ws + m.redo);
        const QueryTiles qt = {a.weights ? a.ws + m.images : nullptr, reinterpret_cast<float*>(a.ws + m.units), m.per_head};
        err = launch_attn_prompt(c, r, a, lse, qt, redo_n, redo, stream);
        if (err != cudaSuccess) return err;
        note_launch();
        err = launch_pdl(attn_redo_kernel<NB, T>, dim3(c.sms), dim3(kRedoWarps * 32), 0, stream, c, r, a, lse, redo_n,
                         static_cast<const unsigned*>(redo));
        if (err != cudaSuccess || !a.weights) return err;
        return launch_attn_weights(c, r, a, qt, lse, stream);
    }
    const int64_t items = static_cast<int64_t>(r.n_tokens) * a.heads;
    note_launch();
    err = launch_pdl(attn_plain_kernel<NB, T>, dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps)),
                     dim3(kWarps * 32), 0, stream, c, r, a, lse);
    if (err != cudaSuccess || !a.weights || c.max_len == 0) return err;
    note_launch();
    return launch_pdl(attn_weights_plain_kernel<NB, T>,
                      dim3(static_cast<unsigned>((c.max_len + kWarps - 1) / kWarps), c.heads, c.n_seqs),
                      dim3(kWarps * 32), 0, stream, c, r, a, lse);
}

template <int NB>
cudaError_t launch_plain(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    return a.type == KvType::kF32 ? launch_plain<NB, float>(c, r, a, stream)
                                  : launch_plain<NB, __nv_bfloat16>(c, r, a, stream);
}

}  // namespace

int64_t attn_workspace_bytes(const KvView& c, int heads, int64_t n_tokens, int64_t max_q, bool weights) {
    if (attn_step_takes(c, heads, max_q)) return attn_step_workspace(c, heads, n_tokens, max_q, weights);
    return room_of(c, heads, n_tokens, weights).bytes;
}

int64_t attn_workspace_most(const KvView& c, int heads, int64_t n_tokens, int64_t max_q, bool weights) {
    // Both kernels' needs grow with the rows and with weights; the step kernel takes calls up to a number of rows.
    const int64_t step = attn_step_most(c, heads, max_q);
    int64_t most = step > 0 ? attn_step_workspace(c, heads, n_tokens, step, weights) : 0;
    if (step < max_q) most = std::max(most, room_of(c, heads, n_tokens, weights).bytes);
    return most;
}

cudaError_t launch_attn(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    if (attn_step_takes(c, a.heads, r.max_q)) return launch_attn_step(c, r, a, stream);
    switch (c.dim / 32) {
        case 1: return launch_plain<1>(c, r, a, stream);
        case 2: return launch_plain<2>(c, r, a, stream);
        case 3: return launch_plain<3>(c, r, a, stream);
        case 4: return launch_plain<4>(c, r, a, stream);
        case 5: return launch_plain<5>(c, r, a, stream);
        case 6: return launch_plain<6>(c, r, a, stream);
        case 7: return launch_plain<7>(c, r, a, stream);
        default: return launch_plain<8>(c, r, a, stream);
    }
}

}  // namespace qm
