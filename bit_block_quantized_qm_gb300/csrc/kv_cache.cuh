// The paged Q4_0 key/value cache as the kernels see it: layout of cells and
// pages, the rows of a call, and bounds-checked look-ups.  Everything is read by
// plain loads: a kernel may start while the one before it still writes lengths,
// tables or cells, and read-only loads want memory that nothing writes as long as
// the kernel lives.
#pragma once

#include "qm_device.cuh"
#include "qm_internal.h"

namespace qm {

// A cell holds 16 tokens of one kv head: [D/32][16 tokens][16 quant bytes],
// then [16 tokens][D/32] f16 scales.  Eight tokens' quants of one block are
// 128 consecutive bytes, which is what ldmatrix reads without bank conflicts,
// and a token's scales are one aligned word or two.
constexpr int kCellTokens = 16;
__host__ __device__ constexpr int cell_bytes(int D) { return 9 * D; }
__host__ __device__ constexpr int cell_scales(int D) { return 8 * D; }  // offset of the scales

// Tokens in the cache of sequence b, and what is wrong with the number.
__device__ __forceinline__ int kv_length(const KvView& c, int b, unsigned int* err) {
    const int n = c.lengths[b];
    if (n < 0 || n > c.max_len) {
        atomicOr(err, kErrRange);
        return n < 0 ? 0 : static_cast<int>(c.max_len);
    }
    return n;
}

// First row and number of rows of sequence b in this call.
__device__ __forceinline__ void kv_rows(const KvRows& r, int b, int* first, int* count, unsigned int* err) {
    if (!r.starts) {
        *first = b * r.uniform;
        *count = r.uniform;
        return;
    }
    int a = r.starts[b], e = r.starts[b + 1];
    if (a < 0 || e < a || e > r.n_tokens || e - a > r.max_q) {
        atomicOr(err, kErrRange);
        a = min(max(a, 0), r.n_tokens);
        e = a + min(min(max(e, a), r.n_tokens) - a, r.max_q);
    }
    *first = a;
    *count = e - a;
}

// The page that holds token `pos` of sequence b; -1 past the page table.
__device__ __forceinline__ int kv_page_id(const KvView& c, int b, int pos) {
    const int page = pos >> c.page_shift;
    return page < c.table_stride ? c.table[b * c.table_stride + page] : -1;
}
// Byte offset in the pool of the cell that holds token `pos` of a sequence, in page
// `id`, of kv head h; -1 (and the error bit) where `id` is no page.
__device__ __forceinline__ int64_t kv_cell_in(const KvView& c, int id, int h, int pos, unsigned int* err) {
    if (id < 0 || id >= c.n_pages) {
        atomicOr(err, kErrRange);
        return -1;
    }
    const int cells = 1 << (c.page_shift - 4);
    return ((static_cast<int64_t>(id) * c.heads + h) * cells + ((pos >> 4) & (cells - 1))) * cell_bytes(c.dim);
}
__device__ __forceinline__ int64_t kv_cell(const KvView& c, int b, int h, int pos, unsigned int* err) {
    return kv_cell_in(c, kv_page_id(c, b, pos), h, pos, err);
}

// The sequence that row `row` belongs to, or -1.
__device__ __forceinline__ int kv_seq_of_row(const KvRows& r, int n_seqs, int row) {
    if (!r.starts) return row / r.uniform;
    int lo = 0, hi = n_seqs;  // the last b with starts[b] <= row
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (r.starts[mid + 1] <= row) lo = mid + 1;
        else hi = mid;
    }
    return lo < n_seqs && r.starts[lo] <= row ? lo : -1;
}

// Tiles of kTokens tokens that rows at positions pos_lo and up read of seen_len
// tokens: all, or the first ones' and those from the window's lower end on.
struct TileList {
    int n1;  // tiles 0 .. n1 - 1, then
    int t2;  // tiles t2 ..
    int count;
    __device__ __forceinline__ int at(int i) const { return i < n1 ? i : t2 + (i - n1); }
};
template <int kTokens>
__device__ __forceinline__ TileList tile_list(int seen_len, int pos_lo, int window, int sinks) {
    const int total = (seen_len + kTokens - 1) / kTokens;
    TileList t{0, 0, total};
    if (window > 0) {
        const int lo = max(0, pos_lo - window + 1);
        t.n1 = min((min(sinks, lo) + kTokens - 1) / kTokens, total);
        t.t2 = max(t.n1, lo / kTokens);
        t.count = t.n1 + max(0, total - t.t2);
    }
    return t;
}

// Four elements of a row, 16-byte (bf16: 8-byte) aligned.
__device__ __forceinline__ float4 load_q4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load_q4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store_o4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store_o4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^e for e in -126 .. 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace qm
