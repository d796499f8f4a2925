// Attention of few rows over the paged Q4_0 cache: the step of a decoder
// (single tokens, drafts of a few), where every byte of the cache is read for
// a handful of query rows.
//
// Mathematics.  Both products run on tensor cores (mma.sync m16n8k16, f16 in,
// f32 out) on the *quants themselves*, n - 8 as exact f16 numbers.  (A nibble is
// an f16 subnormal as it stands, but the tensor cores align products by their
// exponents, and a subnormal's is up to 10 bits above its value: that cost
// errors of 2^-17.)
//   scores  s_j = sum_b d_jb sum_i q_i (n_ji - 8): tokens are the 16 rows, query
//     rows the 8 columns; each query row takes two columns, its values rounded
//     to f16 and what that leaves (22 bits together), scaled by a power of two
//     to the top of f16's range; each block of 32 is scaled by d_jb in f32.
//   output  o = sum_j (p_j d_jb) (n_j - 8): dims are the rows, query rows again
//     two columns each, p_j d_jb as f16 and the exact f16 remainder (two packed
//     FMAs per two tokens).  p is scaled by 2^15, or less where the largest
//     scale seen would take p d out of f16's range (then the sums follow).
// The softmax runs in one pass with a running maximum and sum in f32.
//
// Bytes bound it: 9 D / 8 per token and kv head.  A tensor-core product covers
// 256 quants = 144 bytes, which HBM delivers in 6 cycles per SM; unpacking on
// the FP32 pipe alone (one FMA per quant and query row) would need 3 times
// that at four rows.
//
// Split.  A CTA of four warps takes one (sequence, kv head, 4 or 8 rows) and a
// range of 64-token tiles; each warp runs its own tiles through its own
// two-stage ring, filled with bulk copies (a cell is contiguous, a page is
// too), and meets the others once at the end.  Ranges of one sequence meet in
// the workspace: the last CTA to arrive adds them up in range order, so the
// result does not depend on which one that is.
#include <algorithm>

#include "kv_cache.cuh"

namespace qm {

__device__ unsigned int g_attn_step_error = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;  // tokens of a warp's tile
constexpr int kStages = 2;
constexpr float kTiny = 0x1p-23f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct StepPlan {
    int tiles_per_cta;  // of one range
    int splits;         // ranges at most
    int groups;         // row groups
    int pad_len;        // tokens per row of the stashed scores (0: none)
    int64_t part_off, stash_off, lse_off, bytes;  // offsets in the workspace
};

// The workspace begins with arrival counters, zero between calls: 4 KB of it
// are never anything else, whatever calls share the workspace.  Ranges are cut
// only where there are at most kTargetCtas / 2 of (sequence, kv head, rows).
constexpr int kTargetCtas = 152 * 3 * 4;
constexpr int64_t kCtrBytes = 4096;
static_assert(kTargetCtas / 2 * 4 <= kCtrBytes, "a counter for each");

// Tiles that rows at positions pos0 .. L - 1 read: all of 0 .. L - 1, or the
// first ones' and those from the window's lower end on.
struct TileList {
    int n1;     // tiles 0 .. n1 - 1, then
    int t2;     // tiles t2 ..
    int count;
    __device__ __forceinline__ int at(int i) const { return i < n1 ? i : t2 + (i - n1); }
};
__device__ __forceinline__ TileList tile_list(int L, int pos0, int window, int sinks) {
    const int total = (L + kTile - 1) / kTile;
    TileList t{0, 0, total};
    if (window > 0) {
        const int lo = max(0, pos0 - window + 1);
        t.n1 = min((min(sinks, lo) + kTile - 1) / kTile, total);
        t.t2 = max(t.n1, lo / kTile);
        t.count = t.n1 + max(0, total - t.t2);
    }
    return t;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {  // lo in bits 0..15
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

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

// N consecutive 32-bit words, aligned to all of them (N = 1, 2 or 4).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t w[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
}

// n - 8 as f16 pairs for the low nibbles n of bytes 0 and 2 of w, and for their
// high nibbles: OR-ed into the mantissa of 1024 a nibble reads 1024 + n (or
// 1024 + 16 n), and one packed operation, exact, takes the rest away.
__device__ __forceinline__ uint32_t minus8_low(uint32_t w) {
    return as_word(__hadd2(as_half2((w & 0x000F000Fu) | 0x64006400u), as_half2(0xE408E408u)));  // - 1032
}
__device__ __forceinline__ uint32_t minus8_high(uint32_t w) {
    return as_word(__hfma2(as_half2((w & 0x00F000F0u) | 0x64006400u), as_half2(0x2C002C00u),  // / 16
                           as_half2(0xD480D480u)));                                            // - 72
}

// 2^e for e in -126 .. 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

template <int D, int NT>
struct StepShape {
    static constexpr int kBlocks = D / 32;
    static constexpr int kRows = 4 * NT;                // query rows of a CTA
    static constexpr int kHalf = (kTile / 16) * 9 * D;  // bytes of a tile's keys (or values)
    static constexpr int kRing = kStages * 2 * kHalf;   // of one warp
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kRows * D * 4 + 2 * kRows * 4 <= kRing, "a warp's sums fit in its ring");
};

template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    attn_step_kernel(KvView c, KvRows r, AttnCall a, StepPlan plan) {
    using S = StepShape<D, NT>;
    constexpr int NB = S::kBlocks;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ int s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    if (threadIdx.x < kWarps * kStages) mbar_init(&bars[0][0] + threadIdx.x, 1);
    fence_barrier_init();
    __syncthreads();
    grid_launch_dependents();
    grid_dependency_wait();

    const int split = blockIdx.x % plan.splits, rg = blockIdx.x / plan.splits;
    const int h = blockIdx.y, b = blockIdx.z;
    int first, count;
    kv_rows(r, b, &first, &count, &g_attn_step_error);
    const int L = kv_length(c, b, &g_attn_step_error);
    const int group = a.heads / c.heads;
    const int n_rows = count * group;  // rows of this (sequence, kv head): token-major, then query head
    const int row0 = rg * S::kRows;
    if (row0 >= n_rows) return;
    const int base_pos = L - count;  // position of the sequence's first row (may be negative)
    const int pos_lo = base_pos + row0 / group;
    const int pos_hi = base_pos + min(n_rows - 1, row0 + S::kRows - 1) / group;
    const int seen_len = max(0, min(L, pos_hi + 1));
    const TileList tiles = tile_list(seen_len, max(pos_lo, 0), a.window, a.sinks);
    const int n_splits = max(1, (tiles.count + plan.tiles_per_cta - 1) / plan.tiles_per_cta);
    if (split >= n_splits) return;
    const int tile_end = min(tiles.count, (split + 1) * plan.tiles_per_cta);

    // This thread's query row in score and output accumulators is 4 j + t; in
    // the operands it feeds it is 4 j + g / 2, piece g % 2.
    uint32_t bq[NT][NB][4];
    float to_log2[NT];  // accumulated score -> logarithm to base 2
    int pos[NT];        // position of row 4 j + t; -1: no such row
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int rr = row0 + 4 * j + (g >> 1);
        const bool in = rr < n_rows;
        const int head = h * group + (in ? rr % group : 0);
        const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(first + (in ? rr / group : 0)) * a.q_stride +
                     static_cast<int64_t>(head) * D;
        float4 x[NB][2];
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[k][u] = in ? load_q4(q + 32 * k + 16 * u + 4 * t) : make_float4(0.f, 0.f, 0.f, 0.f);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[k][u].x), fabsf(x[k][u].y)),
                                         fmaxf(fabsf(x[k][u].z), fabsf(x[k][u].w))));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        // Powers of two that take the row's largest value to 2^13 .. 2^14.
        const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // -127 for 0 and subnormals
        const int up = min(126, 13 - ex);
        const float f = pow2(up);
        to_log2[j] = a.scale * kLog2e * pow2(-up);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float v[4] = {x[k][u].x * f, x[k][u].y * f, x[k][u].z * f, x[k][u].w * f};
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float hi = __half2float(__float2half_rn(v[e]));
                    w[e] = (g & 1) ? v[e] - hi : hi;
                }
                bq[j][k][2 * u] = pack_f16(w[0], w[2]);
                bq[j][k][2 * u + 1] = pack_f16(w[1], w[3]);
            }
        }
        to_log2[j] = __shfl_sync(0xFFFFFFFFu, to_log2[j], 8 * t);
        const int mine = row0 + 4 * j + t;
        pos[j] = mine < n_rows ? base_pos + mine / group : -1;
    }

    uint8_t* my_ring = ring + warp * S::kRing;
    // Lanes 0..7 copy a tile: keys' cells 0..3, then values'.  Where a page
    // holds a tile, one copy takes all four cells.
    const bool whole = c.page_shift >= 6;
    auto source = [&](int i) -> int64_t {  // byte offset of this lane's part of tile i, -1: nothing to copy
        if (lane >= 8 || i >= tile_end) return -1;
        const int cell = lane & 3;
        const int p = tiles.at(i) * kTile + cell * 16;
        if (p >= seen_len || (whole && cell)) return -1;
        return kv_cell(c, b, h, p, &g_attn_step_error);
    };
    auto issue = [&](int i, int stage, int64_t off) {
        const int left = seen_len - tiles.at(i) * kTile;
        const int cells = whole ? min(4, (left + 15) >> 4) : 1;
        const uint32_t bytes = off >= 0 ? static_cast<uint32_t>(cells * cell_bytes(D)) : 0u;
        const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, bytes);
        if (lane == 0) mbar_arrive_expect_tx(&bars[warp][stage], total);
        __syncwarp();
        if (off >= 0) {
            uint8_t* dst = my_ring + stage * 2 * S::kHalf + (lane >> 2) * S::kHalf + (lane & 3) * cell_bytes(D);
            bulk_load_1d(dst, ((lane & 4) ? c.v : c.k) + off, bytes, &bars[warp][stage]);
        }
    };

    float m[NT], l[NT];
    float o[NT][NB][2][4];  // [low, high nibbles][accumulator]
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        m[j] = -INFINITY;
        l[j] = 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][k][0][e] = o[j][k][1][e] = 0.f;
    }
    int v_up = 15;  // p is scaled by 2^v_up

    const int tile_first = split * plan.tiles_per_cta + warp;
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
        const int i = tile_first + s * kWarps;
        if (i < tile_end) issue(i, s, source(i));
    }
    int64_t off_next = source(tile_first + kStages * kWarps);  // looked up a tile ahead

    int n = 0, i = tile_first;
    bool ok = true;
    for (; i < tile_end; i += kWarps, ++n) {
        const int stage = n % kStages;
        const uint8_t* kt = my_ring + stage * 2 * S::kHalf;
        uint8_t* vt = my_ring + stage * 2 * S::kHalf + S::kHalf;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bars[warp][stage], (n / kStages) & 1, &g_attn_step_error));
        if (!ok) break;
        const int key0 = tiles.at(i) * kTile;

        // The largest scale of the values; tokens past the end do not count.
        uint32_t bad0 = 0, bad1 = 0;  // tokens with a scale that is not finite
        {
            uint32_t top = 0;
            bool odd = false;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = u * 32 + lane;
                uint8_t* sc = vt + (key >> 4) * cell_bytes(D) + cell_scales(D) + (key & 15) * 2 * NB;
                uint32_t w[NB / 2];
                load_words<NB / 2>(sc, w);
                uint32_t mx = w[0] & 0x7FFF7FFFu;
#pragma unroll
                for (int e = 1; e < NB / 2; ++e) mx = __vmaxu2(mx, w[e] & 0x7FFF7FFFu);
                mx = max(mx & 0xFFFFu, mx >> 16);
                const bool past = key0 + key >= seen_len;
                const bool wild = !past && mx >= 0x7C00u;
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, wild);
                if (u == 0) bad0 = bits;
                else bad1 = bits;
                if (past || wild) {
#pragma unroll
                    for (int e = 0; e < NB / 2; ++e) reinterpret_cast<uint32_t*>(sc)[e] = 0u;
                    odd = true;
                    mx = 0;
                }
                top = max(top, mx);
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (__any_sync(0xFFFFFFFFu, odd)) __syncwarp();
            // 2^v_up d <= 2^15 for d < 2^(exponent + 1).
            const int need = min(15, 14 - (static_cast<int>(top >> 10) - 15));
            if (need < v_up) {
                const float down = pow2(need - v_up);
                v_up = need;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int k = 0; k < NB; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            o[j][k][0][e] *= down;
                            o[j][k][1][e] *= down;
                        }
            }
        }

        // Scores of the tile: s[cell][j][0]: token 16 cell + g, [1]: + 8.
        float s[4][NT][2];
#pragma unroll
        for (int cell = 0; cell < 4; ++cell) {
            const uint8_t* cp = kt + cell * cell_bytes(D);
            uint32_t d0[NB / 2], d1[NB / 2];
            load_words<NB / 2>(cp + cell_scales(D) + g * 2 * NB, d0);
            load_words<NB / 2>(cp + cell_scales(D) + (g + 8) * 2 * NB, d1);
#pragma unroll
            for (int j = 0; j < NT; ++j) s[cell][j][0] = s[cell][j][1] = 0.f;
#pragma unroll
            for (int k2 = 0; k2 < NB; k2 += 2) {
                uint32_t w[4];
                ldmatrix_x4(smem_addr(cp) + k2 * 256 + lane * 16, w);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int k = k2 + u;
                    const uint32_t w0 = w[2 * u], w1 = w[2 * u + 1];
                    const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
                    const uint32_t l0 = minus8_low(w0), l1 = minus8_low(w1), l2 = minus8_low(y0), l3 = minus8_low(y1);
                    const uint32_t h0 = minus8_high(w0), h1 = minus8_high(w1), h2 = minus8_high(y0),
                                   h3 = minus8_high(y1);
                    const float2 dd0 = __half22float2(as_half2(d0[k2 / 2]));
                    const float2 dd1 = __half22float2(as_half2(d1[k2 / 2]));
                    const float e0 = u ? dd0.y : dd0.x, e1 = u ? dd1.y : dd1.x;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_f16(acc, l0, l1, l2, l3, bq[j][k][0], bq[j][k][1]);
                        mma_f16(acc, h0, h1, h2, h3, bq[j][k][2], bq[j][k][3]);
                        s[cell][j][0] = fmaf(e0, acc[0] + acc[1], s[cell][j][0]);
                        s[cell][j][1] = fmaf(e1, acc[2] + acc[3], s[cell][j][1]);
                    }
                }
            }
        }

        // To base 2, masked where some row does not see some token.
        const bool all_seen = key0 + kTile <= min(pos_lo + 1, L) && !(bad0 | bad1) &&
                              (a.window == 0 || key0 > pos_hi - a.window || key0 + kTile <= a.sinks);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float mx = -INFINITY;
#pragma unroll
            for (int cell = 0; cell < 4; ++cell) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = s[cell][j][e] * to_log2[j];
                    if (!all_seen) {
                        const int in_tile = 16 * cell + 8 * e + g;
                        const int key = key0 + in_tile;
                        const bool sees = key <= pos[j] && key < L &&
                                          (a.window == 0 || key > pos[j] - a.window || key < a.sinks);
                        if (((in_tile < 32 ? bad0 : bad1) >> (in_tile & 31)) & 1u) x = NAN;
                        if (!sees) x = -INFINITY;
                    }
                    s[cell][j][e] = x;
                    mx = fmaxf(mx, x);
                }
            }
            if (plan.pad_len) {
                const int rr = row0 + 4 * j + t;
                if (rr < n_rows) {
                    float* st = reinterpret_cast<float*>(a.ws + plan.stash_off) +
                                ((static_cast<int64_t>(b) * c.heads + h) * (r.max_q * group) + rr) * plan.pad_len + key0;
#pragma unroll
                    for (int cell = 0; cell < 4; ++cell) {
                        st[16 * cell + g] = s[cell][j][0];
                        st[16 * cell + g + 8] = s[cell][j][1];
                    }
                }
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
            const float m2 = fmaxf(m[j], mx);
            const float base = m2 == -INFINITY ? 0.f : m2;
            if (mx > m[j]) {
                const float keep = exp2f(m[j] - base);
                l[j] *= keep;
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[j][k][0][e] *= keep;
                        o[j][k][1][e] *= keep;
                    }
            }
            m[j] = m2;
#pragma unroll
            for (int cell = 0; cell < 4; ++cell) {
                s[cell][j][0] = exp2f(s[cell][j][0] - base);
                s[cell][j][1] = exp2f(s[cell][j][1] - base);
                l[j] += s[cell][j][0] + s[cell][j][1];
            }
        }

        // Output of the tile.  An f16 pair holds p to 2^-17 of itself down to
        // 2^-23 of the running maximum.  Tokens below that (rare: 16 in natural
        // logarithm) go in a pass of their own with everything lifted by 2^23,
        // so a dim where the large ones happen to be 0 keeps its precision;
        // below 2^-92 they count as 0.
        const float up = pow2(v_up);
        float lift = 1.f;
        for (;;) {
            float rest[4][NT][2];
            bool more = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int cell = 0; cell < 4; ++cell)
#pragma unroll
                    for (int e = 0; e < 2; ++e) more |= s[cell][j][e] < kTiny && s[cell][j][e] > 0.f;
            more = __any_sync(0xFFFFFFFFu, more) && lift < 0x1p69f;
            if (more) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int cell = 0; cell < 4; ++cell)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool small = s[cell][j][e] < kTiny;  // (false for NaN)
                            rest[cell][j][e] = small ? s[cell][j][e] * (1.f / kTiny) : 0.f;
                            if (small) s[cell][j][e] = 0.f;
                        }
            }
#pragma unroll
            for (int cell = 0; cell < 4; ++cell) {
                const uint8_t* cp = vt + cell * cell_bytes(D);
                // p of tokens 2 t, 2 t + 1 and 8 further, of row 4 j + g / 2: f16
                // value and remainder, fetched from the lanes that hold them.
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float p0 = s[cell][j][0] * up, p1 = s[cell][j][1] * up;
                    const uint32_t hw = pack_f16(p0, p1);
                    const float2 hf = __half22float2(as_half2(hw));
                    const uint32_t lw = pack_f16(p0 - hf.x, p1 - hf.y);
                    const uint32_t x0 = __byte_perm(hw, lw, 0x5410), x1 = __byte_perm(hw, lw, 0x7632);
                    const int from = 8 * t + (g >> 1);
                    const uint32_t a0 = __shfl_sync(0xFFFFFFFFu, x0, from), a1 = __shfl_sync(0xFFFFFFFFu, x0, from + 4);
                    const uint32_t c0 = __shfl_sync(0xFFFFFFFFu, x1, from), c1 = __shfl_sync(0xFFFFFFFFu, x1, from + 4);
                    ph[j][0] = __byte_perm(a0, a1, 0x5410);
                    pl[j][0] = __byte_perm(a0, a1, 0x7632);
                    ph[j][1] = __byte_perm(c0, c1, 0x5410);
                    pl[j][1] = __byte_perm(c0, c1, 0x7632);
                }
                // Scales of tokens 2 t, 2 t + 1 and 8 further.
                uint32_t dw[2][NB];
                load_words<NB>(cp + cell_scales(D) + 2 * t * 2 * NB, dw[0]);
                load_words<NB>(cp + cell_scales(D) + (2 * t + 8) * 2 * NB, dw[1]);
#pragma unroll
                for (int k2 = 0; k2 < NB; k2 += 2) {
                    uint32_t w[4];
                    ldmatrix_x4_trans(smem_addr(cp) + k2 * 256 + lane * 16, w);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int k = k2 + u;
                        const uint32_t w0 = w[2 * u], w1 = w[2 * u + 1];
                        const uint32_t y0 = w0 >> 8, y1 = w1 >> 8;
                        const uint32_t sel = u ? 0x7632u : 0x5410u;
                        const __half2 da = as_half2(__byte_perm(dw[0][k2 / 2], dw[0][NB / 2 + k2 / 2], sel));
                        const __half2 db = as_half2(__byte_perm(dw[1][k2 / 2], dw[1][NB / 2 + k2 / 2], sel));
                        const uint32_t l0 = minus8_low(w0), l1 = minus8_low(y0), l2 = minus8_low(w1), l3 = minus8_low(y1);
                        const uint32_t h0 = minus8_high(w0), h1 = minus8_high(y0), h2 = minus8_high(w1),
                                       h3 = minus8_high(y1);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const __half2 pa = as_half2(ph[j][0]), pb = as_half2(ph[j][1]);
                            const __half2 xa = __hmul2(pa, da), xb = __hmul2(pb, db);
                            const __half2 ra = __hfma2(as_half2(pl[j][0]), da, __hfma2(pa, da, __hneg2(xa)));
                            const __half2 rb = __hfma2(as_half2(pl[j][1]), db, __hfma2(pb, db, __hneg2(xb)));
                            const uint32_t b0 = as_word((g & 1) ? ra : xa), b1 = as_word((g & 1) ? rb : xb);
                            mma_f16(o[j][k][0], l0, l1, l2, l3, b0, b1);
                            mma_f16(o[j][k][1], h0, h1, h2, h3, b0, b1);
                        }
                    }
                }
            }
            if (!more) break;
            lift *= 1.f / kTiny;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int cell = 0; cell < 4; ++cell) s[cell][j][0] = rest[cell][j][0], s[cell][j][1] = rest[cell][j][1];
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[j][k][0][e] *= 1.f / kTiny;
                        o[j][k][1][e] *= 1.f / kTiny;
                    }
            }
        }
        if (lift != 1.f) {
            const float back = 1.f / lift;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[j][k][0][e] *= back;
                        o[j][k][1][e] *= back;
                    }
        }

        __syncwarp();
        const int nx = i + kStages * kWarps;
        if (nx < tile_end) {
            fence_proxy_async_shared();  // scales zeroed above, then overwritten by the copy
            issue(nx, stage, off_next);
            off_next = source(nx + kWarps);
        }
    }
    if (!ok && i + kWarps < tile_end) {  // a copy that did not land: wait for the other stage's too
        mbar_wait_bounded(&bars[warp][(n + 1) % kStages], ((n + 1) / kStages) & 1, &g_attn_step_error);
    }

    // The warps' sums meet in shared memory: [row][D] sums, then maxima, then l.
    __syncthreads();
    float* mine = reinterpret_cast<float*>(my_ring);
    const float unit = pow2(-v_up);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[j] += __shfl_xor_sync(0xFFFFFFFFu, l[j], x);
        float* dst = mine + (4 * j + t) * D + 2 * g;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const float* lo = o[j][k][0];
            const float* hi = o[j][k][1];
            *reinterpret_cast<float2*>(dst + 32 * k) =
                make_float2((lo[0] + lo[1]) * unit, (lo[2] + lo[3]) * unit);
            *reinterpret_cast<float2*>(dst + 32 * k + 16) =
                make_float2((hi[0] + hi[1]) * unit, (hi[2] + hi[3]) * unit);
        }
        if (g == 0) {
            mine[S::kRows * D + 4 * j + t] = m[j];
            mine[S::kRows * D + S::kRows + 4 * j + t] = l[j];
        }
    }
    __syncthreads();

    auto finish = [&](int rr, int d4, float4 v, float mm, float ll) {  // row rr, dims d4 .. d4 + 3
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int64_t row = first + rr / group;
        const int head = h * group + rr % group;
        store_o4(static_cast<T*>(a.out) + row * a.out_stride + static_cast<int64_t>(head) * D + d4,
                 make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        if (d4 == 0) {
            const float lse2 = ll == 0.f ? -INFINITY : mm + log2f(ll);
            if (a.lse) a.lse[row * a.heads + head] = lse2 * kLn2;
            if (plan.pad_len) reinterpret_cast<float*>(a.ws + plan.lse_off)[row * a.heads + head] = lse2;
        }
    };

    const int64_t pair = (static_cast<int64_t>(b) * c.heads + h) * plan.groups + rg;
    constexpr int kPart = S::kRows * (D + 2);  // floats of one range's sums
    float* part = reinterpret_cast<float*>(a.ws + plan.part_off) + (pair * plan.splits + split) * kPart;
    for (int it = threadIdx.x; it < S::kRows * D / 4; it += kThreads) {
        const int rl = it / (D / 4), d4 = (it % (D / 4)) * 4;
        float mm = -INFINITY;
        float mw[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mw[w] = reinterpret_cast<const float*>(ring + w * S::kRing)[S::kRows * D + rl];
            mm = fmaxf(mm, mw[w]);
        }
        const float base = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float* src = reinterpret_cast<const float*>(ring + w * S::kRing);
            const float f = exp2f(mw[w] - base);
            ll = fmaf(f, src[S::kRows * D + S::kRows + rl], ll);
            const float4 x = *reinterpret_cast<const float4*>(src + rl * D + d4);
            v.x = fmaf(f, x.x, v.x);
            v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z);
            v.w = fmaf(f, x.w, v.w);
        }
        if (n_splits == 1) {
            if (row0 + rl < n_rows) finish(row0 + rl, d4, v, mm, ll);
        } else {
            *reinterpret_cast<float4*>(part + rl * D + d4) = v;
            if (d4 == 0) {
                part[S::kRows * D + rl] = mm;
                part[S::kRows * D + S::kRows + rl] = ll;
            }
        }
    }
    if (n_splits == 1) return;

    // The last range to arrive adds all of them up, in order.
    __threadfence();
    __syncthreads();
    unsigned* ctr = reinterpret_cast<unsigned*>(a.ws) + pair;
    if (threadIdx.x == 0) {
        const unsigned before = atomicAdd(ctr, 1u);
        s_last = before == static_cast<unsigned>(n_splits) - 1;
        if (s_last) *ctr = 0;  // fit for the next call
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const float* parts = reinterpret_cast<const float*>(a.ws + plan.part_off) + pair * plan.splits * kPart;
    for (int it = threadIdx.x; it < S::kRows * D / 4; it += kThreads) {
        const int rl = it / (D / 4), d4 = (it % (D / 4)) * 4;
        if (row0 + rl >= n_rows) continue;
        float mm = -INFINITY;
        for (int x = 0; x < n_splits; ++x) mm = fmaxf(mm, __ldcg(parts + x * kPart + S::kRows * D + rl));
        const float base = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int x = 0; x < n_splits; ++x) {
            const float* p = parts + x * kPart;
            const float4 y = __ldcg(reinterpret_cast<const float4*>(p + rl * D + d4));
            const float f = exp2f(__ldcg(p + S::kRows * D + rl) - base);
            ll = fmaf(f, __ldcg(p + S::kRows * D + S::kRows + rl), ll);
            v.x = fmaf(f, y.x, v.x);
            v.y = fmaf(f, y.y, v.y);
            v.z = fmaf(f, y.z, v.z);
            v.w = fmaf(f, y.w, v.w);
        }
        finish(row0 + rl, d4, v, mm, ll);
    }
}

// weights[b][h][j] += sum over rows of exp(s - lse), from the scores that the
// step left in the workspace: one thread per token.  Reads 4 bytes per row
// and token; recomputing the scores would read the keys again (72 bytes per
// token at D = 128, as much as 18 rows).
__global__ void __launch_bounds__(256) attn_step_weights_kernel(KvView c, KvRows r, AttnCall a, StepPlan plan) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int h = blockIdx.y, b = blockIdx.z;
    const int j = blockIdx.x * 256 + threadIdx.x;
    int first, count;
    kv_rows(r, b, &first, &count, &g_attn_step_error);
    const int L = kv_length(c, b, &g_attn_step_error);
    if (j >= L) return;
    const int group = a.heads / c.heads;
    const int base_pos = L - count;
    const float* stash = reinterpret_cast<const float*>(a.ws + plan.stash_off) +
                         (static_cast<int64_t>(b) * c.heads + h) * (r.max_q * group) * plan.pad_len + j;
    const float* lse = reinterpret_cast<const float*>(a.ws + plan.lse_off);
    float acc = 0.f;
    for (int i = max(0, j - base_pos); i < count; ++i) {
        const int pos = base_pos + i;
        if (a.window > 0 && j <= pos - a.window && j >= a.sinks) break;
        for (int x = 0; x < group; ++x) {
            const float s = __ldcs(stash + static_cast<int64_t>(i * group + x) * plan.pad_len);
            acc += exp2f(s - __ldg(lse + static_cast<int64_t>(first + i) * a.heads + h * group + x));
        }
    }
    float* w = a.weights + (static_cast<int64_t>(b) * c.heads + h) * a.weights_stride + j;
    *w += acc;
}

// Rows of a CTA: 4 where that is all there are, else 8.
int row_tiles(int rows) { return rows <= 4 ? 1 : 2; }

StepPlan make_plan(const KvView& c, int heads, int64_t n_tokens, int64_t max_q, int window, int sinks, bool weights) {
    StepPlan p = {};
    const int64_t rows = max_q * (heads / c.heads);
    const int per = 4 * row_tiles(static_cast<int>(rows));
    p.groups = static_cast<int>((rows + per - 1) / per);
    int64_t tiles = (c.max_len + kTile - 1) / kTile;
    if (window > 0)
        tiles = std::min<int64_t>(tiles, (sinks + kTile - 1) / kTile + (window + max_q + kTile - 1) / kTile + 1);
    tiles = std::max<int64_t>(tiles, 1);
    // Ranges long enough that their ends cost little, and enough of them to
    // fill the SMs several times over when sequences differ in length.
    const int64_t pairs = static_cast<int64_t>(c.n_seqs) * c.heads * p.groups;
    const int64_t want = std::max<int64_t>(1, kTargetCtas / std::max<int64_t>(1, pairs));
    int64_t per_cta = (tiles + want - 1) / want;
    per_cta = (per_cta + kWarps - 1) / kWarps * kWarps;
    p.tiles_per_cta = static_cast<int>(per_cta);
    p.splits = static_cast<int>((tiles + per_cta - 1) / per_cta);
    // Room for the partial sums of the most ranges that any window gives.
    const int64_t most = std::min<int64_t>(want, (c.max_len + kTile * kWarps - 1) / (kTile * kWarps));
    auto take = [&](int64_t bytes) {
        const int64_t at = p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    if (most > 1) {
        take(kCtrBytes);
        p.part_off = take(pairs * most * per * (c.dim + 2) * 4);
    }
    if (weights) {
        p.pad_len = static_cast<int>((c.max_len + kTile - 1) / kTile * kTile);
        if (most <= 1) take(kCtrBytes);
        p.lse_off = take(n_tokens * heads * 4);
        p.stash_off = take(static_cast<int64_t>(c.n_seqs) * c.heads * rows * p.pad_len * 4);
    }
    return p;
}

template <int D, int NT, typename T>
cudaError_t launch_step(const KvView& c, const KvRows& r, const AttnCall& a, const StepPlan& p, cudaStream_t stream) {
    using S = StepShape<D, NT>;
    static SmemOnce once;
    cudaError_t err = once.set(attn_step_kernel<D, NT, T>, S::kSmem);
    if (err != cudaSuccess) return err;
    note_launch();
    err = launch_pdl(attn_step_kernel<D, NT, T>, dim3(p.splits * p.groups, c.heads, c.n_seqs),
                                 dim3(kThreads), S::kSmem, stream, c, r, a, p);
    if (err != cudaSuccess || !a.weights || c.max_len == 0) return err;
    note_launch();
    return launch_pdl(attn_step_weights_kernel, dim3(static_cast<unsigned>((c.max_len + 255) / 256), c.heads, c.n_seqs),
                      dim3(256), 0, stream, c, r, a, p);
}

template <int D, typename T>
cudaError_t launch_step(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    const StepPlan p = make_plan(c, a.heads, r.n_tokens, r.max_q, a.window, a.sinks, a.weights != nullptr);
    return row_tiles(r.max_q * (a.heads / c.heads)) == 1 ? launch_step<D, 1, T>(c, r, a, p, stream)
                                                         : launch_step<D, 2, T>(c, r, a, p, stream);
}

}  // namespace

bool attn_step_takes(const KvView& c, int heads, int64_t max_q) {
    return (c.dim == 64 || c.dim == 128) && max_q * (heads / c.heads) <= kStepRows;
}

int64_t attn_step_workspace(const KvView& c, int heads, int64_t n_tokens, int64_t max_q, bool weights) {
    return make_plan(c, heads, n_tokens, max_q, 0, 0, weights).bytes;
}

cudaError_t launch_attn_step(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    if (c.dim == 64)
        return a.type == KvType::kF32 ? launch_step<64, float>(c, r, a, stream)
                                      : launch_step<64, __nv_bfloat16>(c, r, a, stream);
    return a.type == KvType::kF32 ? launch_step<128, float>(c, r, a, stream)
                                  : launch_step<128, __nv_bfloat16>(c, r, a, stream);
}

cudaError_t attn_step_read_device_error(unsigned int* bits, bool clear) {
    unsigned int v = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_attn_step_error, sizeof(v));
    if (err != cudaSuccess) return err;
    *bits |= v;
    if (clear && v) {
        const unsigned int zero = 0;
        err = cudaMemcpyToSymbol(g_attn_step_error, &zero, sizeof(zero));
    }
    return err;
}

}  // namespace qm
