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
//     FMAs per two tokens).
// The softmax runs in one pass with a running maximum and sum in f32.  Each tile has
// its own maximum per row (rounded up to a whole power of two, so the factor to the
// running one is exact) and its own power of two for the value scales: p d then
// begins at the top of f16's range whatever the scores and scales are, and a pair
// holds 2^-21 of it down to 2^-18 of the tile's largest, 2^-17 down to 2^-22.  A tile
// that spans more (scores of deviation 3 or so, or scales far apart) takes three
// bf16 pieces (24 bits, f32's range) in a loop of its own: 64 sequences of 8192 tokens
// 188 us in place of 136 where every tile does.  A tile's products join the sums by
// f32 FMAs.  (Sums left in the tensor cores' accumulators, one power of two for all
// tiles and p from the running maximum took 129 us, but were off by 3e-6 over 16384
// values of one sign, by 2^-10 and more among scales far apart, and 206 us with one
// token 8 nats above the others, where this takes 138.)
//
// Bytes are its floor: 9 D / 8 per token and kv head.  A tensor-core product covers
// 256 quants = 144 bytes, which HBM delivers in 6 cycles per SM; unpacking on
// the FP32 pipe alone (one FMA per quant and query row) would need 3 times
// that at four rows.  What bounds it as it is: 366 instructions per 16 tokens,
// keys, softmax and values together, in chains that 12 warps per SM cannot hide.
// Measured, 32 heads of 8 kv heads, D = 128: 64 sequences of 8192 tokens 136 us,
// 4.4 TB/s; ragged ones of up to 8192 101 us, 3.7 TB/s; one of 131071 48 us, 3.1 TB/s.
//
// Split.  All (sequence, kv head, 4 or 8 rows) lists of 64-token tiles lie end to
// end, and every CTA of a grid that fills the GPU once takes an equal stretch
// of them, so sequences of any lengths keep all SMs busy to the end.  A CTA's
// four warps take the tiles of a list in turn, each through its own two-stage
// ring, filled with bulk copies (a cell is contiguous, a page is too), and
// meet once at the list's or the stretch's end.  Where a list is cut, its
// parts meet in the workspace: the last CTA to arrive adds them up in order,
// so the result does not depend on which one that is.
#include <algorithm>

#include "kv_cache.cuh"

namespace qm {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;  // tokens of a warp's tile
constexpr int kStages = 2;  // tiles in a warp's ring
constexpr int kCtasPerSm = 3;
// How far (log2) below a tile's largest p d its smallest may lie in f16 pairs.
constexpr float kPairSpan = 22.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The grid: as many CTAs as the GPU holds at once (three per SM), each with an
// equal share of all tiles, but no more than the workspace has room for.
constexpr int kMaxCtas = 456;

struct StepPlan {
    int groups;   // row groups
    int pad_len;  // tokens per row of the stashed scores (0: none)
    int64_t part_off, stash_off, lse_off, bytes;  // offsets in the workspace
    uint32_t k1024;                               // two f16 1024
};

// The workspace begins with arrival counters, zero between calls: 4 KB of it
// are never anything else, whatever calls share the workspace.
constexpr int64_t kCtrBytes = kAttnZeroed;
static_assert(kMaxCtas * 4 <= kCtrBytes - 16, "a counter for each (the last 16 bytes are the prompt kernel's)");

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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_first(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The bf16 product, from zero and onto a sum.
__device__ __forceinline__ void mma_bf16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {  // lo in bits 0..15
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_word(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

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
// 1024 + 16 n), and one packed operation, exact, takes the rest away.  `k1024`
// (two f16 1024) comes from memory: with both constants known the compiler
// makes two logic instructions of the AND and the OR, and those bound the
// kernel (131 of 432 instructions per 16 tokens, at half rate).
__device__ __forceinline__ uint32_t minus8_low(uint32_t w, uint32_t k1024) {
    return as_word(__hadd2(as_half2((w & 0x000F000Fu) | k1024), as_half2(0xE408E408u)));  // - 1032
}
__device__ __forceinline__ uint32_t minus8_high(uint32_t w, uint32_t k1024) {
    return as_word(__hfma2(as_half2((w & 0x00F000F0u) | k1024), as_half2(0x2C002C00u),  // / 16
                           as_half2(0xD480D480u)));                                      // - 72
}

// n - 8 as bf16 pairs for the low nibbles of bytes 0 and 2: OR-ed into the mantissa of
// 128 a nibble reads 128 + n.
__device__ __forceinline__ uint32_t minus8_bf16(uint32_t w) {
    const uint32_t x = (w & 0x000F000Fu) | 0x43004300u, m136 = 0xC308C308u;
    const __nv_bfloat162 y = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&m136));
    return *reinterpret_cast<const uint32_t*>(&y);
}
// Three bf16 pieces of two f32 numbers (lo in bits 0..15): 24 bits, with f32's range.
__device__ __forceinline__ void pieces_bf16(float lo, float hi, uint32_t w[3]) {
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
        w[e] = *reinterpret_cast<const uint32_t*>(&y);
        lo -= __uint_as_float(w[e] << 16);
        hi -= __uint_as_float(w[e] & 0xFFFF0000u);
    }
}

// o += acc f, two at a time.
__device__ __forceinline__ void add_to(float o[4], const float acc[4], float f) {
#pragma unroll
    for (int e = 0; e < 4; e += 2)
        asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4}; mov.b64 z, {%0, %1};\n"
            "fma.rn.f32x2 z, x, y, z; mov.b64 {%0, %1}, z;}"
            : "+f"(o[e]), "+f"(o[e + 1])
            : "f"(acc[e]), "f"(acc[e + 1]), "f"(f));
}

template <int D, int NT>
struct StepShape {
    static constexpr int kBlocks = D / 32;
    static constexpr int kRows = 4 * NT;                // query rows of a CTA
    static constexpr int kHalf = (kTile / 16) * 9 * D;  // bytes of a tile's keys (or values)
    static constexpr int kRing = kStages * 2 * kHalf;   // of one warp
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kRows * D * 4 + 2 * kRows * 4 <= kRing, "a warp's sums fit in its ring");
};

// Tiles of sequence b for one kv head and row group: at least one where it has
// rows (their outputs are written even if they see nothing).
__device__ __forceinline__ TileList seq_tiles(const KvView& c, const KvRows& r, const AttnCall& a, int b, int* first,
                                              int* count, int* L) {
    kv_rows(r, b, first, count, c.err);
    *L = kv_length(c, b, c.err);
    TileList t{0, 0, 0};
    if (*count > 0) {
        t = tile_list<kTile>(*L, max(*L - *count, 0), a.window, a.sinks);
        t.count = max(t.count, 1);
    }
    return t;
}

// Sum of `v` over the threads before this one (*total: over all of them).
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kCtasPerSm : 2)
    attn_step_kernel(KvView c, KvRows r, AttnCall a, StepPlan plan) {
    using S = StepShape<D, NT>;
    constexpr int NB = S::kBlocks;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ int64_t scan[kWarps];
    __shared__ int s_seq, s_last;
    __shared__ int64_t s_seq_off;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    if (threadIdx.x < kWarps * kStages) mbar_init(&bars[0][0] + threadIdx.x, 1);
    if (threadIdx.x == 0) s_seq = -1;
    fence_barrier_init();
    __syncthreads();
    grid_launch_dependents();
    grid_dependency_wait();

    // How the tiles go to CTAs.  Where lists are few or short, every list is cut
    // into ranges of `per` tiles and every range has a CTA; else the lists lie
    // end to end and CTA x takes tiles x per .. (x + 1) per - 1 of them all.
    const int64_t lists = static_cast<int64_t>(c.heads) * plan.groups;  // tile lists per sequence
    auto sum_over = [&](auto&& of) {  // sum over the sequences of of(tiles of it) * lists
        int64_t total = 0;
        for (int b0 = 0; b0 < c.n_seqs; b0 += kThreads) {
            int f, n, L;
            const int bb = b0 + threadIdx.x;
            int64_t all;
            cta_scan(bb < c.n_seqs ? of(seq_tiles(c, r, a, bb, &f, &n, &L).count) * lists : 0, scan, &all);
            total += all;
        }
        return total;
    };
    const int64_t grid = gridDim.x;
    int64_t total = sum_over([](int n) -> int64_t { return n; });
    int64_t per = (total + grid - 1) / grid;
    per = max(static_cast<int64_t>(kWarps), (per + kWarps - 1) / kWarps * kWarps);
    bool ranges = false;
    for (int64_t p = per; p <= max(per + per / 4, static_cast<int64_t>(2 * kWarps)); p += kWarps) {
        const int64_t n = sum_over([p](int n) -> int64_t { return (n + p - 1) / p; });
        if (n <= grid) {
            ranges = true;
            per = p;
            total = n;  // of ranges from here on
            break;
        }
    }
    int64_t tile_at = ranges ? blockIdx.x : per * blockIdx.x;
    const int64_t tile_stop = ranges ? min(total, tile_at + 1) : min(total, tile_at + per);
    if (tile_at >= tile_stop) return;
    {
        int64_t seen = 0;
        for (int b0 = 0; b0 < c.n_seqs; b0 += kThreads) {
            int f, n, L;
            const int bb = b0 + threadIdx.x;
            int64_t all;
            int64_t mine = bb < c.n_seqs ? seq_tiles(c, r, a, bb, &f, &n, &L).count : 0;
            mine = (ranges ? (mine + per - 1) / per : mine) * lists;
            const int64_t off = seen + cta_scan(mine, scan, &all);
            if (off <= tile_at && tile_at < off + mine) {
                s_seq = bb;
                s_seq_off = off;
            }
            seen += all;
            if (seen > tile_at) break;
        }
        __syncthreads();
    }
    int b = s_seq;
    int64_t seq_off = s_seq_off;  // of sequence b's first tile (or range)
    int first, count, L;
    TileList tiles = seq_tiles(c, r, a, b, &first, &count, &L);
    const int group = a.heads / c.heads;
    int n = 0;  // tiles that this warp has been through, for its ring
    bool ok = true;

    while (tile_at < tile_stop) {
    // This segment: tiles seg_begin .. tile_end - 1 of a list, one of n_parts of it.
    int list, seg_begin, tile_end, n_parts;
    int64_t c0;     // the CTA that has the list's first tiles
    bool first_in;  // ... as its first segment
    bool at_start = true;
    if (ranges) {
        n_parts = static_cast<int>((tiles.count + per - 1) / per);
        const int64_t x = tile_at - seq_off;
        list = static_cast<int>(x / n_parts);
        const int part = static_cast<int>(x % n_parts);
        c0 = tile_at - part;
        first_in = true;
        seg_begin = static_cast<int>(part * per);
        tile_end = static_cast<int>(min(seg_begin + per, static_cast<int64_t>(tiles.count)));
        ++tile_at;
    } else {
        while (tile_at >= seq_off + tiles.count * lists) {  // on to the next sequence with rows
            seq_off += tiles.count * lists;
            tiles = seq_tiles(c, r, a, ++b, &first, &count, &L);
        }
        list = static_cast<int>((tile_at - seq_off) / tiles.count);
        const int64_t list_off = seq_off + static_cast<int64_t>(list) * tiles.count;
        seg_begin = static_cast<int>(tile_at - list_off);
        tile_end = static_cast<int>(min(tile_stop - list_off, static_cast<int64_t>(tiles.count)));
        at_start = tile_at == per * blockIdx.x;
        c0 = list_off / per;
        first_in = list_off == c0 * per;
        n_parts = static_cast<int>((list_off + tiles.count - 1) / per - c0) + 1;
        tile_at = list_off + tile_end;
    }
    const int h = list / plan.groups, rg = list % plan.groups;

    const int n_rows = count * group;  // rows of this (sequence, kv head): token-major, then query head
    const int row0 = rg * S::kRows;
    const int base_pos = L - count;  // position of the sequence's first row (may be negative)
    if (row0 >= n_rows) continue;    // (a sequence with fewer rows than others: every thread alike)
    const int pos_lo = base_pos + row0 / group;
    const int pos_hi = base_pos + min(n_rows - 1, row0 + S::kRows - 1) / group;
    const int seen_len = max(0, min(L, pos_hi + 1));

    uint8_t* my_ring = ring + warp * S::kRing;
    // Eight lanes copy a tile: keys' cells 0..3, then values'.  Where a page
    // holds a tile, one copy takes all four cells.  Lanes 8 u .. 8 u + 7 look
    // up the pages of this warp's tile 4 x + u, four tiles at a time and four
    // ahead.
    const bool whole = c.page_shift >= 6;
    const int tile_first = seg_begin + warp;
    const int my_tiles = ok && tile_first < tile_end ? (tile_end - tile_first + kWarps - 1) / kWarps : 0;
    auto look_up = [&](int x) -> int64_t {  // for this warp's tiles 4 x .. 4 x + 3
        const int i = tile_first + (4 * x + (lane >> 3)) * kWarps;
        if (i >= tile_end) return -1;
        const int p = tiles.at(i) * kTile + (lane & 3) * 16;
        if (p >= seen_len || (whole && (lane & 3))) return -1;
        return kv_cell(c, b, h, p, c.err);
    };
    int64_t off4 = look_up(0), off4_next = look_up(1);
    auto issue = [&](int x, int stage) {  // this warp's tile x, looked up
        const int left = seen_len - tiles.at(tile_first + x * kWarps) * kTile;
        const bool mine = (lane >> 3) == (x & 3) && off4 >= 0;
        const int cells = whole ? min(4, (left + 15) >> 4) : 1;
        const uint32_t bytes = static_cast<uint32_t>(cells * cell_bytes(D));
        const uint32_t copies = __popc(__ballot_sync(0xFFFFFFFFu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&bars[warp][stage], copies * bytes);
        __syncwarp();
        if (mine) {
            uint8_t* dst = my_ring + stage * 2 * S::kHalf + ((lane >> 2) & 1) * S::kHalf + (lane & 3) * cell_bytes(D);
            bulk_load_1d(dst, ((lane & 4) ? c.v : c.k) + off4, bytes, &bars[warp][stage]);
        }
    };
#pragma unroll
    for (int x = 0; x < kStages; ++x)
        if (x < my_tiles) issue(x, (n + x) % kStages);

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
    const uint32_t k1024 = plan.k1024;

    // Scores of a tile, to base 2: s[cell][j][0] of token 16 cell + g, [1]: 8 further.
    auto score_cell = [&](const uint8_t* kt, int cell, float (&s)[4][NT][2]) {
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
                const uint32_t l0 = minus8_low(w0, k1024), l1 = minus8_low(w1, k1024), l2 = minus8_low(y0, k1024),
                               l3 = minus8_low(y1, k1024);
                const uint32_t h0 = minus8_high(w0, k1024), h1 = minus8_high(w1, k1024), h2 = minus8_high(y0, k1024),
                               h3 = minus8_high(y1, k1024);
                const float2 dd0 = __half22float2(as_half2(d0[k2 / 2]));
                const float2 dd1 = __half22float2(as_half2(d1[k2 / 2]));
                const float e0 = u ? dd0.y : dd0.x, e1 = u ? dd1.y : dd1.x;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float acc[4];
                    mma_f16_first(acc, l0, l1, l2, l3, bq[j][k][0], bq[j][k][1]);
                    mma_f16(acc, h0, h1, h2, h3, bq[j][k][2], bq[j][k][3]);
                    s[cell][j][0] = fmaf(e0, acc[0] + acc[1], s[cell][j][0]);
                    s[cell][j][1] = fmaf(e1, acc[2] + acc[3], s[cell][j][1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            s[cell][j][0] *= to_log2[j];
            s[cell][j][1] *= to_log2[j];
        }
    };
    // o += f * sum over the cell's tokens of up p d (n - 8); s holds p.  The products of a
    // cell start from zero: the tensor cores cut their sums off instead of rounding them,
    // which over many tiles would show (3e-6 of sums of one sign after 64 tiles).
    auto output_cell = [&](const uint8_t* vt, int cell, const float (&s)[4][NT][2], float up, const float (&f)[NT]) {
        const uint8_t* cp = vt + cell * cell_bytes(D);
        // p of tokens 2 t, 2 t + 1 and 8 further, of row 4 j + g / 2: f16 value
        // and remainder, fetched from the lanes that hold them.
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
                const uint32_t l0 = minus8_low(w0, k1024), l1 = minus8_low(y0, k1024), l2 = minus8_low(w1, k1024),
                               l3 = minus8_low(y1, k1024);
                const uint32_t h0 = minus8_high(w0, k1024), h1 = minus8_high(y0, k1024), h2 = minus8_high(w1, k1024),
                               h3 = minus8_high(y1, k1024);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const __half2 pa = as_half2(ph[j][0]), pb = as_half2(ph[j][1]);
                    const __half2 xa = __hmul2(pa, da), xb = __hmul2(pb, db);
                    const __half2 ra = __hfma2(as_half2(pl[j][0]), da, __hfma2(pa, da, __hneg2(xa)));
                    const __half2 rb = __hfma2(as_half2(pl[j][1]), db, __hfma2(pb, db, __hneg2(xb)));
                    const uint32_t b0 = as_word((g & 1) ? ra : xa), b1 = as_word((g & 1) ? rb : xb);
                    float acc[4];
                    mma_f16_first(acc, l0, l1, l2, l3, b0, b1);
                    add_to(o[j][k][0], acc, f[j]);
                    mma_f16_first(acc, h0, h1, h2, h3, b0, b1);
                    add_to(o[j][k][1], acc, f[j]);
                }
            }
        }
    };
    // The same where p d spans more than f16 pairs hold: three bf16 pieces of p d (24
    // bits, f32's range) in three of every four columns of two products.
    auto output_wide = [&](const uint8_t* cp, const float (&s)[NT][2], const float (&f)[NT]) {
        const int from = 8 * t + (g >> 1);
        float p[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[j][e] = __shfl_sync(0xFFFFFFFFu, s[j][e >> 1], from + 4 * (e & 1));
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
                const uint32_t sel = u ? 0x7632u : 0x5410u;
                const float2 da = __half22float2(as_half2(__byte_perm(dw[0][k2 / 2], dw[0][NB / 2 + k2 / 2], sel)));
                const float2 db = __half22float2(as_half2(__byte_perm(dw[1][k2 / 2], dw[1][NB / 2 + k2 / 2], sel)));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    uint32_t x[3], y[3];
                    pieces_bf16(p[j][0] * da.x, p[j][1] * da.y, x);
                    pieces_bf16(p[j][2] * db.x, p[j][3] * db.y, y);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t w0 = w[2 * u] >> (4 * half), w1 = w[2 * u + 1] >> (4 * half);
                        const uint32_t a[4] = {minus8_bf16(w0), minus8_bf16(w0 >> 8), minus8_bf16(w1), minus8_bf16(w1 >> 8)};
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_bf16(acc, a, (g & 1) ? 0u : x[2], (g & 1) ? 0u : y[2]);
                        mma_bf16(acc, a, (g & 1) ? x[1] : x[0], (g & 1) ? y[1] : y[0]);
                        add_to(o[j][k][half], acc, f[j]);
                    }
                }
            }
        }
    };

    float s[4][NT][2];
    int x = 0;
    for (; x < my_tiles; ++x, ++n) {
        const int stage = n % kStages;
        const uint8_t* kt = my_ring + stage * 2 * S::kHalf;
        uint8_t* vt = my_ring + stage * 2 * S::kHalf + S::kHalf;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bars[warp][stage], (n / kStages) & 1, c.err));
        if (!ok) break;
        const int key0 = tiles.at(tile_first + x * kWarps) * kTile;
#pragma unroll
        for (int cell = 0; cell < 4; ++cell) score_cell(kt, cell, s);

        // Scales of the values: the largest and the smallest that is not 0.  Tokens past
        // the end and those with a scale that is not finite get scales of 0.
        uint32_t bad0 = 0, bad1 = 0;  // tokens with a scale that is not finite
        uint32_t top, low;            // bits of the largest; of the smallest, less 1
        uint32_t w[NB];               // two tokens' scales
        uint8_t* const my_scales = vt + (lane >> 3) * cell_bytes(D) + cell_scales(D) + (lane & 7) * 4 * NB;
        auto extremes = [&]() {
            load_words<NB>(my_scales, w);
            uint32_t hi2 = 0x80008000u, lo2 = 0xFFFFFFFFu;
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const uint32_t y = w[e] | 0x80008000u;
                hi2 = __vmaxu2(hi2, y);
                lo2 = __vminu2(lo2, (y - 0x00010001u) ^ 0x80008000u);  // (0 becomes the largest)
            }
            top = __reduce_max_sync(0xFFFFFFFFu, max(hi2 & 0x7FFFu, (hi2 >> 16) & 0x7FFFu));
            low = __reduce_min_sync(0xFFFFFFFFu, min(lo2 & 0xFFFFu, lo2 >> 16));
        };
        extremes();
        if (top >= 0x7C00u || key0 + kTile > seen_len) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = u * 32 + lane;
                uint8_t* sc = vt + (key >> 4) * cell_bytes(D) + cell_scales(D) + (key & 15) * 2 * NB;
                uint32_t y[NB / 2];
                load_words<NB / 2>(sc, y);
                uint32_t mx = y[0] & 0x7FFF7FFFu;
#pragma unroll
                for (int e = 1; e < NB / 2; ++e) mx = __vmaxu2(mx, y[e] & 0x7FFF7FFFu);
                mx = max(mx & 0xFFFFu, mx >> 16);
                const bool past = key0 + key >= seen_len;
                const bool wild = !past && mx >= 0x7C00u;
                const uint32_t bits = __ballot_sync(0xFFFFFFFFu, wild);
                if (u == 0) bad0 = bits;
                else bad1 = bits;
                if (past || wild) {  // such tokens' products are 0; NaN comes with the scores
#pragma unroll
                    for (int e = 0; e < NB / 2; ++e) reinterpret_cast<uint32_t*>(sc)[e] = 0u;
                }
            }
            __syncwarp();
            extremes();
        }
        // p d goes to the top of f16's range, p 2^p_up times d 2^d_up below 2^16: p takes
        // up to 2^15, the scales in shared memory (exactly) what is left.
        const int top_e = max(1, static_cast<int>(top >> 10));
        const int p_up = min(15, 30 - top_e), d_up = max(0, 15 - top_e);
        if (d_up) {
            const uint32_t twice = static_cast<uint32_t>(15 + d_up) * 0x04000400u;
#pragma unroll
            for (int e = 0; e < NB; ++e) reinterpret_cast<uint32_t*>(my_scales)[e] = as_word(__hmul2(as_half2(w[e]), as_half2(twice)));
            __syncwarp();
        }
        // How far below the row's largest a token's p may be for f16 pairs (log2).
        const float span = low == 0xFFFFu ? kPairSpan
                                          : kPairSpan - static_cast<float>((__float_as_uint(f16_bits_to_float(top)) >> 23) -
                                                                           (__float_as_uint(f16_bits_to_float(low + 1)) >> 23));

        // What a row does not see, and tokens whose values are not finite.
        const bool all_seen = key0 + kTile <= min(pos_lo + 1, L) && !(bad0 | bad1) &&
                              (a.window == 0 || key0 > pos_hi - a.window || key0 + kTile <= a.sinks);
        float mn[NT];  // of the scores that the row sees, this thread's
#pragma unroll
        for (int j = 0; j < NT; ++j) mn[j] = INFINITY;
        if (all_seen) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int cell = 0; cell < 4; ++cell) mn[j] = fminf(fminf(mn[j], s[cell][j][0]), s[cell][j][1]);
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int cell = 0; cell < 4; ++cell)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int in_tile = 16 * cell + 8 * e + g;
                        const int key = key0 + in_tile;
                        const bool sees = key <= pos[j] && key < L &&
                                          (a.window == 0 || key > pos[j] - a.window || key < a.sinks);
                        if (((in_tile < 32 ? bad0 : bad1) >> (in_tile & 31)) & 1u) s[cell][j][e] = NAN;
                        if (sees) mn[j] = fminf(mn[j], s[cell][j][e]);
                        else s[cell][j][e] = -INFINITY;
                    }
        }
        if (plan.pad_len) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
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
        }
        // p is taken from the tile's own maximum, rounded up to a whole power of two, and
        // the tile's sums join the running ones with an exact factor f.
        bool wide = false;  // p d spans more than f16 pairs hold
        float f[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float mx = -INFINITY;
#pragma unroll
            for (int cell = 0; cell < 4; ++cell) mx = fmaxf(fmaxf(mx, s[cell][j][0]), s[cell][j][1]);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, y));
            mx = ceilf(mx);
            const float base = mx == -INFINITY ? 0.f : mx;
            wide |= base - mn[j] > span;
            if (mx > m[j]) {
                const float keep = exp2_approx(m[j] - mx);
                m[j] = mx;
                l[j] *= keep;
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[j][k][0][e] *= keep;
                        o[j][k][1][e] *= keep;
                    }
            }
            f[j] = exp2_approx(mx - (m[j] == -INFINITY ? 0.f : m[j]));
            float sum = 0.f;
#pragma unroll
            for (int cell = 0; cell < 4; ++cell) {
                s[cell][j][0] = exp2_approx(s[cell][j][0] - base);
                s[cell][j][1] = exp2_approx(s[cell][j][1] - base);
                sum += s[cell][j][0] + s[cell][j][1];
            }
            l[j] = fmaf(f[j], sum, l[j]);
        }
        if (!__any_sync(0xFFFFFFFFu, wide)) {
            const float up = pow2(p_up), unit = pow2(-p_up - d_up);
#pragma unroll
            for (int j = 0; j < NT; ++j) f[j] *= unit;
#pragma unroll
            for (int cell = 0; cell < 4; ++cell) output_cell(vt, cell, s, up, f);
        } else {
            const float unit = pow2(-d_up);
#pragma unroll
            for (int j = 0; j < NT; ++j) f[j] *= unit;
#pragma unroll 1
            for (int cell = 0; cell < 4; ++cell) {
                float one[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        one[j][e] = cell == 0 ? s[0][j][e] : cell == 1 ? s[1][j][e] : cell == 2 ? s[2][j][e] : s[3][j][e];
                output_wide(vt + cell * cell_bytes(D), one, f);
            }
        }
        __syncwarp();
        const int nx = x + kStages;
        if (nx < my_tiles) {
            if ((nx & 3) == 0) {
                off4 = off4_next;
                off4_next = look_up((nx >> 2) + 1);
            }
            fence_proxy_async_shared();  // scales zeroed above, then overwritten by the copy
            issue(nx, stage);
        }
    }
    if (!ok) {  // a copy that did not land: wait for the other stage's too
        if (x + 1 < my_tiles)
            mbar_wait_bounded(&bars[warp][(n + 1) % kStages], ((n + 1) / kStages) & 1, c.err);
    }

    // The warps' sums meet in shared memory: [row][D] sums, then maxima, then l.
    __syncthreads();
    float* mine = reinterpret_cast<float*>(my_ring);
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
                make_float2(lo[0] + lo[1], lo[2] + lo[3]);
            *reinterpret_cast<float2*>(dst + 32 * k + 16) =
                make_float2(hi[0] + hi[1], hi[2] + hi[3]);
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

    constexpr int kPart = S::kRows * (D + 2);  // floats of one segment's sums
    const bool alone = n_parts == 1;
    // A CTA's first segment has slot 0, its last one (if another) slot 1.
    float* parts = reinterpret_cast<float*>(a.ws + plan.part_off);
    float* part = parts + (static_cast<int64_t>(blockIdx.x) * 2 + (at_start ? 0 : 1)) * kPart;
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
            const float f = exp2_approx(mw[w] - base);
            ll = fmaf(f, src[S::kRows * D + S::kRows + rl], ll);
            const float4 y = *reinterpret_cast<const float4*>(src + rl * D + d4);
            v.x = fmaf(f, y.x, v.x);
            v.y = fmaf(f, y.y, v.y);
            v.z = fmaf(f, y.z, v.z);
            v.w = fmaf(f, y.w, v.w);
        }
        if (alone) {
            if (row0 + rl < n_rows) finish(row0 + rl, d4, v, mm, ll);
        } else {
            *reinterpret_cast<float4*>(part + rl * D + d4) = v;
            if (d4 == 0) {
                part[S::kRows * D + rl] = mm;
                part[S::kRows * D + S::kRows + rl] = ll;
            }
        }
    }
    if (!alone) {
        // The last segment of a list to arrive adds all of them up, in order.
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            // No two lists that are cut begin in the same CTA.
            unsigned* ctr = reinterpret_cast<unsigned*>(a.ws) + c0;
            const unsigned before = atomicAdd(ctr, 1u);
            s_last = before == static_cast<unsigned>(n_parts) - 1;
            if (s_last) *ctr = 0;  // fit for the next call
        }
        __syncthreads();
        if (s_last) {
            __threadfence();
            const float* p0 = parts + (c0 * 2 + (first_in ? 0 : 1)) * kPart;
            auto part_of = [&](int y) { return y == 0 ? p0 : parts + (c0 + y) * 2 * kPart; };
            for (int it = threadIdx.x; it < S::kRows * D / 4; it += kThreads) {
                const int rl = it / (D / 4), d4 = (it % (D / 4)) * 4;
                if (row0 + rl >= n_rows) continue;
                float mm = -INFINITY;
#pragma unroll 8
                for (int y = 0; y < n_parts; ++y) mm = fmaxf(mm, __ldcg(part_of(y) + S::kRows * D + rl));
                const float base = mm == -INFINITY ? 0.f : mm;
                float ll = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int y = 0; y < n_parts; ++y) {
                    const float* p = part_of(y);
                    const float4 w = __ldcg(reinterpret_cast<const float4*>(p + rl * D + d4));
                    const float f = exp2_approx(__ldcg(p + S::kRows * D + rl) - base);
                    ll = fmaf(f, __ldcg(p + S::kRows * D + S::kRows + rl), ll);
                    v.x = fmaf(f, w.x, v.x);
                    v.y = fmaf(f, w.y, v.y);
                    v.z = fmaf(f, w.z, v.z);
                    v.w = fmaf(f, w.w, v.w);
                }
                finish(row0 + rl, d4, v, mm, ll);
            }
        }
    }
    fence_proxy_async_shared();
    __syncthreads();  // the rings are free for the next segment's copies
    }  // segments
}

// weights[b][h][j] += sum over rows of exp(s - lse), from the scores that the
// step left in the workspace: one thread per token.  Reads 4 bytes per row
// and token; recomputing the scores would read the keys again (72 bytes per
// token at D = 128, as much as 18 rows).  32 sequences of 4096 (ragged), 4 rows
// each: 14 us beside the step's 40.
constexpr int kMostRows = std::max(kStepRows, kStepRowsFew);  // of a list
__global__ void __launch_bounds__(256) attn_step_weights_kernel(KvView c, KvRows r, AttnCall a, StepPlan plan) {
    grid_launch_dependents();
    grid_dependency_wait();
    __shared__ float row_lse[kMostRows];
    const int h = blockIdx.y, b = blockIdx.z;
    const int j = blockIdx.x * 256 + threadIdx.x;
    int first, count;
    kv_rows(r, b, &first, &count, c.err);
    const int L = kv_length(c, b, c.err);
    const int group = a.heads / c.heads;
    const float* lse = reinterpret_cast<const float*>(a.ws + plan.lse_off) + h * group;
    for (int x = threadIdx.x; x < count * group; x += 256) {
        const int i = x / group;
        row_lse[x] = lse[static_cast<int64_t>(first + i) * a.heads + (x - i * group)];
    }
    __syncthreads();
    if (j >= L) return;
    const int base_pos = L - count;
    const float* stash = reinterpret_cast<const float*>(a.ws + plan.stash_off) +
                         (static_cast<int64_t>(b) * c.heads + h) * (r.max_q * group) * plan.pad_len + j;
    // The rows that see token j lie together.
    const int end = a.window > 0 && j >= a.sinks ? min(count, max(0, j + a.window - base_pos)) : count;
    float acc = 0.f;
#pragma unroll 8
    for (int x = max(0, j - base_pos) * group; x < end * group; ++x)
        acc += exp2_approx(__ldcs(stash + static_cast<int64_t>(x) * plan.pad_len) - row_lse[x]);
    float* w = a.weights + (static_cast<int64_t>(b) * c.heads + h) * a.weights_stride + j;
    *w += acc;
}

// Rows of a CTA: 4 where that is all there are, else 8.
int row_tiles(int rows) { return rows <= 4 ? 1 : 2; }

StepPlan make_plan(const KvView& c, int heads, int64_t n_tokens, int64_t max_q, bool weights) {
    StepPlan p = {};
    p.k1024 = 0x64006400u;
    const int64_t rows = max_q * (heads / c.heads);
    const int per = 4 * row_tiles(static_cast<int>(rows));
    p.groups = static_cast<int>((rows + per - 1) / per);
    auto take = [&](int64_t bytes) {
        const int64_t at = p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    take(kCtrBytes);
    p.part_off = take(static_cast<int64_t>(kMaxCtas) * 2 * per * (c.dim + 2) * 4);
    if (weights) {
        p.pad_len = static_cast<int>((c.max_len + kTile - 1) / kTile * kTile);
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
    const int64_t n_lists = static_cast<int64_t>(c.n_seqs) * c.heads * p.groups;
    // At most this many tiles (a window or shorter sequences make fewer).
    const int64_t tiles = std::max<int64_t>(1, (c.max_len + kTile - 1) / kTile) * n_lists;
    const int64_t room = std::min(kMaxCtas, c.sms * (NT == 1 ? kCtasPerSm : 2));
    const int grid = static_cast<int>(std::min(room, std::max((tiles + kWarps - 1) / kWarps, n_lists)));
    err = launch_pdl(attn_step_kernel<D, NT, T>, dim3(grid), dim3(kThreads), S::kSmem, stream, c, r, a, p);
    if (err != cudaSuccess || !a.weights || c.max_len == 0) return err;
    note_launch();
    return launch_pdl(attn_step_weights_kernel, dim3(static_cast<unsigned>((c.max_len + 255) / 256), c.heads, c.n_seqs),
                      dim3(256), 0, stream, c, r, a, p);
}

template <int D, typename T>
cudaError_t launch_step(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    const StepPlan p = make_plan(c, a.heads, r.n_tokens, r.max_q, a.weights != nullptr);
    return row_tiles(r.max_q * (a.heads / c.heads)) == 1 ? launch_step<D, 1, T>(c, r, a, p, stream)
                                                         : launch_step<D, 2, T>(c, r, a, p, stream);
}

}  // namespace

bool attn_step_takes(const KvView& c, int heads, int64_t max_q) {
    if (c.dim != 64 && c.dim != 128) return false;
    const int64_t rows = max_q * (heads / c.heads), all = c.n_seqs * max_q * heads;
    return rows <= kStepRows || (rows <= kStepRowsFew && all <= kStepAll);
}

int64_t attn_step_most(const KvView& c, int heads, int64_t max_q) {
    if (c.dim != 64 && c.dim != 128) return 0;
    const int64_t group = heads / c.heads, all = static_cast<int64_t>(c.n_seqs) * heads;
    const int64_t few = all > 0 ? std::min(kStepRowsFew / group, kStepAll / all) : kStepRowsFew / group;
    return std::min(max_q, std::max(kStepRows / group, few));
}

int64_t attn_step_workspace(const KvView& c, int heads, int64_t n_tokens, int64_t max_q, bool weights) {
    return make_plan(c, heads, n_tokens, max_q, weights).bytes;
}

cudaError_t launch_attn_step(const KvView& c, const KvRows& r, const AttnCall& a, cudaStream_t stream) {
    if (c.dim == 64)
        return a.type == KvType::kF32 ? launch_step<64, float>(c, r, a, stream)
                                      : launch_step<64, __nv_bfloat16>(c, r, a, stream);
    return a.type == KvType::kF32 ? launch_step<128, float>(c, r, a, stream)
                                  : launch_step<128, __nv_bfloat16>(c, r, a, stream);
}

}  // namespace qm
