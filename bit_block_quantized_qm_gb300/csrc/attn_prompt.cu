// Attention of many rows over the paged Q4_0 cache (prompts and their chunks)
// on the 5th-generation tensor cores.
//
// Mathematics.  Tiles of 128 query rows (token-major, then the query heads of a
// kv head) meet tiles of 128 tokens: S = Q K^T and P V as tcgen05.mma into TMEM,
// one pass with a running maximum and sum per row.  A query row is scaled to the
// top of f16's range, a key tile by the power of two that takes its largest
// scale to 2^11 .. 2^12; both are then f16 pieces.
// A value tile is scaled likewise, and P takes that on (P = exp2(s + e - maximum of
// s + e)).  A value is 15 bits times its tile's power of two and never below 2^-24 of
// binary16, so two pieces hold every one exactly, unless a tile has scales of 2^12 and
// more among some below 2^-10: then its rows are done again by the plain kernel.
//   f32 rows: two pieces each (22 bits of Q and P, K and V exact) and the three
//     products that are not 2^-22 of the first, smallest first.  P's second
//     piece is kept 2^11 up, with an accumulator of its own.  Every token tile's
//     P V starts from 0 and is added to the row's sums in registers: the tensor
//     cores cut their sums off instead of rounding them, which over a long row
//     would show (2e-6 at 300 tokens, growing).
//   bf16 rows: Q in one piece (exact) and K in two, so scores, maxima and sums are as
//     exact as an f32 row's: K cut to 11 bits would move a score by 2^-12 of itself,
//     2e-3 in lse at scores of deviation 3, and a row's weights off 1 by as much. P and
//     V in one piece (11 bits; the output keeps 8), and the output accumulates in TMEM.
// What f16's range loses are tokens 2^-33 (bf16: 2^-26) below a row's maximum.
// They can matter only to an output element to which all larger tokens add up
// to about nothing: rows that have both are listed and done again by the plain
// kernel.  (bf16 pieces, which have the range, need 4 products for 2^-17, or
// give 2^-9.)  The sign of it that the kernel goes by, an element near 0, is a
// cautious one, and a row that is done again costs a CTA its whole context: where
// rows put most of their weight on one token, or values have channels that are
// always 0, that is most rows and most of the time.  4096 rows, bf16 / f32:
// scores of deviation 1 0.19 / 0.38 ms, 2 0.54 / 0.38, 3 1.2 / 0.38; deviation 2 and
// the first token 4 nats above the others 5.0 / 0.38, 8 nats 196 / 0.74, 12 nats 246 /
// 48; deviation 4 and 16 channels of 0 246 / 233.
//
// What bounds it: f32 rows the tensor cores (6 products of 2^21 MACs per pair of
// tiles at D = 128) behind the roles' waits for one another; bf16 rows (3
// products) those waits.  Measured, 32 heads of 8 kv heads, D = 128, causal: f32 rows,
// prompt of 4096 / 8192: 379 / 1280 us, 362 / 428 TFLOP/s of the formula's
// operations (three times that in products); bf16, 8192: 648 us, 848 TFLOP/s (562 us
// with K in one piece; 693 with one tile of K and two of V in shared memory, where
// there is room for three in all), D = 64 596 us (the softmax is the same).
//
// Structure, one CTA of 24 (bf16: 20) warps per (sequence, kv head, 128 or 2 x 128 rows):
//   8 decode warps read cells, a step ahead, and unpack them into 128-byte
//     swizzled tiles (dims of a block in the order the nibbles unpack; Q and the
//     output follow it); an examiner warp finds each tile's largest scales;
//   one warp issues the MMAs: S of the next tile is queued before P V of this
//     one (f32), or two row tiles take turns (bf16), so the softmax of one
//     always has products of another to run beside (bf16 with 64-token tiles, of
//     which two S per row tile fit TMEM: 755 us against 560 for 8192 rows with K in
//     one piece, a step's fixed costs double);
//   8 softmax warps hold a row per thread (f32: half a row): maximum, exponentials,
//     P back to TMEM over S (P is the A operand from there).  bf16: only when a
//     row's maximum grows by more than 2^5 is its accumulator scaled down
//     (by 2^3 that came in every sixth tile: 4% slower);
//   f32: 4 collector warps add the tiles' products up.
// Code is kept short on purpose (rolled loops over 32-column chunks): unrolled,
// the roles of the four schedulers evicted one another's instructions (805 us
// against 449 for a prompt of 4096 f32 rows).
// Registers move between the warps (setmaxnreg), from what the CTA has at launch:
// f32 768 x 80 = 256 x 72 (softmax) + 256 x 64 (decode) + 128 x 168 (collectors) +
// 128 x 40; bf16 640 x 96 >= 256 x 136 + 256 x 80 + 128 x 40.
// Every wait is bounded; a wait that gives up sets the device error word.
#include <algorithm>
#include <type_traits>

#include "tcgen05.cuh"

namespace qm {

namespace {

constexpr int kSoftmaxWarps = 8, kDecodeWarps = 8;
constexpr int kRing = 8;      // tiles whose scale factors are kept
constexpr int kKeepRing = 4;  // tiles whose rows' factors are kept for the collectors
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Bounded wait for up to three barriers in one loop: what costs a wait on the
// issuing thread is not the barrier but fetching the wait's code.
__device__ __forceinline__ bool wait_all(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc,
                                         unsigned int* err) {
#pragma unroll 1
    for (uint32_t i = 0; i < kMaxWaitPolls; ++i)
        if (mbar_try_wait(a, pa) && mbar_try_wait(b, pb) && mbar_try_wait(c, pc)) return true;
    atomicOr(err, kErrWaitTimeout);
    return false;
}

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, bool F32>
struct Shape {
    static constexpr int kBlocks = D / 32;
    static constexpr int kM = F32 ? 1 : 2;            // row tiles of a CTA
    static constexpr int kPieces = F32 ? 2 : 1;       // of Q, V and P (K always has two)
    static constexpr int kStagesK = F32 ? 1 : 2, kStagesV = F32 || D == 128 ? 1 : 2;  // tiles of K, of V
    static constexpr int kPiece = kTile * D * 2;      // bytes of one piece of a tile
    static constexpr int kOperand = kPieces * kPiece, kOperandK = 2 * kPiece;
    static constexpr int kAhead = F32 ? 2 : 1;        // tiles whose S of a row tile is queued
    static constexpr int kHalves = F32 ? 2 : 1;       // softmax threads of a row
    // Warps: softmax, decode, (f32) collectors, then MMA issue, examiner, two idle.
    static constexpr int kCollectWarps = F32 ? 4 : 0;
    static constexpr int kIssuer = kSoftmaxWarps + kDecodeWarps + kCollectWarps;
    static constexpr int kThreads = (kIssuer + 4) * 32;
    static constexpr int kSmem = kM * kOperand + kStagesK * kOperandK + kStagesV * kOperand + 1024;
    // Registers of a thread: the kernel's, and what setmaxnreg makes of them.
    static constexpr int kRegs = F32 ? 80 : 96, kSoftmaxRegs = F32 ? 72 : 136, kDecodeRegs = F32 ? 64 : 80;
    static constexpr int kCollectRegs = 168, kOtherRegs = 40;
    static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kDecodeWarps * kDecodeRegs + kCollectWarps * kCollectRegs +
                        4 * kOtherRegs) <= kThreads * kRegs, "registers of one CTA");
    static_assert(kSmem + (F32 ? 6144 : 2048) <= 232448, "shared memory of one CTA, with the static arrays");
};

// TMEM columns: S and P over it 0 .. 255 in two buffers (f32: tiles in turn, the
// pieces of 32 scores' P in 16 columns each; bf16: a row tile each), then P V in
// two of 128 (f32: with P's first and second piece; bf16: a row tile each).
constexpr uint32_t kTmemO = 256;
constexpr float kLazy = 5.f;  // bf16: how far (log2) a maximum may be overtaken
// P is 2^kPTop at the maximum in use, and loses bits kFarBelow (log2) below it.
template <bool F32>
constexpr float kPTop = F32 ? 15.f : 10.f;
template <bool F32>
constexpr float kFarBelow = F32 ? 34.f : 26.f;
// An element is safe from what is lost if it is this much times the square root
// of the number of tokens: each one's error is at most 2^-25 in P's last piece
// times a value of at most 2^15, either sign, to be 2^-18 (2^-11) of the element
// with a margin of 4.
template <bool F32>
constexpr float kSafe = F32 ? 0x1p-1f : 0x1p3f;
constexpr float kLowUp = 2048.f;  // f32: what P's second piece is scaled by

struct PromptPlan {
    int items_per_list;  // row tiles (or pairs of them) of a (sequence, kv head) at most
    uint32_t k1024;      // two f16 1024, kept from the compiler (see attn_step.cu)
    float* lse2;         // logarithms to base 2 for the weights, or null
    QueryTiles q;        // where the queries' pieces go, if they are wanted
    unsigned* redo_n;    // how many rows are listed to be done again,
    unsigned* redo;      // and which: row * heads + head
    unsigned int* err;
    unsigned redo_room;  // entries that the list has room for: each row once
};

// A row's end: its output, 32 dims at a time, its logarithm, and the list of rows
// to be done again.
template <int D, bool F32, typename T>
struct RowEnd {
    const AttnCall& a;
    const PromptPlan& plan;
    int64_t item;  // row * heads + head
    T* out;
    bool in;
    float sum, inv, least = INFINITY;
    __device__ RowEnd(const AttnCall& a_, const PromptPlan& plan_, int first, int group, int h, int rr, bool in_, float sum_)
        : a(a_), plan(plan_), in(in_), sum(sum_), inv(sum_ == 0.f ? 0.f : 1.f / sum_) {
        const int64_t row = first + (in ? rr / group : 0);
        const int head = h * group + (in ? rr % group : 0);
        item = row * a.heads + head;
        out = static_cast<T*>(a.out) + row * a.out_stride + static_cast<int64_t>(head) * D;
    }
    __device__ __forceinline__ void store32(const float v[32], int q) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                least = fminf(least, fabsf(v[8 * k + e]));
                y[e] = sum == 0.f ? 0.f : v[8 * k + e] * inv;
            }
            if (in) {
                store_o4(out + 32 * q + 4 * k, make_float4(y[0], y[2], y[1], y[3]));
                store_o4(out + 32 * q + 16 + 4 * k, make_float4(y[4], y[6], y[5], y[7]));
            }
        }
    }
    // `coarse`: some tile's values did not fit their pieces.
    __device__ __forceinline__ void finish(float top, float lowest, int n_tiles, bool coarse) {
        if (!in) return;
        const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum) - kPTop<F32>;
        if (a.lse) a.lse[item] = lse2 * kLn2;
        if (plan.lse2) plan.lse2[item] = lse2;
        if (coarse ||
            (lowest < top - kFarBelow<F32> && least < sqrtf(static_cast<float>(n_tiles * kTile)) * kSafe<F32>)) {
            // (Once per row, unless row offsets that go back give a row to two sequences.)
            const unsigned at = atomicAdd(plan.redo_n, 1u);
            if (at < plan.redo_room) plan.redo[at] = static_cast<unsigned>(item);
            else atomicOr(plan.err, kErrRange);
        }
    }
};

struct Bars {
    uint64_t exam, exam_go;
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], pv_done[2];  // f32: of tile i at i % 2; bf16: of row tile m
    uint64_t o_free;
};

template <int D, bool F32, typename T>
__global__ void __launch_bounds__(Shape<D, F32>::kThreads, 1)
    attn_prompt_kernel(KvView c, KvRows r, AttnCall a, PromptPlan plan) {
    using S = Shape<D, F32>;
    constexpr int NB = S::kBlocks;
    constexpr int kM = S::kM;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Bars bar;
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t s_coarse;           // a tile's value scales span more than its pieces do
    __shared__ float row_unit[kM * kTile];  // 1 / (power of two that a row of Q was scaled by)
    __shared__ float key_unit[kRing];       // the same of a key tile, tile i in i % kRing
    __shared__ float value_exp[kRing];          // log2 of the same of a value tile
    __shared__ float key_up[kRing], value_up[kRing];  // the powers of two themselves
    __shared__ __align__(16) uint8_t wild[kRing][32];     // bit t of byte l: token 4 l + t of tile i has a wild value scale
    // f32: what the two softmax threads of a row tell each other, and the collector.
    __shared__ float half_max[F32 ? 2 : 1][S::kHalves][F32 ? kTile : 1];
    __shared__ float row_keep[F32 ? kKeepRing : 1][kTile], row_top[F32 ? kTile : 1];
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* q_sm = base;                             // [kM][pieces]
    uint8_t* k_sm = q_sm + kM * S::kOperand;          // [stages][pieces]
    uint8_t* v_sm = k_sm + S::kStagesK * S::kOperandK;  // [stages][pieces]
    unsigned int* const err = c.err;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (threadIdx.x == 0) {
        mbar_init(&bar.exam, 1);
        mbar_init(&bar.exam_go, kDecodeWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.k_full[i], kDecodeWarps);
            mbar_init(&bar.v_full[i], kDecodeWarps);
            mbar_init(&bar.k_empty[i], 1);
            mbar_init(&bar.v_empty[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4 * S::kHalves);
            mbar_init(&bar.pv_done[i], 1);
        }
        mbar_init(&bar.o_free, 4);
        s_coarse = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();

    // Work item: the longest lists of token tiles first.
    const int lists = c.n_seqs * c.heads;
    const int item = plan.items_per_list - 1 - static_cast<int>(blockIdx.x) / lists;
    const int list = static_cast<int>(blockIdx.x) % lists;
    const int b = list / c.heads, h = list % c.heads;
    int first, count;
    kv_rows(r, b, &first, &count, err);
    const int L = kv_length(c, b, err);
    const int group = a.heads / c.heads;
    const int n_rows = count * group;
    const int row0 = item * kM * kTile;
    if (row0 >= n_rows) return;
    const int base_pos = L - count;
    const int pos_lo = base_pos + row0 / group;
    const int pos_hi = base_pos + min(n_rows - 1, row0 + kM * kTile - 1) / group;
    const int seen_len = max(0, min(L, pos_hi + 1));
    const TileList tiles = tile_list<kTile>(seen_len, max(pos_lo, 0), a.window, a.sinks);
    const int n_tiles = tiles.count;

    // (The GEMM takes its TMEM before it waits for the kernel before it; it cannot
    // do so beside a CTA of this one, which leaves fewer registers than it needs.)
    if (warp == S::kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Q: four threads per row, each a quarter of the dims; a row is scaled by the
    // power of two that takes its largest value to 2^13 .. 2^14.
    const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll 1
    for (int m = 0; m < kM && threadIdx.x < 4 * kTile; ++m) {
        const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
        const int rr = row0 + m * kTile + row;
        const bool in = rr < n_rows;
        const T* q = static_cast<const T*>(a.q) + static_cast<int64_t>(first + (in ? rr / group : 0)) * a.q_stride +
                     static_cast<int64_t>(h * group + (in ? rr % group : 0)) * D;
        constexpr int kEach = D / 32;  // chunks of 8 elements of this thread
        float4 x[kEach][2];
        float amax = 0.f;
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            const int chunk = part * kEach + y, blk = chunk >> 2, k = chunk & 3;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[y][u] = in ? load_q4(q + 32 * blk + 16 * u + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[y][u].x), fabsf(x[y][u].y)),
                                         fmaxf(fabsf(x[y][u].z), fabsf(x[y][u].w))));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        const int up = min(126, 13 - ex);
        const float f = sign * pow2(up);
        if (part == 0) row_unit[m * kTile + row] = pow2(-up);
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            // The order in which a word's quants unpack (decode_block).
            const float v[8] = {x[y][0].x, x[y][0].z, x[y][0].y, x[y][0].w, x[y][1].x, x[y][1].z, x[y][1].y, x[y][1].w};
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v0 = v[2 * e] * f, v1 = v[2 * e + 1] * f;
                const __half2 hh = __floats2half2_rn(v0, v1);
                const float2 back = __half22float2(hh);
                hw[e] = word(hh);
                lw[e] = word(__floats2half2_rn(v0 - back.x, v1 - back.y));
            }
            uint8_t* dst = q_sm + m * S::kOperand + tile_off(row, part * kEach + y);
            *reinterpret_cast<uint4*>(dst) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            if (F32) *reinterpret_cast<uint4*>(dst + S::kPiece) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (plan.q.images) {
        const int64_t tile = query_tile(plan.q, h, first, b, group) + item * kM;
        if (threadIdx.x == 0) bulk_store_1d(plan.q.images + tile * S::kOperand, q_sm, kM * S::kOperand);
        if (threadIdx.x < kM * kTile)
            plan.q.units[tile * kTile + threadIdx.x] = fabsf(a.scale) * kLog2e * row_unit[threadIdx.x];
    }

    if (warp < kSoftmaxWarps) {
        // ---- softmax: this thread's row
        if (F32) regs_down<S::kSoftmaxRegs>();
        else regs_up<S::kSoftmaxRegs>();
        // f32: the warps w and w + 4 share 32 rows, each has half of a tile's columns
        // and half of the dims; bf16: they have a row tile each.
        const int m = F32 ? 0 : warp >> 2, half = F32 ? warp >> 2 : 0;
        constexpr int kChunks = kTile / 32 / S::kHalves;     // of 32 columns, this thread's of a tile
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const int row = 32 * (warp & 3) + lane;
        const int rr = row0 + m * kTile + row;
        const bool in = rr < n_rows;
        const int pos = in ? base_pos + rr / group : -1;
        const int win_lo = a.window > 0 ? pos - a.window + 1 : 0;  // tokens from here on, and below sinks
        const int wr0 = row0 + m * kTile + 32 * (warp & 3);        // the warp's rows' extreme positions
        const int w_lo = base_pos + wr0 / group, w_hi = base_pos + (wr0 + 31) / group;
        const float unit = fabsf(a.scale) * kLog2e * row_unit[m * kTile + row];
        const uint32_t t_o = tmem + lanes + kTmemO + m * 128;  // (bf16)
        float mx_used = -INFINITY, sum = 0.f;
        float lowest = INFINITY;  // of the row's scores (with the value tile's exponent)
        bool ok = true;
        // f32: what the row's other thread has.
        auto other = [&](float x, int buf) {
            half_max[buf][half][row] = x;
            named_barrier_sync(1 + (warp & 3), 64);
            return half_max[buf][half ^ 1][row];
        };
#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i) {
            const int buf = F32 ? i & 1 : m;
            const uint32_t t_s = tmem + lanes + buf * kTile + half * 64;
            // (After a wait that gave up, none is begun: the two warps of a row go on
            // through their barriers to the end.)
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.s_full[buf], F32 ? (i >> 1) & 1 : i & 1, err));
            tc_fence_after();
            const int key0 = tiles.at(i) * kTile;
            const float f = fmaxf(unit * key_unit[i % kRing], 0x1p-100f);  // (not 0: it meets -infinity)
            const float v_exp = value_exp[i % kRing];
            const uint8_t* wild_i = wild[i % kRing];
            bool any_wild;
            {
                const uint4 w0 = *reinterpret_cast<const uint4*>(wild_i);
                const uint4 w1 = *reinterpret_cast<const uint4*>(wild_i + 16);
                any_wild = (w0.x | w0.y | w0.z | w0.w | w1.x | w1.y | w1.z | w1.w) != 0;
            }
            const bool masked = any_wild || key0 + kTile > min(w_lo + 1, L) ||
                                (a.window > 0 && key0 <= w_hi - a.window && key0 + kTile > a.sinks);
            // Tokens that the row does not see become -infinity, those that it sees
            // and whose values are not finite NaN, in TMEM, where there are any.
            const int k0 = key0 + half * 64;
            float mn = INFINITY;
            if (masked) {
                const int k_end = min(pos, L - 1) + 1 - k0, k_lo = win_lo - k0, k_sink = a.sinks - k0;
                auto below = [](int n) -> uint32_t { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; };
#pragma unroll 1
                for (int q = 0; q < kChunks; ++q) {
                    const uint32_t sees = below(k_end - 32 * q) & (~below(k_lo - 32 * q) | below(k_sink - 32 * q));
                    float v[32];
                    tmem_ld32(t_s + 32 * q, v);
                    tc_wait_ld();
                    if (any_wild) {
                        uint32_t bad = 0;
#pragma unroll 1
                        for (int y = 0; y < 8; ++y)
                            bad |= static_cast<uint32_t>(wild_i[16 * half + 8 * q + y]) << (4 * y);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if ((bad >> e) & 1u) v[e] = NAN;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if ((sees >> e) & 1u) mn = fminf(mn, v[e]);
                        else v[e] = -INFINITY;
                    }
                    tmem_st32(t_s + 32 * q, v);
                }
                tc_wait_st();
            }
            // f32: two passes over the row's scores in TMEM, its maximum, then P;
            // bf16: the scores stay in registers between the two.
            {
                constexpr int kHeld = F32 ? 32 : 64;
                float v[kHeld];
                float mx = -INFINITY, low = INFINITY;
#pragma unroll 1
                for (int q = 0; q < kTile / S::kHalves / kHeld; ++q) {
#pragma unroll
                    for (int y = 0; y < kHeld; y += 32) tmem_ld32(t_s + kHeld * q + y, v + y);
                    tc_wait_ld();
                    float mx2 = -INFINITY, low2 = INFINITY;
#pragma unroll
                    for (int e = 0; e < kHeld; e += 4) {
                        mx = fmaxf(fmaxf(mx, v[e]), v[e + 1]);
                        mx2 = fmaxf(fmaxf(mx2, v[e + 2]), v[e + 3]);
                        low = fminf(fminf(low, v[e]), v[e + 1]);
                        low2 = fminf(fminf(low2, v[e + 2]), v[e + 3]);
                    }
                    mx = fmaxf(mx, mx2);
                    low = fminf(low, low2);
                }
                if (!masked) mn = low;
                lowest = fminf(lowest, fmaf(mn, f, v_exp));
                mx = fmaf(mx, f, v_exp);
                if (F32) {
                    const float next = fmaxf(mx_used, fmaxf(mx, other(mx, i & 1)));
                    const float keep = exp2_approx(mx_used - (next == -INFINITY ? 0.f : next));
                    mx_used = next;
                    sum *= keep;
                    if (half == 0) row_keep[F32 ? i % kKeepRing : 0][row] = keep;  // what the sums so far are scaled by
                } else {
                    // The maximum in use follows only where it is overtaken by 2^5.
                    const bool grow = mx > mx_used + kLazy;
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float next = grow ? mx : mx_used;
                        const float keep = grow ? exp2_approx(mx_used - next) : 1.f;
                        mx_used = next;
                        sum *= keep;
                        if (i > 0) {
#pragma unroll 1
                            for (int q = 0; q < D / 32; ++q) {
                                float w[32];
                                tmem_ld32(t_o + 32 * q, w);
                                tc_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) w[e] *= keep;
                                tmem_st32(t_o + 32 * q, w);
                            }
                            tc_wait_st();
                        }
                    }
                }
                const float off = (mx_used == -INFINITY ? 0.f : mx_used) - v_exp - kPTop<F32>;
                const float2 f2 = make_float2(f, f), off2 = make_float2(-off, -off);
                float2 part[2] = {};
#pragma unroll 1
                for (int q = 0; q < kTile / S::kHalves / kHeld; ++q) {
#pragma unroll
                    for (int y = 0; y < kHeld; y += 32) tmem_ld32(t_s + kHeld * q + y, v + y);
                    tc_wait_ld();
                    uint32_t hi[kHeld / 2], lo[16];
#pragma unroll
                    for (int e = 0; e < kHeld; e += 2) {
                        const float2 x = fma2(make_float2(v[e], v[e + 1]), f2, off2);
                        const float2 pp = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        part[e / 2 & 1] = add2(part[e / 2 & 1], pp);
                        const __half2 hw = __floats2half2_rn(pp.x, pp.y);
                        hi[e / 2] = word(hw);
                        if (F32) {
                            const float2 back = __half22float2(hw);
                            lo[e / 2 & 15] = word(__floats2half2_rn((pp.x - back.x) * kLowUp, (pp.y - back.y) * kLowUp));
                        }
                    }
                    if (F32) {
                        tmem_st16(t_s + 32 * q, hi);
                        tmem_st16(t_s + 32 * q + 16, lo);
                    } else {
#pragma unroll
                        for (int y = 0; y < kHeld / 2; y += 16) tmem_st16(t_s + kHeld / 2 * q + y, hi + y);
                    }
                }
                sum = fmaf((part[0].x + part[0].y) + (part[1].x + part[1].y), exp2_approx(-v_exp), sum);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[buf]);
        }
        // A row's output (columns in the order the quants unpack) and logarithm.
        if constexpr (F32) {
            sum += other(sum, n_tiles & 1);
            lowest = fminf(lowest, other(lowest, (n_tiles + 1) & 1));
            // To the collector: its barrier comes after these.
            if (half == 0) {
                row_top[row] = mx_used;
                half_max[n_tiles & 1][0][row] = sum;
                half_max[n_tiles & 1][1][row] = lowest;
            }
            named_barrier_sync(5, (kSoftmaxWarps + S::kCollectWarps) * 32);
        } else {
            if (n_tiles > 0 && ok)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.pv_done[m], (n_tiles - 1) & 1, err));
            tc_fence_after();
            RowEnd<D, false, T> end(a, plan, first, group, h, rr, in, sum);
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                float v[32];
                if (n_tiles > 0) {
                    tmem_ld32(t_o + 32 * q, v);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                end.store32(v, q);
            }
            end.finish(mx_used, lowest, n_tiles, s_coarse != 0);
        }
    } else if (warp < kSoftmaxWarps + kDecodeWarps) {
        // ---- decode: cells -> swizzled tiles.  A thread has a token and every other
        // block of it (D = 64 and bf16: one at most); what it needs next is on its
        // way while it unpacks.
        regs_down<S::kDecodeRegs>();
        const int dt = threadIdx.x - kSoftmaxWarps * 32;
        const int tok = dt & (kTile - 1), blk0 = dt / kTile;
        constexpr int kStride = kDecodeWarps * 32 / kTile, kTurns = NB / kStride;
        bool ok = true;
        auto pos_at = [&](int i) { return i < n_tiles ? tiles.at(i) * kTile + tok : seen_len; };
        auto page_at = [&](int i) {  // of this token in tile i
            const int p = pos_at(i);
            return p < seen_len ? kv_page_id(c, b, p) : 0;
        };
        auto cell_at = [&](int i, int id) -> int64_t {
            const int p = pos_at(i);
            return p < seen_len ? kv_cell_in(c, id, h, p, err) : -1;
        };
        // What this thread unpacks next of a tile's keys (f32: or values) and values.
        const int in_cell = blk0 * 256 + (tok & 15) * 16, in_scales = cell_scales(D) + ((tok & 15) * NB + blk0) * 2;
        struct Blocks {
            uint4 q[kTurns];
            uint32_t sc[kTurns];
        };
        auto fetch = [&](Blocks& x, const uint8_t* pool, int64_t off) {
#pragma unroll
            for (int y = 0; y < kTurns; ++y) {
                x.q[y] = make_uint4(0, 0, 0, 0);
                x.sc[y] = 0;
                if (off >= 0) {
                    x.q[y] = *reinterpret_cast<const uint4*>(pool + off + in_cell + y * kStride * 256);
                    x.sc[y] = *reinterpret_cast<const uint16_t*>(pool + off + in_scales + y * kStride * 2);
                }
            }
        };
        auto unpack = [&](auto two, const Blocks& x, bool v, float f, uint8_t* hi) {
#pragma unroll
            for (int y = 0; y < kTurns; ++y) {
                // Values that are not finite (NaN then comes with the scores): 0.
                const float d = v && (x.sc[y] & 0x7C00u) == 0x7C00u ? 0.f : f16_bits_to_float(x.sc[y]) * f;
                decode_block<decltype(two)::value>(x.q[y], d, tok, blk0 + y * kStride, hi, hi + S::kPiece, plan.k1024);
            }
        };
        if constexpr (!F32) {
            // Keys a tile ahead of values.
            Blocks k, v;
            int64_t off = cell_at(0, page_at(0)), off_next = -1;  // of this thread's token in tile i, and in tile i + 1
            fetch(k, c.k, off);
            fetch(v, c.v, off);
            int page = page_at(1);
#pragma unroll 1
            for (int i = 0; i <= n_tiles; ++i) {
                if (i < n_tiles) {
                    const int at = i % S::kStagesK;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.exam, i & 1, err));
                    if (ok && lane == 0) mbar_arrive(&bar.exam_go);
                    if (ok && i >= S::kStagesK) ok = mbar_wait_bounded(&bar.k_empty[at], (i / S::kStagesK - 1) & 1, err);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    const Blocks now = k;
                    off_next = cell_at(i + 1, page);
                    page = page_at(i + 2);
                    fetch(k, c.k, off_next);
                    unpack(std::true_type{}, now, false, key_up[i % kRing], k_sm + at * S::kOperandK);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.k_full[at]);
                }
                if (i > 0) {
                    const int at = (i - 1) % S::kStagesV;
                    if (i > S::kStagesV) ok = mbar_wait_bounded(&bar.v_empty[at], ((i - 1) / S::kStagesV - 1) & 1, err);
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    const Blocks now = v;
                    fetch(v, c.v, off);
                    unpack(std::false_type{}, now, true, value_up[(i - 1) % kRing], v_sm + at * S::kOperand);
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.v_full[at]);
                }
                off = off_next;
            }
        } else {
            int64_t off_v = -1, off_k = cell_at(0, page_at(0));  // of the tile whose values come next, and of the one after
            Blocks x;
            fetch(x, c.k, off_k);
            int page_k = page_at(1);  // of the keys to fetch after those
            // Keys one tile ahead of values: keys 0, keys 1, values 0, keys 2, ...
            // One body for keys and values: the code of all roles together has to stay
            // in the instruction cache.
#pragma unroll 1
            for (int step = 0; step < 2 * n_tiles; ++step) {
                const bool v = step > 0 && ((step & 1) == 0 || step == 2 * n_tiles - 1);
                const int i = v ? (step - 1) >> 1 : (step + 1) >> 1;
                static_assert(!F32 || (S::kStagesK == 1 && S::kStagesV == 1), "one tile of each");
                if (!v) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.exam, i & 1, err));
                    if (ok && lane == 0) mbar_arrive(&bar.exam_go);
                }
                if (ok && i >= 1) ok = mbar_wait_bounded(v ? bar.v_empty : bar.k_empty, (i - 1) & 1, err);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                const float f = v ? value_up[i % kRing] : key_up[i % kRing];
                uint8_t* hi = v ? v_sm : k_sm;
                const Blocks now = x;
                // The next step: keys i + 1 (i + 2 after values i), or values i - 1.
                if (v || step == 0) {
                    off_v = off_k;
                    off_k = cell_at(i + (v ? 2 : 1), page_k);
                    if (step + 1 == 2 * n_tiles - 1) fetch(x, c.v, off_v);  // no more keys
                    else fetch(x, c.k, off_k);
                } else {
                    fetch(x, c.v, off_v);
                    page_k = page_at(i + 1);
                }
                unpack(std::true_type{}, now, v, f, hi);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(v ? bar.v_full : bar.k_full);
            }
        }
    } else if (warp < S::kIssuer) {
        // ---- collectors (f32): a row's sums in registers, o = o keep + P V tile by tile.
        regs_up<S::kCollectRegs>();
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const int row = 32 * (warp & 3) + lane, rr = row0 + row;
        float o[F32 ? D : 1];
#pragma unroll
        for (int e = 0; e < (F32 ? D : 1); ++e) o[e] = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i) {
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.pv_done[i & 1], (i >> 1) & 1, err));
            if (!ok) break;
            tc_fence_after();
            const float keep = row_keep[F32 ? i % kKeepRing : 0][row];
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                float v[16], w[16];
                tmem_ld16(tmem + lanes + kTmemO + 16 * x, v);
                tmem_ld16(tmem + lanes + kTmemO + 128 + 16 * x, w);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float& y = o[F32 ? 16 * x + e : 0];
                    y = fmaf(y, keep, fmaf(w[e], 1.f / kLowUp, v[e]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_free);
        }
        named_barrier_sync(5, (kSoftmaxWarps + S::kCollectWarps) * 32);
        if constexpr (F32) {
            RowEnd<D, true, T> end(a, plan, first, group, h, rr, rr < n_rows, half_max[n_tiles & 1][0][row]);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) end.store32(o + 32 * x, x);
            end.finish(row_top[row], half_max[n_tiles & 1][1][row], n_tiles, s_coarse != 0);
        }
    } else {
        regs_down<S::kOtherRegs>();
    if (warp == S::kIssuer) {
        // ---- MMA issue
        if (n_tiles > 0) {
            const uint32_t lead = elect_one();
            constexpr uint32_t id_s = idesc_f16(kTile, false), id_o = idesc_f16(D, true);
            bool ok = true;
            auto scores = [&](int i, int m) {
                const int stage = i % S::kStagesK;
                ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.k_full[stage], (i / S::kStagesK) & 1, err));
                if (!ok) return;
                tc_fence_after();
                const uint32_t t_s = tmem + (F32 ? i & 1 : m) * kTile;
                const uint32_t q0 = smem_addr(q_sm + m * S::kOperand), k0 = smem_addr(k_sm + stage * S::kOperandK);
                constexpr int kProducts = F32 ? 3 : 2;  // (low x high,) high x low, high x high
#pragma unroll 1
                for (int p = 0; p < kProducts; ++p) {
                    const uint64_t da = desc_base(q0 + (F32 && p == 0 ? S::kPiece : 0), 16);
                    const uint64_t db = desc_base(k0 + (p == kProducts - 2 ? S::kPiece : 0), 16);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t o = static_cast<uint64_t>((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
                        mma_ss(t_s, da + o, db + o, id_s, (p | kk) != 0, lead);
                    }
                }
                mma_commit(&bar.s_full[F32 ? i & 1 : m], lead);
                if (m == kM - 1) mma_commit(&bar.k_empty[stage], lead);
            };
            auto output = [&](int i, int m) {
                const int stage = i % S::kStagesV, buf = F32 ? i & 1 : m;
                const uint32_t p_phase = F32 ? (i >> 1) & 1 : i & 1;
                // P, V, and (f32) the accumulators that the collectors have read.
                ok = ok && __all_sync(0xFFFFFFFFu, wait_all(&bar.p_full[buf], p_phase, &bar.v_full[stage],
                                                            (i / S::kStagesV) & 1, F32 && i > 0 ? &bar.o_free : &bar.p_full[buf],
                                                            F32 && i > 0 ? (i - 1) & 1 : p_phase, err));
                if (!ok) return;
                tc_fence_after();
                const uint32_t v0 = smem_addr(v_sm + stage * S::kOperand);
                constexpr int kProducts = F32 ? 3 : 1;  // low x high apart, high x low, high x high
#pragma unroll 1
                for (int p = 0; p < kProducts; ++p) {
                    const uint32_t t_p = tmem + buf * kTile + (F32 && p == 0 ? 16 : 0);
                    const uint32_t t_o = tmem + kTmemO + (F32 ? (p == 0 ? 128 : 0) : m * 128);
                    // V is [token][dim]: rows are the contraction, 64-dim columns kTile * 128 bytes apart.
                    const uint64_t db = desc_base(v0 + (F32 && p == 1 ? S::kPiece : 0), kTile * 128);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_ts(t_o, t_p + (F32 ? (kk >> 1) * 32 + (kk & 1) * 8 : 8 * kk),
                               db + (static_cast<uint64_t>(kk * 16 * 128) >> 4), id_o,
                               (F32 ? (p == 2) | kk : i | kk) != 0, lead);
                }
                mma_commit(&bar.pv_done[buf], lead);
                if (m == kM - 1) mma_commit(&bar.v_empty[stage], lead);
            };
#pragma unroll 1
            for (int x = -S::kAhead * kM; x < kM * n_tiles && ok; ++x) {  // x = kM i + m
                const int i = (x + S::kAhead * kM) / kM - S::kAhead, m = (x + S::kAhead * kM) % kM;
                if (i >= 0) output(i, m);
                if (i + S::kAhead < n_tiles) scores(i + S::kAhead, m);
            }
        }
    } else if (warp == S::kIssuer + 1) {
        // ---- examiner: what the decode warps and the softmax need to know of a
        // tile's scales.  Lane l looks at tokens 4 l .. 4 l + 3 (of one cell).
        constexpr int kWords = 2 * NB;  // of four tokens' scales
        uint32_t x[kWords], v[kWords];
        auto fetch = [&](int i) {
            const int p = i < n_tiles ? tiles.at(i) * kTile + 4 * lane : seen_len;
            const int64_t off = p < seen_len ? kv_cell(c, b, h, p, err) : -1;
            const int64_t at = off + cell_scales(D) + (p & 15) * 2 * NB;
#pragma unroll
            for (int e = 0; e < kWords; e += 4) {
                uint4 y = make_uint4(0, 0, 0, 0), z = y;
                if (off >= 0) {
                    y = *reinterpret_cast<const uint4*>(c.k + at + 4 * e);
                    z = *reinterpret_cast<const uint4*>(c.v + at + 4 * e);
                }
                x[e] = y.x, x[e + 1] = y.y, x[e + 2] = y.z, x[e + 3] = y.w;
                v[e] = z.x, v[e + 1] = z.y, v[e + 2] = z.z, v[e + 3] = z.w;
            }
        };
        fetch(0);
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n_tiles && ok; ++i) {
            const int left = seen_len - tiles.at(i) * kTile - 4 * lane;  // of this lane's tokens that count
            uint32_t top = 0, top_v = 0, low_v = 0xFFFFu, bad = 0;  // (low_v: the smallest that is not 0)
#pragma unroll
            for (int e = 0; e < kWords; ++e) {
                const int u = e / (NB / 2);
                const uint32_t a0 = x[e] & 0x7FFFu, a1 = (x[e] >> 16) & 0x7FFFu;
                const uint32_t v0 = v[e] & 0x7FFFu, v1 = (v[e] >> 16) & 0x7FFFu;
                if (u < left) {
                    top = max(top, max(a0 < 0x7C00u ? a0 : 0u, a1 < 0x7C00u ? a1 : 0u));
                    top_v = max(top_v, max(v0 < 0x7C00u ? v0 : 0u, v1 < 0x7C00u ? v1 : 0u));
                    low_v = min(low_v, min(v0 ? v0 : 0xFFFFu, v1 ? v1 : 0xFFFFu));
                    if (v0 >= 0x7C00u || v1 >= 0x7C00u) bad |= 1u << u;
                }
            }
            fetch(i + 1);
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            top_v = __reduce_max_sync(0xFFFFFFFFu, top_v);
            low_v = __reduce_min_sync(0xFFFFFFFFu, low_v);
            // The decode warps have begun tile i - 1, so at most kRing tiles are in use.
            if (i > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&bar.exam_go, (i - 1) & 1, err));
            wild[i % kRing][lane] = static_cast<uint8_t>(bad);
            if (lane == 0) {
                const int up = 26 - max(1, static_cast<int>(top >> 10));      // largest scale to 2^11 .. 2^12
                const int up_v = 26 - max(1, static_cast<int>(top_v >> 10));
                // Bits of n d below 2^-24: there are some if a scale's last bit goes below it.
                if (max(1, static_cast<int>(low_v >> 10)) < 1 - up_v) s_coarse = 1;
                key_up[i % kRing] = pow2(up);
                key_unit[i % kRing] = pow2(-up);
                value_up[i % kRing] = pow2(up_v);
                value_exp[i % kRing] = static_cast<float>(-up_v);
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&bar.exam);
        }
    }
    }

    if (plan.q.images && threadIdx.x == 0) bulk_store_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == S::kIssuer) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int D, bool F32, typename T>
cudaError_t launch_prompt(const KvView& c, const KvRows& r, const AttnCall& a, float* lse2, const QueryTiles& qt,
                          unsigned* redo_n, unsigned* redo, cudaStream_t stream) {
    using S = Shape<D, F32>;
    static SmemOnce once;
    cudaError_t err = once.set(attn_prompt_kernel<D, F32, T>, S::kSmem, S::kRegs);
    if (err != cudaSuccess) return err;
    const int64_t rows = static_cast<int64_t>(r.max_q) * (a.heads / c.heads);
    PromptPlan p = {};
    p.items_per_list = static_cast<int>((rows + S::kM * kTile - 1) / (S::kM * kTile));
    p.k1024 = 0x64006400u;
    p.lse2 = lse2;
    p.q = qt;
    p.redo_n = redo_n;
    p.redo = redo;
    p.err = c.err;
    p.redo_room = static_cast<unsigned>(static_cast<int64_t>(r.n_tokens) * a.heads);
    const int64_t grid = static_cast<int64_t>(p.items_per_list) * c.n_seqs * c.heads;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    note_launch();
    return launch_pdl(attn_prompt_kernel<D, F32, T>, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), S::kSmem, stream,
                      c, r, a, p);
}

}  // namespace

bool attn_prompt_takes(const KvView& c) { return c.dim == 64 || c.dim == 128; }

cudaError_t launch_attn_prompt(const KvView& c, const KvRows& r, const AttnCall& a, float* lse2, const QueryTiles& qt,
                               unsigned* redo_n, unsigned* redo, cudaStream_t stream) {
    if (c.dim == 64)
        return a.type == KvType::kF32 ? launch_prompt<64, true, float>(c, r, a, lse2, qt, redo_n, redo, stream)
                                      : launch_prompt<64, false, __nv_bfloat16>(c, r, a, lse2, qt, redo_n, redo, stream);
    return a.type == KvType::kF32 ? launch_prompt<128, true, float>(c, r, a, lse2, qt, redo_n, redo, stream)
                                  : launch_prompt<128, false, __nv_bfloat16>(c, r, a, lse2, qt, redo_n, redo, stream);
}

}  // namespace qm
