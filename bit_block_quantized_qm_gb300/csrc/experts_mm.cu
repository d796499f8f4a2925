// The experts' products (qm_experts_q4_0) on tcgen05 tensor cores.
//
// The weights are the 128-row operand and the token rows the columns, so a tile is
// 256 weight rows (128 of gate and 128 of up, or 256 of one matrix) by up to 128 rows of
// one expert, rounded up to 16.
//
// Bound: many rows, what L2 gives an SM, some 32 bytes a cycle, for token rows that every CTA loads for
// itself (8192 rows through 8 experts of 14336 x 4096, three products: 2.46 ms in all, 1170 TFLOP/s; an
// instruction with 128 columns takes 64 cycles, one with 16 nine); fewer, the unpacking: 8 weights of
// each lane of a warp take 21 cycles, fp16 and integer instructions going at half rate, and a unit (256
// rows by 256 of K) 1340, where memory would bring one every 1570.
//
//   D[w][t] = sum_k (q_wk - 8) d_wb  x_tk
//
// Operands are f16.  A weight is (q - 8) d 2^8, at most 15 significant bits: its f16
// rounding, and for f32 rows the exact rest as a second piece.  The 2^8 keeps the rest of
// scales from 2^-10 up out of f16's subnormal numbers.  Token rows come as f16 pieces of
// x times a power of two that takes the row's largest value to 2^13 .. 2^14 (one piece
// holds a bf16 row's 8 bits, two an f32 row's 22).  f32 rows take three products, the
// fourth being 2^-22 of the first.  Tensor cores cut sums off instead of rounding them, each
// addition by 2^-26 of the sum and more (256 of them 4e-6), so f32 rows' large products have
// sums apart from the small ones', and go to registers after every unit (16 additions) to be
// added there; bf16 rows' stay in TMEM.  The element order inside a block of 32 is that in
// which quants unpack, in weights and pieces alike.
//
// Weights never lie unpacked in shared memory: raw Q4_0 rows come by TMA, 256 elements
// (144 bytes) at a time, a thread unpacks 64 elements of its row into registers and
// stores them to TMEM, from where the tensor cores take them.  Per CTA: 16 warps
// unpack (and write the outputs), one loads weights, one token pieces, one issues the
// products.
//
// Rows whose length is no multiple of 256 start at odd places, which TMA does not take
// (16 bytes).  G = 16 / gcd(16, row bytes) rows together are a multiple of it: the matrix
// is seen as groups of G rows, the rows of each number within the group are one box that
// starts at the 16-byte boundary below, and the unpacking threads shift.
//
// Work: whole tiles, a CTA each, as long as they fill all CTAs; the units (256 elements of
// K) of those left over are dealt out evenly, where that saves more than it costs, and the CTA that comes last to a shared tile
// adds its parts in the CTAs' order.
//
// Sums that come out infinite or NaN (a scale of 32 and more overflows f16) are left so, and
// taken again by the kernels that read them.
//
// No register may spill: with most of the SM's memory shared memory, what is spilled comes back from L2,
// and each reload costs some 300 cycles (bf16 rows' products went at 817 instead of 1065 TFLOP/s; f32 rows'
// tiles of 64 keep in shared memory what they need once a tile, which took 500 rows from 1211 to 1187 us).
//
// Every wait is bounded; a wait that gives up sets the device error word.
#include <type_traits>

#include "experts.cuh"
#include "tcgen05.cuh"

namespace qm {

namespace {

constexpr int kHalf = kExpertHalf;
constexpr int kDecodeWarps = 16;
constexpr int kRawWarp = 16, kTokenWarp = 17, kMmaWarp = 18;  // and 19: the products of a half each
constexpr int kThreads = 20 * 32;
constexpr float kWeightUnit = 0x1p-8f;

template <bool F32, int TOKENS, bool WIDE>
struct Cfg {
    static constexpr int kTokens = TOKENS;  // token rows of a tile
    // Columns of a half's sums.  F32: the second pieces' products are columns of their own beside the
    // first ones', so that a product with both is one instruction.
    static constexpr int kColumns = F32 ? 2 * kTokens : kTokens;
    static constexpr int kSums = F32 || kTokens > 32 ? 1 : 2;     // sets of sums in TMEM
    static constexpr int kChunk = kTokens > 32 ? 16 : 8;          // columns of sums that a thread has at a time
    // The warps that unpack and keep sums get registers from the others: what the CTA has at launch,
    // 20 * 96 a lane, is 16 * 112 + 4 * 32.
    static constexpr bool kMoveRegs = F32 && kTokens > 32;
    static constexpr int kLaunchRegs = 96, kDecodeRegs = 112, kOtherRegs = 32;
    static_assert(kDecodeWarps * kDecodeRegs + 4 * kOtherRegs <= 20 * kLaunchRegs, "a warp would wait for ever");
    // Sharing the tiles left over saves ku (ctas - rest) / ctas units, and the joining costs what this many do
    // (16 experts of 4096 x 4096, 64 bf16 rows each: shared above 4 saved 181 us, above 9 177; 2 of 8192 x 2048,
    // 512 each: 156 and 145; 64 of 2048 x 1408, 32 f32 rows each: above 1 236, above 6 250).
    static constexpr int kJoinUnits = F32 ? 2 : 9;
    // Stages of unpacked weights, 128 columns of TMEM (bf16 rows: 128 elements, f32 rows: 64), and of
    // the token rows that they meet.  Long ones, because an issuing warp takes 300 cycles and more for a
    // stage besides its products.
    static constexpr int kStageK = F32 ? 64 : 128;
    static constexpr int kTmemA = kSums * 2 * kColumns;  // (the sums come first)
    static constexpr int kStages = (512 - kTmemA) / 128;
    static constexpr int kPitch = WIDE ? 176 : 144;  // bytes of a raw row in shared memory, an odd number of 16s
    static constexpr int kRawBytes = 2 * kHalf * kPitch;
    static constexpr int kTokenBytes = 2 * kTokens * 128;  // bf16 rows: two panels of 64 elements, f32 rows: two pieces
    // Narrow tiles: a stage of weights and its token rows have one barrier.  Wide ones of bf16 rows: the
    // token rows have stages of their own, further ahead (4096 tokens through 2 of 8 of 14336 x 4096: 2460 us
    // against 2530 with one barrier).
    static constexpr bool kJoint = F32 || kTokens <= 32;
    static constexpr int kTokenStages = kJoint ? kStages : WIDE ? 2 : 3;
    static constexpr int kRawStages = WIDE || !kJoint ? 3 : 4;
    static constexpr int kSmem = kRawStages * kRawBytes + kTokenStages * kTokenBytes + 1024;
    static_assert(kTmemA % 128 == 0 && kStages >= 2, "room for the weights");
};

struct Barriers {
    uint64_t raw_full[4], raw_empty[4];
    uint64_t tok_full[3], tok_empty[3];
    uint64_t full[3], empty[3];
    uint64_t acc_full[2], acc_empty[2];
};

using qm::warp_wait;
__device__ __forceinline__ bool warp_wait(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, unsigned int* err) {
    for (uint32_t i = 0; i < kMaxWaitPolls; ++i) {
        const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
        if (__all_sync(kAll, x && y)) return true;
    }
    atomicOr(err, kErrWaitTimeout);
    return false;
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ldn(uint32_t addr, float (&v)[16]) { tmem_ld16(addr, v); }
__device__ __forceinline__ void tmem_ldn(uint32_t addr, float (&v)[8]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}

// Quant words K0 .. K0 + N - 1 (of 4) of a block of a weight row, number `b` of the two that words 0 .. 8
// (36 bytes) hold, in the order in which quants unpack; F32: with the second pieces.
template <bool F32, int K0 = 0, int N = 4>
__device__ __forceinline__ void unpack_block(const uint32_t (&w)[9], int b, uint32_t k1024, uint32_t* h, uint32_t* l) {
    const uint32_t d_bits = __byte_perm(b ? w[4] : w[0], 0, b ? 0x3232 : 0x1010);
    const __half2 d = __hmul2(half2_of(d_bits), half2_of(0x5C005C00u));  // times 2^8
    const __half2 m1032 = half2_of(0xE408E408u), sixteenth = half2_of(0x2C002C00u), m72 = half2_of(0xD480D480u);
#pragma unroll
    for (int k = K0; k < K0 + N; ++k) {
        const uint32_t q = b ? w[5 + k] : __byte_perm(w[k], w[k + 1], 0x5432);
        const uint32_t y = q >> 8;
        const __half2 n[4] = {__hadd2(half2_of((q & 0x000F000Fu) | k1024), m1032),
                              __hadd2(half2_of((y & 0x000F000Fu) | k1024), m1032),
                              __hfma2(half2_of((q & 0x00F000F0u) | k1024), sixteenth, m72),
                              __hfma2(half2_of((y & 0x00F000F0u) | k1024), sixteenth, m72)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 x = __hmul2(n[e], d);
            h[4 * (k - K0) + e] = word(x);
            if (F32) l[4 * (k - K0) + e] = word(__hfma2(n[e], d, __hneg2(x)));
        }
    }
}

// The nine words of a unit's 64 elements number KS.
template <int KS, bool WIDE>
__device__ __forceinline__ void load_words(const uint8_t* row, int shift, uint32_t (&w)[9]) {
    if constexpr (!WIDE) {
        // Bytes 36 KS .. + 35 lie KS words into the 48 bytes from the 16-byte boundary below.
        uint32_t v[12];
        constexpr int kFrom = 36 * KS & ~15;
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(row + kFrom);
        *reinterpret_cast<uint4*>(v + 4) = *reinterpret_cast<const uint4*>(row + kFrom + 16);
        *reinterpret_cast<uint4*>(v + 8) = *reinterpret_cast<const uint4*>(row + kFrom + 32);
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = v[i + KS];
    } else {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row + 36 * KS + (shift & ~3));
        const uint32_t sel = shift & 2 ? 0x5432 : 0x3210;
        uint32_t v = p[0];
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const uint32_t next = p[i + 1];
            w[i] = __byte_perm(v, next, sel);
            v = next;
        }
    }
}

template <bool F32, int TOKENS, bool DOWN, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    experts_mm_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                      const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
                      const ExpertsMm m) {
    using C = Cfg<F32, TOKENS, WIDE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* tok = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint8_t* raw = tok + C::kTokenStages * C::kTokenBytes;
    __shared__ Barriers bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int tiles_before[1024 + 1];  // token tiles of all lower experts
    __shared__ int rows_before[1024 + 1];   // their sorted rows
    __shared__ alignas(16) float units[3][C::kTokens];  // of the columns of this tile, the one before and the one after
    __shared__ int last_of_tile;
    __shared__ Plan plan;  // (not in registers, of which there are few)
    // What an unpacking warp needs once a tile.  All lanes write the same, and meet between writing and reading.
    struct Seldom {
        Cursor cur;
        int tile, units, n;  // of the tile whose outputs are due
        uint32_t buf;
    };
    __shared__ Seldom seldom_of[kDecodeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned int* const err = m.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], kDecodeWarps);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar.full[i], C::kJoint ? 9 : 8);  // the warps that unpack, and the token rows
            mbar_init(&bar.empty[i], 2);  // the products of both halves
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar.tok_full[i], 1);
            mbar_init(&bar.tok_empty[i], 2);  // the products of both halves
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.acc_full[i], 2);
            mbar_init(&bar.acc_empty[i], kDecodeWarps);
        }
        fence_barrier_init();
    }
    if (warp == kRawWarp && lane == 0) {
        prefetch_tensormap(&map_w0);
        prefetch_tensormap(&map_w1);
        prefetch_tensormap(&map_hi);
        if (F32) prefetch_tensormap(&map_lo);
    }
    grid_dependency_wait();
    // (After the wait, so that no kernel before this one can be short of TMEM; before
    // the next one may start, so that this one never is.)
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 0) {
        int sum = 0;
        for (int e0 = 0; e0 < m.n; e0 += 32) {
            const int e = e0 + lane;
            const int end = e < m.n ? m.starts[e + 1] : 0, count = e < m.n ? end - m.starts[e] : 0;
            int v = (count + C::kTokens - 1) / C::kTokens;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kAll, v, d);
                if (lane >= d) v += o;
            }
            if (e < m.n) tiles_before[e + 1] = sum + v, rows_before[e + 1] = end;
            sum += __shfl_sync(kAll, v, 31);
        }
        if (lane == 0) tiles_before[0] = rows_before[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_launch_dependents();
    const uint32_t tmem = tmem_slot;

    const bool two = m.half[0] != m.half[1];  // gate and up (a flag would cost registers: f32 rows' tiles of 64 would spill)
    const int block_rows = two ? kHalf : 2 * kHalf;
    const int blocks = (m.rows + block_rows - 1) / block_rows;
    if (threadIdx.x == 0) {
        Plan p;
        p.tiles = tiles_before[m.n] * blocks;
        p.ctas = gridDim.x;
        p.cta = blockIdx.x;
        p.ku = (m.K + 255) / 256;
        p.full = p.tiles / p.ctas * p.ctas;
        p.rest = p.tiles - p.full;
        p.each = p.rest * p.ku / p.ctas;
        p.more = p.rest * p.ku - p.each * p.ctas;
        p.share = p.rest > 0 && p.ku * (p.ctas - p.rest) > C::kJoinUnits * p.ctas;
        plan = p;
    }
    __syncthreads();
    auto place = [&](int tile) {
        const int tt = tile / blocks;
        int lo = 0, hi = m.n;  // the first expert with tiles_before[e + 1] > tt
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tiles_before[mid + 1] <= tt) lo = mid + 1;
            else hi = mid;
        }
        Place p;
        p.expert = uniform(lo);
        p.block = tile - tt * blocks;
        p.p0 = uniform(rows_before[lo] + (tt - tiles_before[lo]) * C::kTokens);
        p.n = uniform(min(C::kTokens, rows_before[lo + 1] - p.p0));
        return p;
    };
    const int row_bytes = m.K / 32 * 18;
    Cursor cur = first_item(plan);
    Item item;

    if (warp < kDecodeWarps) {
        // ---- unpacking, then the outputs
        if constexpr (C::kMoveRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kDecodeRegs));
        const int group = warp >> 2, half = group & 1, ph = group >> 1;
        const int r = 32 * (warp & 3) + lane;  // this thread's weight row of the half, and its TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const int together = WIDE ? 16 / (row_bytes & -row_bytes) : 1;
        const int shift = WIDE ? (r % together) * row_bytes & 15 : 0;
        const int slot = half * kHalf + (WIDE ? (r % together) * (kHalf / together) + r / together : r);
        const uint32_t a_cols = tmem + lanes + C::kTmemA + half * 64;
        bool ok = true;
        uint32_t it = 0, sums = 0;  // units, sets of sums
        // This phase's next stage of unpacked weights, and how often it has been filled (a unit has two stages,
        // f32 rows' four; phase p fills every second one).
        uint32_t a_stage = ph, a_round = 0;
        constexpr int kChunk = C::kChunk;
        float v0[kChunk], v1[kChunk];  // sums of a chunk of columns of both halves (F32: number `group`, kept from unit to unit)
        // Waits for the set of sums number `sums`.
        auto wait_sums = [&] {
            ok = ok && warp_wait(&bar.acc_full[sums % C::kSums], (sums / C::kSums) & 1, err);
            tc_fence_after();
        };
        auto free_sums = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.acc_empty[sums % C::kSums]);
            ++sums;
        };
        // F32: adds the sums of a unit (of `n` rows) to those of the units before it.
        auto collect = [&](int n) {
            wait_sums();
            if constexpr (F32) {
                if (kChunk * group < n) {
                    const uint32_t d = tmem + lanes + kChunk * group;
                    const int second = (n + 15) & ~15;  // where the products with the second pieces are
                    auto add = [&](float(&v)[kChunk], uint32_t from) {
#pragma unroll
                        for (int e0 = 0; e0 < kChunk; e0 += 8) {
                            float a[8], b[8];
                            tmem_ldn(from + e0, a);
                            tmem_ldn(from + second + e0, b);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e0 + e] += a[e] + b[e];
                        }
                    };
                    add(v0, d);
                    add(v1, d + C::kColumns);
                }
            }
            free_sums();
        };
        auto unpack_unit = [&](int u, int n_before) {
            const int stage = it % C::kRawStages;
            ok = ok && warp_wait(&bar.raw_full[stage], (it / C::kRawStages) & 1, err);
            ++it;
            const uint8_t* row = raw + stage * C::kRawBytes + slot * C::kPitch;
            [[maybe_unused]] const int left = m.K - 256 * u;
            auto begin_stage = [&] {
                ok = ok && (a_round == 0 || warp_wait(&bar.empty[a_stage], (a_round - 1) & 1, err));
                tc_fence_after();
            };
            auto end_stage = [&] {
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.full[a_stage]);
                a_stage += 2;
                if (a_stage >= C::kStages) a_stage -= C::kStages, ++a_round;
            };
            auto load = [&](auto first, auto second, uint32_t(&w)[9]) {
                if (ph) load_words<decltype(second)::value, WIDE>(row, shift, w);
                else load_words<decltype(first)::value, WIDE>(row, shift, w);
            };
            auto done_with_row = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.raw_empty[stage]);
            };
            using I = std::integral_constant<int, 0>;
            // (As much as there are registers for is unpacked before the wait for room.  Stages past a
            // row's end are handed over empty.)
            uint32_t w[9];
            if constexpr (F32) {  // the unit's 64 elements number ph, then ph + 2
                auto unpack_64 = [&](bool there) {
                    uint32_t h[8], l[8];
                    unpack_block<true, 0, 2>(w, 0, m.k1024, h, l);
                    begin_stage();
                    const uint32_t at = a_cols + a_stage * 128;
                    if (there) {
                        tmem_st8(at, h);
                        tmem_st8(at + 32, l);
                        unpack_block<true, 2, 2>(w, 0, m.k1024, h, l);
                        tmem_st8(at + 8, h);
                        tmem_st8(at + 40, l);
                        unpack_block<true, 0, 2>(w, 1, m.k1024, h, l);
                        tmem_st8(at + 16, h);
                        tmem_st8(at + 48, l);
                        unpack_block<true, 2, 2>(w, 1, m.k1024, h, l);
                        tmem_st8(at + 24, h);
                        tmem_st8(at + 56, l);
                    }
                    end_stage();
                };
                load(I{}, std::integral_constant<int, 1>{}, w);
                unpack_64(64 * ph < left);
                if (n_before) collect(n_before);  // (of the unit before: there is one set of sums)
                load(std::integral_constant<int, 2>{}, std::integral_constant<int, 3>{}, w);
                done_with_row();
                unpack_64(64 * (ph + 2) < left);
            } else {  // its elements 128 ph .. + 127
                uint32_t h[32];
                load(I{}, std::integral_constant<int, 2>{}, w);
                unpack_block<false>(w, 0, m.k1024, h, nullptr);
                unpack_block<false>(w, 1, m.k1024, h + 16, nullptr);
                load(std::integral_constant<int, 1>{}, std::integral_constant<int, 3>{}, w);
                done_with_row();
                begin_stage();
                const uint32_t at = a_cols + a_stage * 128;
                tmem_st32(at, reinterpret_cast<const float*>(h));
                unpack_block<false>(w, 0, m.k1024, h, nullptr);
                unpack_block<false>(w, 1, m.k1024, h + 16, nullptr);
                tmem_st32(at + 32, reinterpret_cast<const float*>(h));
                end_stage();
            }
        };
        // A tile's outputs, once all of its products are done.
        auto outputs = [&](int tile, int n_units, uint32_t mine_buf) {
            const Place pl = place(tile);
            if constexpr (!F32) wait_sums();
            named_barrier_sync(2, kDecodeWarps * 32);  // the factors and pairs are there
            const bool whole = n_units == plan.ku;
            const int f0 = pl.block * block_rows + r, f1 = two ? f0 : f0 + kHalf;
            const bool in0 = f0 < m.rows, in1 = f1 < m.rows;
            // Chunk ch of the columns of both halves, as sums of whole rows.
            auto finish = [&](int ch) {
#pragma unroll
                for (int i = 0; i < kChunk; i += 4) {
                    const float4 s = *reinterpret_cast<const float4*>(&units[mine_buf][kChunk * ch + i]);
                    v0[i] *= s.x, v0[i + 1] *= s.y, v0[i + 2] *= s.z, v0[i + 3] *= s.w;
                    v1[i] *= s.x, v1[i + 1] *= s.y, v1[i + 2] *= s.z, v1[i + 3] *= s.w;
                }
                if (!DOWN) {
                    const int kind = m.activation;
                    if (kind == QM_ACT_SILU) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            v0[i] = activate<F32>(v0[i], QM_ACT_SILU);
                            if (!two) v1[i] = activate<F32>(v1[i], QM_ACT_SILU);
                        }
                    } else if (kind == QM_ACT_GELU) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            v0[i] = activate<F32>(v0[i], QM_ACT_GELU);
                            if (!two) v1[i] = activate<F32>(v1[i], QM_ACT_GELU);
                        }
                    }
                    if (two) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) v0[i] *= v1[i];
                    }
                }
                float* out = m.out + static_cast<int64_t>(pl.p0 + kChunk * ch) * m.rows + f0;
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    if (kChunk * ch + i >= pl.n) break;
                    if (in0) out[0] = v0[i];
                    if (in1 && !two) out[kHalf] = v1[i];
                    asm volatile("" ::: "memory");
                    out += m.rows;
                }
            };
            auto load_sums = [&](int ch) {
                if constexpr (!F32) {
                    const uint32_t d = tmem + lanes + (sums % C::kSums) * 2 * C::kColumns + kChunk * ch;
                    tmem_ldn(d, v0);
                    tmem_ldn(d + C::kColumns, v1);
                    tc_wait_ld();
                }
            };
            if (whole) {
                for (int ch = group; kChunk * ch < pl.n; ch += 4) {
                    load_sums(ch);
                    finish(ch);
                }
                if constexpr (!F32) free_sums();
                return;
            }
            // A part of the tile: kept in this CTA's place, [half][column][row].
            const int64_t place_floats = static_cast<int64_t>(2 * kHalf) * m.split_cols;
            const int shared_tile = tile - plan.full;
            auto part_of = [&](int c) {  // CTA c's part of this tile
                return m.split + (2 * c + (plan.unit_of(c) < shared_tile * plan.ku)) * place_floats;
            };
            float* mine = part_of(plan.cta);
            for (int ch = group; kChunk * ch < pl.n; ch += 4) {
                load_sums(ch);
                float* at = mine + kChunk * ch * kHalf + r;
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    at[i * kHalf] = v0[i];
                    at[(m.split_cols + i) * kHalf] = v1[i];
                }
            }
            if constexpr (!F32) free_sums();
            named_barrier_sync(1, kDecodeWarps * 32);
            if (threadIdx.x == 0) {
                const unsigned n = static_cast<unsigned>(n_units);
                last_of_tile = atom_add_acq_rel(&m.counters[shared_tile], n) + n == static_cast<unsigned>(plan.ku);
            }
            named_barrier_sync(1, kDecodeWarps * 32);
            if (!last_of_tile) return;
            // The CTAs that have units of it, in order.
            const int begin = shared_tile * plan.ku;
            int c_lo = plan.cta;
            while (plan.unit_of(c_lo) > begin) --c_lo;
            for (int ch = group; kChunk * ch < pl.n; ch += 4) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float(&v)[kChunk] = half ? v1 : v0;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v[i] = 0.f;
#pragma unroll 1
                    for (int c = c_lo; plan.unit_of(c) < begin + plan.ku; ++c) {
                        const float* part = part_of(c) + (half * m.split_cols + kChunk * ch) * kHalf + r;
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) {
                            if (i % 8 == 0) asm volatile("" ::: "memory");  // (8 loads on their way: more would cost registers)
                            v[i] += __ldcg(part + i * kHalf);
                        }
                    }
                }
                finish(ch);
            }
        };

        // Unit by unit.  A tile's outputs wait until the next tile's first unit is unpacked, so that the
        // products of that one can begin as soon as there is room for its sums.
        int n_now = 0;
        Seldom in_registers;
        Seldom& seldom = C::kMoveRegs ? seldom_of[warp] : in_registers;
        uint32_t buf = 0;  // of 3 sets of factors: a warp may be two tiles ahead of another's outputs
        auto next = [&](Cursor c) {
            const bool got = next_item(plan, c, &item);
            __syncwarp();
            seldom.cur = c;
            __syncwarp();
            return got;
        };
        bool more = next(cur), due = false;
        int u = 0;
        auto begin = [&] {
            const Place pl = place(item.tile);
            n_now = pl.n;
            u = item.u0;
            buf = buf == 2 ? 0 : buf + 1;
            if (static_cast<int>(threadIdx.x) < C::kTokens) {
                const int p = pl.p0 + min(static_cast<int>(threadIdx.x), pl.n - 1);
                units[buf][threadIdx.x] = m.unit[p] * kWeightUnit;
            }
        };
        if (more) begin();
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v0[i] = v1[i] = 0.f;
        }
#pragma unroll 1
        while (more || due) {
            if (more) {
                unpack_unit(u, u > item.u0 ? n_now : due ? seldom.n : 0);
            }
            if (due) {
                if (F32 && !more) collect(seldom.n);
                outputs(seldom.tile, seldom.units, seldom.buf);
                due = false;
                if constexpr (F32) {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) v0[i] = v1[i] = 0.f;
                }
            }
            if (more && ++u == item.u1) {
                __syncwarp();
                seldom.n = n_now;
                seldom.tile = item.tile, seldom.units = item.u1 - item.u0, seldom.buf = buf;
                due = true;
                more = next(seldom.cur);
                if (more) begin();
            }
        }
    } else {
    if constexpr (C::kMoveRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == kRawWarp) {
        // ---- raw weights
        bool ok = true;
        uint32_t it = 0;
        const int together = WIDE ? 16 / (row_bytes & -row_bytes) : 1;
        while (ok && next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            for (int u = item.u0; u < item.u1 && ok; ++u, ++it) {
                const int stage = it % C::kRawStages;
                if (it >= C::kRawStages) ok = warp_wait(&bar.raw_empty[stage], (it / C::kRawStages - 1) & 1, err);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&bar.raw_full[stage], C::kRawBytes);
                __syncwarp();
                // Lanes i and 16 + i: the rows i of each group of the two halves.
                const int i = lane & 15, half = lane >> 4;
                if (i < together) {
                    const int row0 = pl.block * block_rows + (two ? 0 : half * kHalf);
                    uint8_t* dst = raw + stage * C::kRawBytes + (half * kHalf + i * (kHalf / together)) * C::kPitch;
                    tma_load_3d(dst, half ? &map_w1 : &map_w0, (i * row_bytes & ~15) + 144 * u, row0 / together, pl.expert,
                                &bar.raw_full[stage]);
                }
                __syncwarp();
            }
        }
        for (uint32_t i = it > C::kRawStages ? it - C::kRawStages : 0; !ok && i < it; ++i)  // what is still on its way
            mbar_wait_bounded(&bar.raw_full[i % C::kRawStages], (i / C::kRawStages) & 1, err);
    } else if (warp == kTokenWarp) {
        // ---- token rows
        bool ok = true;
        uint32_t kt = 0;
        while (ok && next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            const int n16 = (pl.n + 15) & ~15;
            for (int k = 256 * item.u0; k < 256 * item.u1; k += C::kStageK) {
                if (!C::kJoint && k >= m.K) break;
                const int stage = kt % C::kTokenStages;
                uint64_t* const full = C::kJoint ? &bar.full[stage] : &bar.tok_full[stage];
                uint64_t* const empty = C::kJoint ? &bar.empty[stage] : &bar.tok_empty[stage];
                if (kt >= C::kTokenStages) ok = warp_wait(empty, (kt / C::kTokenStages - 1) & 1, err);
                if (!ok) break;
                const int parts = k >= m.K ? 0 : F32 || k + 64 < m.K ? 2 : 1;  // (a row's last stage may be half one, or none)
                if (lane == 0) mbar_arrive_expect_tx(full, parts * n16 * 128);
                __syncwarp();
                // Lane i: 16 rows.
                uint8_t* dst = tok + stage * C::kTokenBytes + lane * 2048;
                if (16 * lane < n16 && parts > 0) {
                    const int p = pl.p0 + 16 * lane;
                    const CUtensorMap* second = F32 ? &map_lo : &map_hi;
                    const int k2 = F32 ? k : k + 64;
                    tma_load_2d(dst, &map_hi, k, p, full);
                    if (parts > 1) tma_load_2d(dst + (F32 ? n16 : C::kTokens) * 128, second, k2, p, full);
                }
                __syncwarp();
                ++kt;
            }
        }
        for (uint32_t i = kt > C::kTokenStages ? kt - C::kTokenStages : 0; !ok && i < kt; ++i)
            mbar_wait_bounded(C::kJoint ? &bar.full[i % C::kStages] : &bar.tok_full[i % C::kTokenStages], (i / C::kTokenStages) & 1, err);
    } else {
        // ---- products of a half of the weight rows
        const uint32_t lead = elect_one();
        const int half = warp - kMmaWarp;
        bool ok = true;
        uint32_t sums = 0, stage = 0, round = 0;  // sets of sums, stages of weights
        [[maybe_unused]] uint32_t t_stage = 0, t_round = 0;  // stages of tokens
        const uint64_t b_first = desc_base(smem_addr(tok), 16);
        const uint32_t d_half = tmem + half * C::kColumns, w_half = tmem + C::kTmemA + half * 64;
        while (ok && next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            const int n16 = (pl.n + 15) & ~15;
            const uint32_t id = idesc_f16(n16, false), id_both = idesc_f16(F32 ? 2 * n16 : n16, false);
            const int k_begin = 256 * item.u0, k_end = 256 * item.u1;
            uint32_t acc = 0, d = d_half;
            for (int k = k_begin; k < k_end && ok; k += C::kStageK) {
                if (k == k_begin || (F32 && k % 256 == 0)) {  // a set of sums: F32 a unit's, else the item's
                    if (sums >= C::kSums)
                        ok = warp_wait(&bar.acc_empty[sums % C::kSums], (sums / C::kSums - 1) & 1, err);
                    d = d_half + (sums % C::kSums) * 2 * C::kColumns;
                    acc = 0;
                }
                if (!C::kJoint && k < m.K) ok = ok && warp_wait(&bar.tok_full[t_stage], t_round & 1, &bar.full[stage], round & 1, err);
                else ok = ok && warp_wait(&bar.full[stage], round & 1, err);
                if (!ok) break;
                tc_fence_after();
                const uint64_t b = b_first + (C::kJoint ? stage : t_stage) * (C::kTokenBytes >> 4);
                const uint32_t w = w_half + stage * 128;
                auto step = [&](int s, uint32_t add) {
                    if constexpr (F32) {
                        mma_ts(d, w + 8 * s, b + 2 * s, id_both, add, lead);
                        mma_ts(d + n16, w + 32 + 8 * s, b + 2 * s, id, 1, lead);
                    } else {
                        mma_ts(d, w + 8 * s, b + (s >> 2) * (C::kTokens * 128 >> 4) + 2 * (s & 3), id, add, lead);
                    }
                };
                if (k + C::kStageK <= m.K) {
                    step(0, acc);
#pragma unroll
                    for (int s = 1; s < C::kStageK / 16; ++s) step(s, 1);
                } else if (k < m.K) {
                    const int steps = (m.K - k) >> 4;
                    step(0, acc);
#pragma unroll 1
                    for (int s = 1; s < steps; ++s) step(s, 1);
                }
                acc = 1;
                mma_commit(&bar.empty[stage], lead);
                if (++stage == C::kStages) stage = 0, ++round;
                if constexpr (!C::kJoint) {
                    if (k < m.K) {
                        mma_commit(&bar.tok_empty[t_stage], lead);
                        if (++t_stage == C::kTokenStages) t_stage = 0, ++t_round;
                    }
                }
                if (k + C::kStageK == k_end || (F32 && k % 256 == 192)) {
                    mma_commit(&bar.acc_full[sums % C::kSums], lead);
                    ++sums;
                }
            }
        }
        // Products still under way (after a wait that gave up) end before the TMEM is given back.
        if (!ok) {
            mma_commit(&bar.acc_full[sums % C::kSums], lead);
            warp_wait(&bar.acc_full[sums % C::kSums], (sums / C::kSums) & 1, err);
        }
    }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <bool F32, int TOKENS, bool DOWN, bool WIDE>
cudaError_t launch_kernel(const ExpertsMm& m, const ExpertsView& e, const void* hi, const void* lo,
                          int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream) {
    using C = Cfg<F32, TOKENS, WIDE>;
    static SmemOnce once;
    cudaError_t err = once.set(experts_mm_kernel<F32, TOKENS, DOWN, WIDE>, C::kSmem, C::kMoveRegs ? C::kLaunchRegs : 0);
    if (err != cudaSuccess) return err;
    const int64_t row_bytes = m.K / 32 * 18;
    const int together = WIDE ? 16 / static_cast<int>(row_bytes & -row_bytes) : 1;
    CUtensorMap w0, w1, t_hi, t_lo;
    if ((err = weight_map(&w0, m.w[0], m.w_stride[0], row_bytes, m.rows, e.n, together, C::kPitch)) != cudaSuccess) return err;
    if ((err = weight_map(&w1, m.w[1], m.w_stride[1], row_bytes, m.rows, e.n, together, C::kPitch)) != cudaSuccess) return err;
    const int64_t dims[2] = {piece_pitch(m.K), n_pieces}, strides[1] = {piece_pitch(m.K) * 2};
    const int box[2] = {64, 16};
    for (int i = 0; i < 2; ++i) {
        err = encode_tiled(i ? &t_lo : &t_hi, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, i ? lo : hi, 2, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
        if (err != cudaSuccess) return err;
    }
    const int ctas = dev.sm_count < kExpertCtas ? dev.sm_count : kExpertCtas;
    err = launch_pdl(experts_mm_kernel<F32, TOKENS, DOWN, WIDE>, dim3(ctas), dim3(kThreads), C::kSmem, stream, w0, w1, t_hi, t_lo, m);
    if (err == cudaSuccess) note_launch();
    return err;
}

}  // namespace

cudaError_t launch_experts_mm(const ExpertsMm& m, const ExpertsView& e, bool down, KvType type, const void* hi,
                              const void* lo, int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream) {
    const bool wide = m.K % 256 != 0;
    auto go = [&](auto f32, auto tokens) {
        constexpr bool kF32 = decltype(f32)::value;
        constexpr int kTokens = decltype(tokens)::value;
        auto run = [&](auto kernel) { return kernel(m, e, hi, kF32 ? lo : hi, n_pieces, dev, stream); };
        if (down) return wide ? run(launch_kernel<kF32, kTokens, true, true>) : run(launch_kernel<kF32, kTokens, true, false>);
        return wide ? run(launch_kernel<kF32, kTokens, false, true>) : run(launch_kernel<kF32, kTokens, false, false>);
    };
    // Narrow tiles where experts have few rows: three stages of weights, bf16 rows two sets of sums (16 experts of
    // 4096 x 4096 with 24 rows each: bf16 146 us against 157, f32 249 against 292; with more, some experts' rows
    // take two tiles: 48 bf16 rows each 247 against 168, uneven f32 rows, 32 on average, 331 against 310).
    const bool narrow = n_pieces <= 24 * static_cast<int64_t>(e.n);
    if (type == KvType::kF32)
        return narrow ? go(std::true_type{}, std::integral_constant<int, 32>{}) : go(std::true_type{}, std::integral_constant<int, 64>{});
    if (narrow) return go(std::false_type{}, std::integral_constant<int, 32>{});
    return go(std::false_type{}, std::integral_constant<int, kExpertTokens>{});
}

}  // namespace qm
