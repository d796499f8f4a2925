// The experts' products (qm_experts_q4_0) on tcgen05 tensor cores.
//
// The weights are the 128-row operand and the token rows the columns, so a tile is
// 256 weight rows (128 of gate and 128 of up, or 256 of one matrix) by 1 to 128 rows of
// one expert, rounded up to 16: the same kernel serves one token and thousands.
//
//   D[w][t] = sum_k (q_wk - 8) d_wb  x_tk
//
// Operands are f16.  A weight is (q - 8) d 2^8, at most 15 significant bits: its f16
// rounding, and for f32 rows the exact rest as a second piece.  The 2^8 keeps the rest of
// scales from 2^-10 up out of f16's subnormal numbers.  Token rows come as f16 pieces of
// x times a power of two that takes the row's largest value to 2^13 .. 2^14 (one piece
// holds a bf16 row's 8 bits, two an f32 row's 22).  f32 rows take three products, the
// fourth being 2^-22 of the first.  Tensor cores cut sums off instead of rounding them: 48
// additions (a unit of three products) cost 8e-7 of a sum of mixed signs, so f32 rows' sums
// go to registers after every unit and are added there; bf16 rows' stay in TMEM.  The element order inside a block of 32 is that in
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
// K) of those left over are dealt out evenly, and the CTA that comes last to a shared tile
// adds its parts in the CTAs' order.
//
// Every wait is bounded; a wait that gives up sets the device error word.
#include "experts.cuh"
#include "tcgen05.cuh"

namespace qm {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kHalf = 128;  // weight rows of a half tile
constexpr int kDecodeWarps = 16;
constexpr int kRawWarp = 16, kTokenWarp = 17, kMmaWarp = 18;
constexpr int kThreads = 19 * 32;
constexpr int kTmemA = 256;  // columns 0 .. 255: sums, [set][half][token row]
constexpr float kWeightUnit = 0x1p-8f;

template <bool F32, bool WIDE>
struct Cfg {
    static constexpr int kTokens = F32 ? kExpertTokens / 2 : kExpertTokens;
    static constexpr int kPanel = kTokens * 128;  // bytes of a piece's 64 elements of all token rows
    static constexpr int kSums = F32 ? 2 : 1;     // sets of sums in TMEM
    // A stage of unpacked weights (there are two, each filled by the warps of one phase) and of
    // token rows: 128 columns of TMEM, two panels.
    static constexpr int kStageK = F32 ? 64 : 128;
    static constexpr int kPitch = WIDE ? 176 : 144;  // bytes of a raw row in shared memory, an odd number of 16s
    static constexpr int kRawBytes = 2 * kHalf * kPitch;
    static constexpr int kRawStages = F32 && !WIDE ? 4 : 3;
    static constexpr int kTokenBytes = 2 * kPanel;
    static constexpr int kTokenStages = F32 ? 4 : WIDE ? 2 : 3;
    static constexpr int kSmem = kRawStages * kRawBytes + kTokenStages * kTokenBytes + 1024;
};

struct Barriers {
    uint64_t raw_full[4], raw_empty[4];
    uint64_t tok_full[4], tok_empty[4];
    uint64_t a_full[2], a_empty[2];
    uint64_t acc_full[2], acc_empty[2];
};

// EXACT: to a few units of f32 (f32 rows); otherwise to about 2^-20.
template <bool EXACT>
__device__ __forceinline__ float activate(float a, int kind) {
    if (kind == 0) return a;
    const float z = kind == 1 ? a : 1.5957691216057308f * (a + 0.044715f * a * a * a);  // tanh(y) = 2 sigmoid(2 y) - 1
    return EXACT ? a / (1.f + expf(-z)) : __fdividef(a, 1.f + __expf(-z));
}

// A whole warp's bounded waits; the answer is the same for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* a, uint32_t pa, unsigned int* err) {
    for (uint32_t i = 0; i < kMaxWaitPolls; ++i)
        if (__all_sync(kAll, mbar_try_wait(a, pa))) return true;
    atomicOr(err, kErrWaitTimeout);
    return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, unsigned int* err) {
    for (uint32_t i = 0; i < kMaxWaitPolls; ++i) {
        const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
        if (__all_sync(kAll, x && y)) return true;
    }
    atomicOr(err, kErrWaitTimeout);
    return false;
}
// A value that all lanes have, in a uniform register.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kAll, v, 0); }

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

// What a CTA does, one piece after the other: tiles, each with a range of units.
struct Plan {
    int tiles, full, rest, ku, ctas, cta;
    bool share;  // the tiles left over are shared by all CTAs
    __device__ __forceinline__ int64_t unit_of(int c) const { return static_cast<int64_t>(rest) * ku * c / ctas; }
};
struct Item {
    int tile, u0, u1;
};
struct Cursor {
    int next;     // of the whole tiles
    int64_t at, end;  // units of shared tiles
};
__device__ __forceinline__ Cursor first_item(const Plan& p) {
    Cursor c{p.cta, 0, 0};
    if (p.share) c.at = p.unit_of(p.cta), c.end = p.unit_of(p.cta + 1);
    return c;
}
// Shared tiles first: the CTA that comes last to one has others to go on with.
__device__ __forceinline__ bool next_item(const Plan& p, Cursor& c, Item* item) {
    if (c.at < c.end) {
        const int t = static_cast<int>(c.at / p.ku);
        item->tile = p.full + t;
        item->u0 = static_cast<int>(c.at - static_cast<int64_t>(t) * p.ku);
        item->u1 = static_cast<int>(min(static_cast<int64_t>(p.ku), item->u0 + (c.end - c.at)));
        c.at += item->u1 - item->u0;
        return true;
    }
    if (c.next >= (p.share ? p.full : p.tiles)) return false;
    *item = {c.next, 0, p.ku};
    c.next += p.ctas;
    return true;
}

// Where a tile lies: its expert, its block of weight rows, its token rows.
struct Place {
    int expert, block, p0, n;
};

// 64 elements of a weight row: words 0 .. 8 are bytes 0 .. 35 of its two blocks.  Stored to
// columns `addr` .. + 31 (F32: the second pieces to the 32 after).
template <bool F32>
__device__ __forceinline__ void unpack_store(const uint32_t (&w)[9], uint32_t addr, uint32_t k1024) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t d_bits = __byte_perm(b ? w[4] : w[0], 0, b ? 0x3232 : 0x1010);
        const __half2 d = __hmul2(half2_of(d_bits), half2_of(0x5C005C00u));  // times 2^8
        const __half2 m1032 = half2_of(0xE408E408u), sixteenth = half2_of(0x2C002C00u), m72 = half2_of(0xD480D480u);
        uint32_t h[16], l[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t q = b ? w[5 + k] : __byte_perm(w[k], w[k + 1], 0x5432);
            const uint32_t y = q >> 8;
            const __half2 n[4] = {__hadd2(half2_of((q & 0x000F000Fu) | k1024), m1032),
                                  __hadd2(half2_of((y & 0x000F000Fu) | k1024), m1032),
                                  __hfma2(half2_of((q & 0x00F000F0u) | k1024), sixteenth, m72),
                                  __hfma2(half2_of((y & 0x00F000F0u) | k1024), sixteenth, m72)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 x = __hmul2(n[e], d);
                h[4 * k + e] = word(x);
                if (F32) l[4 * k + e] = word(__hfma2(n[e], d, __hneg2(x)));
            }
        }
        tmem_st16(addr + 16 * b, h);
        if (F32) tmem_st16(addr + 32 + 16 * b, l);
    }
}

// Words of the 64-element pieces KS0 and KS0 + STEP of a unit's row.
template <int KS0, int STEP, bool WIDE>
__device__ __forceinline__ void load_words(const uint8_t* row, int shift, uint32_t (&w)[2][9]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        constexpr int kStep = 36;
        const int ks = KS0 + STEP * j;
        if constexpr (!WIDE) {
            // Bytes 36 ks .. + 35 lie ks words into the 48 bytes from the 16-byte boundary below.
            uint32_t v[12];
            const int from = kStep * ks & ~15;
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(row + from);
            *reinterpret_cast<uint4*>(v + 4) = *reinterpret_cast<const uint4*>(row + from + 16);
            *reinterpret_cast<uint4*>(v + 8) = *reinterpret_cast<const uint4*>(row + from + 32);
#pragma unroll
            for (int i = 0; i < 9; ++i) w[j][i] = v[i + ks];
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(row + kStep * ks + (shift & ~3));
            const uint32_t sel = shift & 2 ? 0x5432 : 0x3210;
            uint32_t v = p[0];
#pragma unroll
            for (int i = 0; i < 9; ++i) {
                const uint32_t next = p[i + 1];
                w[j][i] = __byte_perm(v, next, sel);
                v = next;
            }
        }
    }
}

template <bool F32, bool DOWN, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    experts_mm_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                      const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
                      const ExpertsMm m) {
    using C = Cfg<F32, WIDE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* tok = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint8_t* raw = tok + C::kTokenStages * C::kTokenBytes;
    __shared__ Barriers bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int tiles_before[1024 + 1];  // token tiles of all lower experts
    __shared__ int rows_before[1024 + 1];   // their sorted rows
    __shared__ float units[2][C::kTokens];  // of the columns of this tile and the one before
    __shared__ int pairs[2][C::kTokens];
    __shared__ int last_of_tile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned int* const err = m.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], kDecodeWarps);
            mbar_init(&bar.tok_full[i], 1);
            mbar_init(&bar.tok_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.a_full[i], 8);
            mbar_init(&bar.a_empty[i], 1);
            mbar_init(&bar.acc_full[i], 1);
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

    const bool two = m.w[0] != m.w[1];  // gate and up
    const int block_rows = two ? kHalf : 2 * kHalf;
    const int blocks = (m.rows + block_rows - 1) / block_rows;
    Plan plan;
    plan.tiles = tiles_before[m.n] * blocks;
    plan.ctas = gridDim.x;
    plan.cta = blockIdx.x;
    plan.ku = (m.K + 255) / 256;
    plan.full = plan.tiles / plan.ctas * plan.ctas;
    plan.rest = plan.tiles - plan.full;
    plan.share = plan.rest > 0 && plan.rest * 8 <= plan.ctas * 7 && plan.ku > 1;
    auto place = [&](int tile) {
        const int tt = tile / blocks;
        int lo = 0, hi = m.n;  // the first expert with tiles_before[e + 1] > tt
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tiles_before[mid + 1] <= tt) lo = mid + 1;
            else hi = mid;
        }
        Place p;
        p.expert = lo;
        p.block = tile - tt * blocks;
        p.p0 = rows_before[lo] + (tt - tiles_before[lo]) * C::kTokens;
        p.n = min(C::kTokens, rows_before[lo + 1] - p.p0);
        return p;
    };
    const int row_bytes = m.K / 32 * 18;
    Cursor cur = first_item(plan);
    Item item;

    if (warp < kDecodeWarps) {
        // ---- unpacking, then the outputs
        const int group = warp >> 2, half = group & 1, ph = group >> 1;
        const int r = 32 * (warp & 3) + lane;  // this thread's weight row of the half, and its TMEM lane
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const int together = WIDE ? 16 / (row_bytes & -row_bytes) : 1;
        const int shift = WIDE ? (r % together) * row_bytes & 15 : 0;
        const int slot = half * kHalf + (WIDE ? (r % together) * (kHalf / together) + r / together : r);
        const uint32_t a_cols = tmem + lanes + kTmemA + ph * 128 + half * 64;
        bool ok = true;
        uint32_t it = 0, sums = 0, n_items = 0;  // units, sets of sums
        uint32_t uses = 0;                       // of this phase's stage
        float v0[16], v1[16];  // F32: this thread's sums, columns 16 group .. + 15 of both halves
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
        // F32: adds the sums of a unit to those of the units before it.
        auto collect = [&](int n) {
            wait_sums();
            if (16 * group < n) {
                const uint32_t d = tmem + lanes + (sums % C::kSums) * 2 * C::kTokens + 16 * group;
                float a[16];
                tmem_ld16(d, a);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] += a[i];
                tmem_ld16(d + C::kTokens, a);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v1[i] += a[i];
            }
            free_sums();
        };
        while (next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            const int buf = n_items++ & 1;
            if (static_cast<int>(threadIdx.x) < C::kTokens) {
                const int p = pl.p0 + min(static_cast<int>(threadIdx.x), pl.n - 1);
                units[buf][threadIdx.x] = m.unit[p] * kWeightUnit;
                if (DOWN) pairs[buf][threadIdx.x] = m.order[p];
            }
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = v1[i] = 0.f;
            }
            for (int u = item.u0; u < item.u1; ++u, ++it) {
                const int stage = it % C::kRawStages;
                ok = ok && warp_wait(&bar.raw_full[stage], (it / C::kRawStages) & 1, err);
                const uint8_t* row = raw + stage * C::kRawBytes + slot * C::kPitch;
                uint32_t w[2][9];
                const int left = m.K - 256 * u;
                if (F32 && ph) load_words<1, 2, WIDE>(row, shift, w);
                else if (F32) load_words<0, 2, WIDE>(row, shift, w);
                else if (ph) load_words<2, 1, WIDE>(row, shift, w);
                else load_words<0, 1, WIDE>(row, shift, w);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.raw_empty[stage]);
                // bf16 rows: 128 elements, a stage; f32 rows: 64 elements twice.
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int ks = F32 ? ph + 2 * j : 2 * ph + j;
                    if (F32 ? 64 * ks >= left : 128 * ph >= left) break;
                    if (F32 || j == 0) {
                        ok = ok && (uses == 0 || warp_wait(&bar.a_empty[ph], (uses - 1) & 1, err));
                        ++uses;
                        tc_fence_after();
                    }
                    unpack_store<F32>(w[j], a_cols + (F32 ? 0 : 32 * j), m.k1024);
                    if (F32 || j == 1) {
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.a_full[ph]);
                    }
                }
                if (F32 && u > item.u0) collect(pl.n);  // of the unit before
            }
            if constexpr (F32) collect(pl.n);
            else wait_sums();
            named_barrier_sync(2, kDecodeWarps * 32);  // the units and pairs are there
            const bool whole = item.u1 - item.u0 == plan.ku;
            const int f0 = pl.block * block_rows + r, f1 = two ? f0 : f0 + kHalf;
            // Columns 16 ch .. 16 ch + 15 of both halves, as sums of whole rows.
            auto finish = [&](int ch) {
                auto again = [&](int which, int f, int c) {
                    const uint8_t* w = m.w[which] + pl.expert * m.w_stride[which] + static_cast<int64_t>(f) * row_bytes;
                    if (DOWN) return exact_dot(w, m.K, static_cast<const float*>(m.x) + (pl.p0 + c) * m.x_stride);
                    const int64_t at = (m.order[pl.p0 + c] / m.top_k) * m.x_stride;
                    if (!F32) return exact_dot(w, m.K, static_cast<const __nv_bfloat16*>(m.x) + at);
                    return exact_dot(w, m.K, static_cast<const float*>(m.x) + at);
                };
                float* out = m.out + static_cast<int64_t>(pl.p0 + 16 * ch) * m.rows + f0;
                const int f_step = f1 - f0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int c = 16 * ch + i;
                    if (c >= pl.n) break;
                    const float s = units[buf][c];
                    float a = v0[i] * s, b = v1[i] * s;
                    if (!(fabsf(a) + fabsf(b) < INFINITY)) {
                        if (f0 < m.rows && !isfinite(a)) a = again(0, f0, c);
                        if (f1 < m.rows && !isfinite(b)) b = again(1, f1, c);
                    }
                    if (DOWN) {
                        out = m.out + static_cast<int64_t>(pairs[buf][c]) * m.rows + f0;
                        if (f0 < m.rows) out[0] = a;
                        if (f1 < m.rows) out[kHalf] = b;
                    } else if (two) {
                        if (f0 < m.rows) out[0] = activate<F32>(a, m.activation) * b;
                    } else {
                        if (f0 < m.rows) out[0] = activate<F32>(a, m.activation);
                        if (f1 < m.rows) out[f_step] = activate<F32>(b, m.activation);
                    }
                    if (!DOWN) out += m.rows;
                }
            };
            auto load_sums = [&](int ch) {
                if constexpr (!F32) {
                    tmem_ld16(tmem + lanes + 16 * ch, v0);
                    tmem_ld16(tmem + lanes + C::kTokens + 16 * ch, v1);
                    tc_wait_ld();
                }
            };
            if (whole) {
                for (int ch = group; 16 * ch < pl.n; ch += 4) {
                    load_sums(ch);
                    finish(ch);
                }
                if constexpr (!F32) free_sums();
                continue;
            }
            // A part of the tile: kept in this CTA's place, [half][column][row].
            const int64_t place_floats = static_cast<int64_t>(2 * kHalf) * m.split_cols;
            const int shared_tile = item.tile - plan.full;
            auto part_of = [&](int c) {  // CTA c's part of this tile
                const int first = static_cast<int>(plan.unit_of(c) / plan.ku);
                return m.split + (2 * c + (shared_tile - first)) * place_floats;
            };
            float* mine = part_of(plan.cta);
            for (int ch = group; 16 * ch < pl.n; ch += 4) {
                load_sums(ch);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    mine[(16 * ch + i) * kHalf + r] = v0[i];
                    mine[(m.split_cols + 16 * ch + i) * kHalf + r] = v1[i];
                }
            }
            if constexpr (!F32) free_sums();
            __threadfence();
            named_barrier_sync(1, kDecodeWarps * 32);
            if (threadIdx.x == 0) {
                const unsigned n = static_cast<unsigned>(item.u1 - item.u0);
                last_of_tile = atomicAdd(&m.counters[shared_tile], n) + n == static_cast<unsigned>(plan.ku);
                __threadfence();
            }
            named_barrier_sync(1, kDecodeWarps * 32);
            if (!last_of_tile) continue;
            // The CTAs that have units of it, in order.
            const int64_t total = static_cast<int64_t>(plan.rest) * plan.ku, u_lo = static_cast<int64_t>(shared_tile) * plan.ku;
            const int c_lo = static_cast<int>(((u_lo + 1) * plan.ctas - 1) / total);
            const int c_hi = static_cast<int>(((u_lo + plan.ku) * plan.ctas - 1) / total);
            for (int ch = group; 16 * ch < pl.n; ch += 4) {
#pragma unroll
                for (int i = 0; i < 16; ++i) v0[i] = v1[i] = 0.f;
                for (int c = c_lo; c <= c_hi; ++c) {
                    if (plan.unit_of(c) == plan.unit_of(c + 1)) continue;
                    const float* part = part_of(c);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v0[i] += __ldcg(part + (16 * ch + i) * kHalf + r);
                        v1[i] += __ldcg(part + (m.split_cols + 16 * ch + i) * kHalf + r);
                    }
                }
                finish(ch);
            }
        }
    } else if (warp == kRawWarp) {
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
        // ---- token pieces
        bool ok = true;
        uint32_t kt = 0;
        while (ok && next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            const int n16 = (pl.n + 15) & ~15;
            const int k_end = min(m.K, 256 * item.u1);
            for (int k = 256 * item.u0; k < k_end && ok; k += C::kStageK, ++kt) {
                const int stage = kt % C::kTokenStages;
                if (kt >= C::kTokenStages) ok = warp_wait(&bar.tok_empty[stage], (kt / C::kTokenStages - 1) & 1, err);
                if (!ok) break;
                const bool both = F32 || k + 64 < k_end;  // (the last 64 elements of a row may be a stage)
                if (lane == 0) mbar_arrive_expect_tx(&bar.tok_full[stage], (both ? 2 : 1) * n16 * 128);
                __syncwarp();
                uint8_t* dst = tok + stage * C::kTokenBytes;
                if (16 * lane < n16) {
                    tma_load_2d(dst + lane * 2048, &map_hi, k, pl.p0 + 16 * lane, &bar.tok_full[stage]);
                    if (F32) tma_load_2d(dst + C::kPanel + lane * 2048, &map_lo, k, pl.p0 + 16 * lane, &bar.tok_full[stage]);
                    else if (both) tma_load_2d(dst + C::kPanel + lane * 2048, &map_hi, k + 64, pl.p0 + 16 * lane, &bar.tok_full[stage]);
                }
                __syncwarp();
            }
        }
        for (uint32_t i = kt > C::kTokenStages ? kt - C::kTokenStages : 0; !ok && i < kt; ++i)
            mbar_wait_bounded(&bar.tok_full[i % C::kTokenStages], (i / C::kTokenStages) & 1, err);
    } else {
        // ---- products
        const uint32_t lead = elect_one();
        bool ok = true;
        uint32_t sums = 0, stage = 0, round = 0;
        uint32_t a_phase = 0;  // a bit per stage
        const uint64_t b_first = desc_base(smem_addr(tok), 16);
        while (ok && next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            const uint32_t id = idesc_f16(uniform(pl.n + 15) & ~15, false);
            const int k_begin = uniform(256 * item.u0), k_end = uniform(min(m.K, 256 * item.u1));
            uint32_t acc = 0, d_set = 0;
            for (int k = k_begin; k < k_end && ok; k += C::kStageK) {
                if (k == k_begin || (F32 && k % 256 == 0)) {  // a set of sums: F32 a unit's, else the item's
                    if (sums >= C::kSums)
                        ok = warp_wait(&bar.acc_empty[sums % C::kSums], (sums / C::kSums - 1) & 1, err);
                    if (!ok) break;
                    d_set = (sums % C::kSums) * 2 * C::kTokens;
                    acc = 0;
                }
                const int a = (k / C::kStageK) & 1;
                ok = warp_wait(&bar.tok_full[stage], round & 1, &bar.a_full[a], (a_phase >> a) & 1, err);
                if (!ok) break;
                a_phase ^= 1u << a;
                tc_fence_after();
                const uint64_t b = b_first + stage * (C::kTokenBytes >> 4);
                const uint32_t d = tmem + d_set, w = tmem + kTmemA + a * 128;
                const int steps = min(C::kStageK, k_end - k) >> 4;
#pragma unroll
                for (int s = 0; s < C::kStageK / 16; ++s) {
                    if (s >= steps) break;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t dh = d + half * C::kTokens, wh = w + half * 64 + 8 * s;
                        const uint64_t bs = b + (F32 ? 2 * s : (s >> 2) * (C::kPanel >> 4) + 2 * (s & 3));
                        mma_ts(dh, wh, bs, id, s > 0 ? 1 : acc, lead);
                        if (F32) {
                            mma_ts(dh, wh, bs + (C::kPanel >> 4), id, 1, lead);
                            mma_ts(dh, wh + 32, bs, id, 1, lead);
                        }
                    }
                }
                acc = 1;
                mma_commit(&bar.a_empty[a], lead);
                mma_commit(&bar.tok_empty[stage], lead);
                if (k + C::kStageK >= k_end || (F32 && k % 256 == 192)) {
                    mma_commit(&bar.acc_full[sums % C::kSums], lead);
                    ++sums;
                }
                if (++stage == C::kTokenStages) stage = 0, ++round;
            }
        }
        // Products still under way (after a wait that gave up) end before the TMEM is given back.
        if (!ok) {
            mma_commit(&bar.acc_full[sums % C::kSums], lead);
            warp_wait(&bar.acc_full[sums % C::kSums], (sums / C::kSums) & 1, err);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// A matrix tensor as groups of `together` rows (a multiple of 16 bytes), one box the rows of
// one number within 128 / together groups.
cudaError_t weight_map(CUtensorMap* map, const uint8_t* w, int64_t stride, int64_t row_bytes, int rows, int n, int together,
                       int pitch) {
    const int64_t dims[3] = {row_bytes * together, rows / together, n};
    const int64_t strides[2] = {row_bytes * together, stride};
    const int box[3] = {pitch, kHalf / together, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, 3, dims, strides, box);
}

template <bool F32, bool DOWN, bool WIDE>
cudaError_t launch_kernel(const ExpertsMm& m, const ExpertsView& e, const void* hi, const void* lo,
                          int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream) {
    using C = Cfg<F32, WIDE>;
    static SmemOnce once;
    cudaError_t err = once.set(experts_mm_kernel<F32, DOWN, WIDE>, C::kSmem);
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
    err = launch_pdl(experts_mm_kernel<F32, DOWN, WIDE>, dim3(ctas), dim3(kThreads), C::kSmem, stream, w0, w1, t_hi, t_lo, m);
    if (err == cudaSuccess) note_launch();
    return err;
}

}  // namespace

cudaError_t launch_experts_mm(const ExpertsMm& m, const ExpertsView& e, bool down, KvType type, const void* hi,
                              const void* lo, int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream) {
    const bool f32 = type == KvType::kF32, wide = m.K % 256 != 0;
    auto go = [&](auto kernel) { return kernel(m, e, hi, f32 ? lo : hi, n_pieces, dev, stream); };
    if (f32) {
        if (down) return wide ? go(launch_kernel<true, true, true>) : go(launch_kernel<true, true, false>);
        return wide ? go(launch_kernel<true, false, true>) : go(launch_kernel<true, false, false>);
    }
    if (down) return wide ? go(launch_kernel<false, true, true>) : go(launch_kernel<false, true, false>);
    return wide ? go(launch_kernel<false, false, true>) : go(launch_kernel<false, false, false>);
}

}  // namespace qm
