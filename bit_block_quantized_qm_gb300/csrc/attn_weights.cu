// Accumulated attention weights of many rows: weights[b][h][j] += the sum over the
// sequence's rows and the query heads of kv head h of exp(s_j - lse), on tcgen05.
//
// The scores are taken again, transposed: a tile of 128 tokens is the M side (a
// TMEM lane, so a thread, per token) and tiles of 128 rows the N side, so a token's
// sum stays in its thread and has one owner and a fixed order.  The keys are
// unpacked once per CTA; the queries come as the f16 pieces that the attention
// kernel before it made of them and left in the workspace (bulk copies of whole
// tiles), with log2 units and the rows' logarithms beside them.
//   f32 rows: the three products of attn_prompt.cu; bf16 rows: the query's one
//   piece by both pieces of the key (here the sums keep f32's bits).
// 2 D flops per row and token and product.  A tile's MMAs need 1.5 K cycles (f32;
// bf16 1 K) and its exponentials 1 K.  Measured: two prompts of 2047 f32 rows,
// window 1024: 87 us, tensor pipe active 54% of the time (150 with masks taken from
// positions in shared memory, 202 also with 8 summing warps); 4096 bf16 rows, causal:
// 140 us, as long as the CTA takes whose tokens all rows see.
//
// A CTA of 18 warps per (sequence, kv head, 128 tokens), the tokens that most rows
// see first: 16 warps sum (four per 32 tokens, a quarter of the rows each), one
// issues the MMAs into two TMEM buffers, one loads.
#include <type_traits>

#include "tcgen05.cuh"

namespace qm {

namespace {

constexpr int kSumWarps = 16;
constexpr int kThreads = (kSumWarps + 2) * 32;
constexpr int kRing = 8;  // row tiles whose factors are kept

template <int D, bool F32>
struct WShape {
    static constexpr int kBlocks = D / 32;
    static constexpr int kPiece = kTile * D * 2;
    static constexpr int kQ = (F32 ? 2 : 1) * kPiece;
    static constexpr int kStages = D == 128 && F32 ? 2 : 4;  // row tiles on their way or in use
    static constexpr int kSmem = 2 * kPiece + kStages * kQ + 1024;
    static_assert(kStages + 2 <= kRing, "a place is free when MMAs two tiles after its own have begun");
};

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    attn_weights_kernel(KvView c, KvRows r, AttnCall a, QueryTiles qt, const float* lse2, uint32_t k1024) {
    using S = WShape<D, F32>;
    constexpr int NB = S::kBlocks;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t q_full[S::kStages], q_empty[S::kStages], s_full[2], s_free[2], f_full[kRing];
    __shared__ uint32_t tmem_slot;
    __shared__ unsigned s_top;
    // Of rows 2 r, 2 r + 1: the units of their scores, minus the log2 of their sums.
    __shared__ __align__(16) float factor[kRing][2 * kTile];
    __shared__ float part_sum[3][kTile];
    uint8_t* base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t* k_sm = base;                 // [2 pieces]
    uint8_t* q_sm = k_sm + 2 * S::kPiece;  // [stages][pieces]
    unsigned int* const err = c.err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], kSumWarps);
        }
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(&f_full[i], 1);
        fence_barrier_init();
        s_top = 0;
    }
    grid_dependency_wait();

    const int lists = c.n_seqs * c.heads;
    const int tt = static_cast<int>(blockIdx.x) / lists, list = static_cast<int>(blockIdx.x) % lists;
    const int b = list / c.heads, h = list % c.heads;
    int first, count;
    kv_rows(r, b, &first, &count, err);
    const int L = kv_length(c, b, err);
    const int group = a.heads / c.heads;
    const int base_pos = L - count;
    const int key0 = tt * kTile;
    // Rows (in tokens) that see some token of the tile.
    const int i_lo = max(0, key0 - base_pos);
    int i_hi = count - 1;
    if (a.window > 0 && key0 >= a.sinks)
        i_hi = min(static_cast<int64_t>(i_hi), static_cast<int64_t>(key0) + kTile - 2 + a.window - base_pos);
    if (key0 >= L || i_lo > i_hi) return;
    const int t_lo = i_lo * group / kTile, t_hi = ((i_hi + 1) * group - 1) / kTile;
    const int64_t tile0 = query_tile(qt, h, first, b, group);  // of the sequence's rows

    // (As in attn_prompt.cu, no CTA that takes its TMEM early fits beside this one.)
    if (warp == kSumWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_addr(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    // The keys: a block of a token per turn; the tile's largest scale to 2^11 .. 2^12.
    constexpr int kTurns = (kTile * NB + kThreads - 1) / kThreads;
    uint4 quants[kTurns];
    uint32_t scale[kTurns];
    uint32_t top = 0;
#pragma unroll
    for (int y = 0; y < kTurns; ++y) {
        const int task = threadIdx.x + y * kThreads;
        const int tok = task & (kTile - 1), blk = task / kTile;
        quants[y] = make_uint4(0, 0, 0, 0);
        scale[y] = 0;
        if (task < kTile * NB && key0 + tok < L) {
            const int64_t off = kv_cell(c, b, h, key0 + tok, err);
            if (off >= 0) {
                quants[y] = *reinterpret_cast<const uint4*>(c.k + off + blk * 256 + (tok & 15) * 16);
                scale[y] = *reinterpret_cast<const uint16_t*>(c.k + off + cell_scales(D) + ((tok & 15) * NB + blk) * 2);
            }
        }
        const uint32_t mag = scale[y] & 0x7FFFu;
        if (mag < 0x7C00u) top = max(top, mag);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) atomicMax(&s_top, top);
    __syncthreads();
    const int up = 26 - max(1, static_cast<int>(s_top >> 10));
#pragma unroll
    for (int y = 0; y < kTurns; ++y) {
        const int task = threadIdx.x + y * kThreads;
        if (task < kTile * NB)
            decode_block<true>(quants[y], f16_bits_to_float(scale[y]) * pow2(up), task & (kTile - 1), task / kTile, k_sm,
                               k_sm + S::kPiece, k1024);
    }
    const float key_unit = pow2(-up);
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp < kSumWarps) {
        const int part = warp >> 2;  // this warp's 32 rows of a row tile
        const int tok = 32 * (warp & 3) + lane, key = key0 + tok;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        // The rows that see this token lie together: from position key on, and (a window)
        // up to key + window - 1.
        const int r_first = min(max(key - base_pos, 0), count) * group;
        const int64_t last = a.window > 0 && key >= a.sinks ? static_cast<int64_t>(key) + a.window - base_pos : count;
        const int r_end = key < L ? static_cast<int>(min(max(last, static_cast<int64_t>(0)), static_cast<int64_t>(count))) * group : 0;
        auto below = [](int n) -> uint32_t { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; };
        float acc = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int t = t_lo, n = 0; t <= t_hi; ++t, ++n) {
            const int buf = n & 1, at = n % kRing;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&f_full[at], (n / kRing) & 1, err) &&
                                             mbar_wait_bounded(&s_full[buf], (n >> 1) & 1, err));
            if (!ok) break;
            tc_fence_after();
            const int col = 32 * part, r0 = t * kTile + col;
            const uint32_t sees = below(r_end - r0) & ~below(r_first - r0);
            if (__any_sync(0xFFFFFFFFu, sees != 0)) {
                float2 sum = make_float2(0.f, 0.f);
                float v[32];
                tmem_ld32(tmem + lanes + 128 * buf + col, v);
                tc_wait_ld();
                // Hidden rows are taken out of the addends, not of the scores: a row whose
                // logarithm is NaN would make NaN of any score.
                auto add = [&](auto masked) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float4 f = *reinterpret_cast<const float4*>(&factor[at][2 * (col + e)]);  // units, then logarithms
                        const float2 x = fma2(make_float2(v[e], v[e + 1]), make_float2(f.x, f.y), make_float2(f.z, f.w));
                        float2 p = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        if (decltype(masked)::value) {
                            if (!((sees >> e) & 1u)) p.x = 0.f;
                            if (!((sees >> (e + 1)) & 1u)) p.y = 0.f;
                        }
                        sum = add2(sum, p);
                    }
                };
                if (__any_sync(0xFFFFFFFFu, sees != ~0u)) add(std::true_type{});
                else add(std::false_type{});
                acc += sum.x + sum.y;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[buf]);
        }
        if (part > 0) part_sum[part - 1][tok] = acc;
        named_barrier_sync(1, kSumWarps * 32);
        if (part == 0 && key < L) {
            float* w = a.weights + (static_cast<int64_t>(b) * c.heads + h) * a.weights_stride + key;
            *w += (acc + part_sum[0][tok]) + (part_sum[1][tok] + part_sum[2][tok]);
        }
    } else if (warp == kSumWarps) {
        {
            const uint32_t lead = elect_one();
            constexpr uint32_t id = idesc_f16(kTile, false);
            bool ok = true;
#pragma unroll 1
            for (int t = t_lo, n = 0; t <= t_hi && ok; ++t, ++n) {
                const int buf = n & 1, stage = n % S::kStages;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&q_full[stage], (n / S::kStages) & 1, err) &&
                                                 (n < 2 || mbar_wait_bounded(&s_free[buf], ((n >> 1) - 1) & 1, err)));
                if (!ok) break;
                tc_fence_after();
                const uint32_t k0 = smem_addr(k_sm), q0 = smem_addr(q_sm + stage * S::kQ);
                constexpr int kProducts = F32 ? 3 : 2;  // low x high, (high x low,) high x high
#pragma unroll 1
                for (int p = 0; p < kProducts; ++p) {
                    const uint64_t da = desc_base(k0 + (p == 0 ? S::kPiece : 0), 16);
                    const uint64_t db = desc_base(q0 + (F32 && p == 1 ? S::kPiece : 0), 16);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t o = static_cast<uint64_t>((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + 128 * buf, da + o, db + o, id, (p | kk) != 0, lead);
                    }
                }
                mma_commit(&q_empty[stage], lead);
                mma_commit(&s_full[buf], lead);
            }
        }
    } else {
        // Loads.  A row's logarithm and unit are read a tile ahead.
        float z[4], u[4];
        auto fetch = [&](int t) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int row = 32 * y + lane, rr = t * kTile + row, i = rr / group;
                z[y] = -INFINITY, u[y] = 0.f;  // no such row
                if (t <= t_hi && rr < count * group) {
                    z[y] = __ldcg(lse2 + static_cast<int64_t>(first + i) * a.heads + h * group + (rr - i * group));
                    u[y] = __ldcg(qt.units + (tile0 + t) * kTile + row);
                }
            }
        };
        fetch(t_lo);
        bool ok = true;
#pragma unroll 1
        for (int t = t_lo, n = 0; t <= t_hi && ok; ++t, ++n) {
            const int stage = n % S::kStages, at = n % kRing;
            // (The MMAs of tile n - kStages came after the sums of two tiles before it.)
            if (n >= S::kStages)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&q_empty[stage], (n / S::kStages - 1) & 1, err));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&q_full[stage], S::kQ);
                bulk_load_1d(q_sm + stage * S::kQ, qt.images + (tile0 + t) * S::kQ, S::kQ, &q_full[stage]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int row = 32 * y + lane;
                // A row that sees nothing adds nothing.  (The unit is never 0: it meets -infinity.)
                const bool sees = z[y] != -INFINITY;
                float* f = &factor[at][4 * (row >> 1) + (row & 1)];
                f[0] = sees ? fmaxf(u[y] * key_unit, 0x1p-100f) : 1.f;
                f[2] = sees ? -z[y] : -INFINITY;
            }
            fetch(t + 1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&f_full[at]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSumWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem) : "memory");
}

template <int D, bool F32>
cudaError_t launch(const KvView& c, const KvRows& r, const AttnCall& a, const QueryTiles& qt, const float* lse2,
                   cudaStream_t stream) {
    using S = WShape<D, F32>;
    static SmemOnce once;
    cudaError_t err = once.set(attn_weights_kernel<D, F32>, S::kSmem);
    if (err != cudaSuccess) return err;
    const int64_t grid = (c.max_len + kTile - 1) / kTile * c.n_seqs * c.heads;
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    note_launch();
    return launch_pdl(attn_weights_kernel<D, F32>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), S::kSmem, stream,
                      c, r, a, qt, lse2, 0x64006400u);
}

}  // namespace

cudaError_t launch_attn_weights(const KvView& c, const KvRows& r, const AttnCall& a, const QueryTiles& qt,
                                const float* lse2, cudaStream_t stream) {
    if (c.dim == 64)
        return a.type == KvType::kF32 ? launch<64, true>(c, r, a, qt, lse2, stream)
                                      : launch<64, false>(c, r, a, qt, lse2, stream);
    return a.type == KvType::kF32 ? launch<128, true>(c, r, a, qt, lse2, stream)
                                  : launch<128, false>(c, r, a, qt, lse2, stream);
}

}  // namespace qm
