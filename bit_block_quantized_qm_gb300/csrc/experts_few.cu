// The experts' products (qm_experts_q4_0) where experts have few rows.
//
//   D[w][c] = sum_b d_wb sum_(k in b) (q_wk - 8) x_ck
//
// Bound: memory, the chosen experts' weights, and close to it the instructions: a warp takes 46 issue
// slots for a block of 16 rows, so 1490 of the 1570 cycles in which memory brings a unit.  One row through 2
// experts of 14336 x 4096 (198 MB) takes 62 us in all, 16 rows through an expert of 4096 x 4096 each 76; the
// copies alone go at 6.8 TB/s, the products of gate and up at 4 to 4.5.
//
// An instruction m16n8k16 takes 16 weight rows (8 of either half of the tile) by 8 columns, each a token
// row's f16 piece (f32 rows have two, next to each other): (q - 8) is exact in f16, the sum over a block is
// scaled by d in f32.  A lane unpacks the four bytes of each of two rows' blocks that its place in the
// fragment asks for, straight from the raw bytes; no unpacked weight is stored anywhere, and no warp waits
// for another but for the copies.
//
// A CTA (one per SM) takes tiles of 256 weight rows by up to 16 columns, in units of 256 elements of K:
// one warp copies units (TMA) and their columns into a ring, sixteen warps have 16 rows each.  An
// expert's tiles with the same weights are next to each other, so that all but the first find them in L2.
// Tiles are dealt out as in experts_mm.cu, and sums that come out infinite or NaN are taken again by the
// kernels that read them.
//
// Every wait is bounded; a wait that gives up sets the device error word.
#include "experts.cuh"
#include "tcgen05.cuh"

namespace qm {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kColumns = 16;
constexpr int kColumnPitch = 512 + 64;  // bytes: a quarter of a warp reads two columns
constexpr int kStages = 4;

template <bool WIDE>
struct Cfg {
    static constexpr int kPitch = WIDE ? 176 : 144;  // bytes of a raw row in shared memory, an odd number of 16s
    static constexpr int kRawBytes = 2 * kExpertHalf * kPitch;
    static constexpr int kStageBytes = kRawBytes + kColumns * kColumnPitch;
    static constexpr int kSmem = kStages * kStageBytes + 128;
};

// Four bytes of quants as (q - 8): the order is that of the token rows' pieces.
__device__ __forceinline__ void unpack(uint32_t q, uint32_t k1024, uint32_t (&n)[4]) {
    const __half2 m1032 = half2_of(0xE408E408u), sixteenth = half2_of(0x2C002C00u), m72 = half2_of(0xD480D480u);
    const uint32_t y = q >> 8;
    n[0] = word(__hadd2(half2_of((q & 0x000F000Fu) | k1024), m1032));
    n[1] = word(__hadd2(half2_of((y & 0x000F000Fu) | k1024), m1032));
    n[2] = word(__hfma2(half2_of((q & 0x00F000F0u) | k1024), sixteenth, m72));
    n[3] = word(__hfma2(half2_of((y & 0x00F000F0u) | k1024), sixteenth, m72));
}

__device__ __forceinline__ void mma16816(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// A lane's two rows of a unit, its blocks 0 .. blocks - 1, with GROUPS x 8 columns.
template <int GROUPS, bool WIDE>
__device__ __forceinline__ void unit_sums(const uint8_t* row0, const uint8_t* row1, bool odd, const uint8_t* column, int t,
                                          int blocks, uint32_t k1024, float (&acc)[2][4]) {
    // (A row starts at a multiple of 4 bytes, or, where `odd`, 2 bytes after one.)
    const uint32_t even_sel = WIDE && odd ? 0x7654u : 0x5432u, odd_sel = WIDE && odd ? 0x5432u : 0x3210u;
    auto words = [&](const uint8_t* row, int at, uint32_t sel) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row + at) + t;
        return __byte_perm(p[0], p[1], sel);
    };
    auto scale = [&](const uint8_t* row, int at) {
        return f16_bits_to_float(*reinterpret_cast<const uint16_t*>(row + at + (WIDE && odd ? 2 : 0)));
    };
    auto block = [&](int b, uint32_t q0, uint32_t q1, float d0, float d1) {
        uint32_t n0[4], n1[4];
        unpack(q0, k1024, n0);
        unpack(q1, k1024, n1);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const uint4 x = *reinterpret_cast<const uint4*>(column + g * 8 * kColumnPitch + b * 64 + t * 16);
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            float s[4];
            mma16816(s, zero, n0[0], n1[0], n0[1], n1[1], x.x, x.y);
            mma16816(s, s, n0[2], n1[2], n0[3], n1[3], x.z, x.w);
            acc[g][0] = fmaf(d0, s[0], acc[g][0]);
            acc[g][1] = fmaf(d0, s[1], acc[g][1]);
            acc[g][2] = fmaf(d1, s[2], acc[g][2]);
            acc[g][3] = fmaf(d1, s[3], acc[g][3]);
        }
    };
    auto even_block = [&](int b) {
        const int at = 18 * b;
        block(b, words(row0, at, even_sel), words(row1, at, even_sel), scale(row0, at), scale(row1, at));
    };
    auto odd_block = [&](int b) {
        const int at = 18 * (b - 1) + 20;
        uint32_t q0, q1;
        if constexpr (WIDE) {
            q0 = words(row0, at, odd_sel), q1 = words(row1, at, odd_sel);
        } else {
            q0 = *(reinterpret_cast<const uint32_t*>(row0 + at) + t), q1 = *(reinterpret_cast<const uint32_t*>(row1 + at) + t);
        }
        block(b, q0, q1, scale(row0, at - 2), scale(row1, at - 2));
    };
    if (!WIDE || blocks == 8) {
#pragma unroll 2
        for (int b = 0; b < 8; b += 2) {
            even_block(b);
            odd_block(b + 1);
        }
    } else {
#pragma unroll 1
        for (int b = 0; b < blocks; b += 2) {
            even_block(b);
            if (b + 1 < blocks) odd_block(b + 1);
        }
    }
}

// A TMA box that is read once: the first to leave L2.
__device__ __forceinline__ void tma_load_3d_once(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b64 once;\n\t"
        "createpolicy.fractional.L2::evict_first.b64 once;\n\t"
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], once;\n\t}" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

struct Barriers {
    uint64_t full[kStages], empty[kStages];
};

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    experts_few_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1, const void* hi,
                       const void* lo, const ExpertsMm m) {
    using C = Cfg<WIDE>;
    constexpr int kTokens = F32 ? kColumns / 2 : kColumns;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((128 - (smem_addr(smem_raw) & 127)) & 127);
    __shared__ Barriers bar;
    __shared__ int tiles_before[1024 + 1];  // token tiles of all lower experts
    __shared__ int rows_before[1024 + 1];   // their sorted rows
    __shared__ Plan plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned int* const err = m.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], kWarps);
        }
        fence_barrier_init();
    }
    if (warp == kWarps && lane == 0) {
        prefetch_tensormap(&map_w0);
        prefetch_tensormap(&map_w1);
    }
    // The down product begins before the kernel that makes its columns has ended: with whose weights, the
    // setup has said, which has ended long since (the kernel between them begins when all CTAs of the first
    // product are past their wait for it).
    if (!m.early) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    const bool two = m.half[0] != m.half[1];  // gate and up
    const int block_rows = two ? kExpertHalf : 2 * kExpertHalf;
    const int blocks = (m.rows + block_rows - 1) / block_rows;
    for (int e = threadIdx.x; e <= m.n; e += kThreads) rows_before[e] = __ldcg(m.starts + e);
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
        for (int e0 = 0; e0 < m.n; e0 += 32) {
            const int e = e0 + lane;
            const int count = e < m.n ? rows_before[e + 1] - rows_before[e] : 0;
            int v = (count + kTokens - 1) / kTokens;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kAll, v, d);
                if (lane >= d) v += o;
            }
            if (e < m.n) tiles_before[e + 1] = sum + v;
            sum += __shfl_sync(kAll, v, 31);
        }
        if (lane == 0) {
            tiles_before[0] = 0;
            Plan p;
            p.tiles = sum * blocks;
            p.ctas = gridDim.x;
            p.cta = blockIdx.x;
            p.ku = (m.K + 255) / 256;
            p.full = p.tiles / p.ctas * p.ctas;
            p.rest = p.tiles - p.full;
            p.each = p.rest * p.ku / p.ctas;
            p.more = p.rest * p.ku - p.each * p.ctas;
            // Sharing the tiles left over saves ku (ctas - rest) / ctas units, and costs what 5 do (8 of 64 experts of
            // 2048 x 1408, where it saves 3.4: 31 us without against 33; with 2 experts of 14336 x 4096, where it saves
            // 8.4, 66 without against 62).  So a CTA has less than a tile of them.
            p.share = p.rest > 0 && p.ku * (p.ctas - p.rest) > 5 * p.ctas;
            plan = p;
        }
    }
    __syncthreads();

    auto place = [&](int tile) {
        int lo = 0, hi = m.n;  // the first expert with tiles_before[e + 1] * blocks > tile
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tiles_before[mid + 1] * blocks <= tile) lo = mid + 1;
            else hi = mid;
        }
        const int first = tiles_before[lo], count = tiles_before[lo + 1] - first;
        const int block = (tile - first * blocks) / count, of = tile - first * blocks - block * count;
        Place p;
        p.expert = uniform(lo);
        p.block = uniform(block);
        p.p0 = uniform(rows_before[lo] + of * kTokens);
        p.n = uniform(min(kTokens, rows_before[lo + 1] - p.p0));
        return p;
    };
    const int row_bytes = m.K / 32 * 18;
    const int together = WIDE ? 16 / (row_bytes & -row_bytes) : 1;
    Cursor cur = first_item(plan);
    Item item;
    bool ok = true;

    if (warp == kWarps) {
        // ---- copies
        uint32_t it = 0;
        const int64_t pitch = piece_pitch(m.K) * 2;
        const uint8_t* pieces = static_cast<const uint8_t*>(F32 && (lane & 1) ? lo : hi);
        auto column_bytes = [&](int u) {
            const int64_t left = pitch - 512 * static_cast<int64_t>(u);
            return left < 512 ? static_cast<uint32_t>(left) : 512u;
        };
        auto copy_weights = [&](const Place& pl, int u, int stage) {
            uint8_t* dst = ring + stage * C::kStageBytes;
            if (lane == 0)
                mbar_arrive_expect_tx(&bar.full[stage], C::kRawBytes + (F32 ? 2 * pl.n : pl.n) * column_bytes(u));
            __syncwarp();
            // Lanes i and 16 + i: the rows i of each group of the two halves.
            const int i = lane & 15, half = lane >> 4;
            if (i < together) {
                const int row0 = pl.block * block_rows + (two ? 0 : half * kExpertHalf);
                tma_load_3d_once(dst + (half * kExpertHalf + i * (kExpertHalf / together)) * C::kPitch, half ? &map_w1 : &map_w0,
                                 (i * row_bytes & ~15) + 144 * u, row0 / together, pl.expert, &bar.full[stage]);
            }
        };
        uint32_t ahead = 0;  // units whose weights are on their way before the wait
        if (m.early) {
            Cursor first = cur;
            while (ahead < kStages && next_item(plan, first, &item)) {
                const Place pl = place(item.tile);
                for (int u = item.u0; u < item.u1 && ahead < kStages; ++u, ++ahead) copy_weights(pl, u, ahead);
            }
            grid_dependency_wait();
            grid_launch_dependents();
        }
        while (ok && next_item(plan, cur, &item)) {
            const Place pl = place(item.tile);
            for (int u = item.u0; u < item.u1; ++u, ++it) {
                const int stage = it % kStages;
                if (it >= kStages) ok = warp_wait(&bar.empty[stage], (it / kStages - 1) & 1, err);
                if (!ok) break;
                if (it >= ahead) copy_weights(pl, u, stage);
                if (lane < (F32 ? 2 * pl.n : pl.n))
                    bulk_load_1d(ring + stage * C::kStageBytes + C::kRawBytes + lane * kColumnPitch,
                                 pieces + (pl.p0 + (F32 ? lane >> 1 : lane)) * pitch + 512 * static_cast<int64_t>(u),
                                 column_bytes(u), &bar.full[stage]);
                __syncwarp();
            }
        }
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)  // what is still on its way
            mbar_wait_bounded(&bar.full[i % kStages], (i / kStages) & 1, err);
        return;
    }

    // ---- sums: this warp's 8 rows of either half
    const int g = lane >> 2, t = lane & 3;
    const int slot = 8 * warp + g;  // of a half's rows in shared memory: those of a number in their group together
    const int number = WIDE ? slot / (kExpertHalf / together) : 0;
    const int r = WIDE ? slot % (kExpertHalf / together) * together + number : slot;  // the row
    const int shift = number * row_bytes & 15;
    const bool odd = shift & 2;
    const int row_at = slot * C::kPitch + (shift & ~3);
    constexpr int kValues = F32 ? 4 : 8;  // sums of a thread: [columns of a group of 8][both halves]
    int stage = 0;
    uint32_t parity = 0;
    constexpr int64_t place_floats = 8 * kWarps * 32;  // (the workspace has room for 256 rows by 16 columns and more)
    if (m.early) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    // The sums of a tile, scaled and activated.
    auto store = [&](const Place& pl, float(&v)[kValues]) {
        const int f0 = pl.block * block_rows + r, f1 = two ? f0 : f0 + kExpertHalf;
        const bool in0 = f0 < m.rows, in1 = !two && f1 < m.rows;
#pragma unroll
        for (int i = 0; i < kValues; i += 2) {
            const int c = F32 ? 4 * (i >> 1) + t : 8 * (i >> 2) + 2 * t + (i >> 1 & 1);
            if (c >= pl.n) continue;
            const float unit = m.unit[pl.p0 + c];
            float a = v[i] * unit, b = v[i + 1] * unit;
            a = activate<F32>(a, m.activation);
            if (two) a *= b;
            else b = activate<F32>(b, m.activation);
            float* out = m.out + static_cast<int64_t>(pl.p0 + c) * m.rows;
            if (in0) out[f0] = a;
            if (in1) out[f1] = b;
        }
    };
    // CTA c's part of the shared tile that begins with unit `begin`: the second one where the CTA begins before it.
    auto part_of = [&](int c, int begin) {
        return m.split + (2 * c + (plan.unit_of(c) < begin)) * place_floats + threadIdx.x;
    };
    while (next_item(plan, cur, &item)) {
        const Place pl = place(item.tile);
        const bool many = (F32 ? 2 * pl.n : pl.n) > 8;
        float acc[2][4] = {};
        for (int u = item.u0; u < item.u1; ++u) {
            ok = ok && warp_wait(&bar.full[stage], parity, err);
            const uint8_t* raw = ring + stage * C::kStageBytes;
            const uint8_t* row0 = raw + row_at;
            const uint8_t* row1 = row0 + kExpertHalf * C::kPitch;
            const uint8_t* column = raw + C::kRawBytes + g * kColumnPitch;
            const int n_blocks = min(8, m.K / 32 - 8 * u);
            if (many) unit_sums<2, WIDE>(row0, row1, odd, column, t, n_blocks, m.k1024, acc);
            else unit_sums<1, WIDE>(row0, row1, odd, column, t, n_blocks, m.k1024, acc);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.empty[stage]);
            if (++stage == kStages) stage = 0, parity ^= 1;
        }
        // F32: columns 2 t and 2 t + 1 are a row's pieces.
        float v[kValues];
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if constexpr (F32) {
                v[2 * c] = acc[c][0] + acc[c][1], v[2 * c + 1] = acc[c][2] + acc[c][3];
            } else {
                v[4 * c] = acc[c][0], v[4 * c + 1] = acc[c][2], v[4 * c + 2] = acc[c][1], v[4 * c + 3] = acc[c][3];
            }
        if (item.u1 - item.u0 == plan.ku) {
            store(pl, v);
        } else {
            float* mine = part_of(plan.cta, (item.tile - plan.full) * plan.ku);
#pragma unroll
            for (int i = 0; i < kValues; ++i) mine[i * kWarps * 32] = v[i];
        }
    }
    // The parts of shared tiles: a warp's meet those of the same warp of other CTAs, and the warp that comes
    // last adds them, in the CTAs' order.  Here, behind all of the CTA's copies: among them, whatever goes
    // to memory and back takes 5 us, and all of the CTA would wait.
    const int from = plan.share ? plan.unit_of(plan.cta) : 0, to = plan.share ? plan.unit_of(plan.cta + 1) : 0;
    if (from == to) return;
    // (A CTA's units are less than a tile's: they are of two tiles at most, which lanes 0 and 1 count in.)
    const int first_tile = from / plan.ku, begin = (first_tile + lane) * plan.ku;
    bool last = false;
    __syncwarp();
    if (lane < 2 && begin < to) {
        const unsigned n = static_cast<unsigned>(min(to, begin + plan.ku) - max(from, begin));
        last = n != static_cast<unsigned>(plan.ku) &&  // (a whole tile after all: stored above)
               atom_add_acq_rel(&m.counters[(first_tile + lane) * kWarps + warp], n) + n == static_cast<unsigned>(plan.ku);
    }
    const unsigned lasts = __ballot_sync(kAll, last);
    __syncwarp();
#pragma unroll 1
    for (int shared_tile = first_tile; shared_tile < first_tile + 2; ++shared_tile) {
        if (!(lasts >> (shared_tile - first_tile) & 1)) continue;
        const int begin = shared_tile * plan.ku;
        int c = plan.cta;
        while (plan.unit_of(c) > begin) --c;
        float v[kValues] = {};
        while (plan.unit_of(c) < begin + plan.ku) {  // four parts on their way at a time
            float a[4][kValues];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool there = plan.unit_of(c + i) < begin + plan.ku;
                const float* part = part_of(there ? c + i : c, begin);
#pragma unroll
                for (int k = 0; k < kValues; ++k) a[i][k] = there ? __ldcg(part + k * kWarps * 32) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < kValues; ++k) v[k] += a[i][k];
            c += 4;
        }
        store(place(plan.full + shared_tile), v);
    }
}

template <bool F32, bool WIDE>
cudaError_t launch_kernel(const ExpertsMm& m, const ExpertsView& e, const void* hi, const void* lo, const DeviceInfo& dev,
                          cudaStream_t stream) {
    using C = Cfg<WIDE>;
    static SmemOnce once;
    cudaError_t err = once.set(experts_few_kernel<F32, WIDE>, C::kSmem);
    if (err != cudaSuccess) return err;
    const int64_t row_bytes = m.K / 32 * 18;
    const int together = WIDE ? 16 / static_cast<int>(row_bytes & -row_bytes) : 1;
    CUtensorMap w0, w1;
    if ((err = weight_map(&w0, m.w[0], m.w_stride[0], row_bytes, m.rows, e.n, together, C::kPitch)) != cudaSuccess) return err;
    if ((err = weight_map(&w1, m.w[1], m.w_stride[1], row_bytes, m.rows, e.n, together, C::kPitch)) != cudaSuccess) return err;
    const int ctas = dev.sm_count < kExpertCtas ? dev.sm_count : kExpertCtas;
    err = launch_pdl(experts_few_kernel<F32, WIDE>, dim3(ctas), dim3(kThreads), C::kSmem, stream, w0, w1, hi, lo, m);
    if (err == cudaSuccess) note_launch();
    return err;
}

}  // namespace

cudaError_t launch_experts_few(const ExpertsMm& m, const ExpertsView& e, KvType type, const void* hi, const void* lo,
                               const DeviceInfo& dev, cudaStream_t stream) {
    const bool wide = m.K % 256 != 0;
    if (type == KvType::kF32)
        return wide ? launch_kernel<true, true>(m, e, hi, lo, dev, stream) : launch_kernel<true, false>(m, e, hi, lo, dev, stream);
    return wide ? launch_kernel<false, true>(m, e, hi, lo, dev, stream) : launch_kernel<false, false>(m, e, hi, lo, dev, stream);
}

}  // namespace qm
