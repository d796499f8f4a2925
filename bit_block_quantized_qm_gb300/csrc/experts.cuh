// What the kernels of qm_experts_q4_0 share.
#pragma once

#include <cuda_bf16.h>

#include "qm.h"
#include "qm_device.cuh"

namespace qm {

// The products run on at most this many CTAs (one per SM): a bound for the
// workspace, whose size the host gives without asking a device.
constexpr int kExpertCtas = 160;
// Most token rows of a tile of the products.
constexpr int kExpertTokens = 128;
constexpr int kExpertHalf = 128;  // weight rows of a half tile
constexpr unsigned kAll = 0xFFFFFFFFu;

// One of the two products: rows of W (gate and up, or down) with the pieces of token
// rows, sorted by expert.
struct ExpertsMm {
    const int32_t* starts;  // [n + 1] sorted rows of each expert
    const float* unit;      // what a sorted row's pieces are to be multiplied by
    float* out;             // [sorted row][rows]
    float* split;           // partial sums of tiles that several CTAs share
    unsigned* counters;     // and how much of each is there
    unsigned int* err;
    const void* half[2];    // what a tile's two halves are of: equal for one matrix, different for gate and up (also
                            // where those are the same memory).  Not read
    int64_t w_stride[2];    // bytes from an expert's matrix to the next
    int n, K, rows;
    int activation;
    int split_cols;         // columns of a partial tile
    uint32_t k1024;         // 0x64006400
    bool early;             // (few rows) this kernel may read weights and `starts` before its wait
    const uint8_t* w[2];    // the halves' matrices
};

// Values of f16 pieces per row: the contraction's length, padded to whole 128-byte lines.
__host__ __device__ inline int64_t piece_pitch(int K) { return (K + 63) / 64 * 64; }

// The products: pieces `hi` (and `lo` for f32 rows) [n_pieces sorted rows][piece_pitch].
cudaError_t launch_experts_mm(const ExpertsMm& m, const ExpertsView& e, bool down, KvType type, const void* hi,
                              const void* lo, int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream);

// The same for few rows an expert.
cudaError_t launch_experts_few(const ExpertsMm& m, const ExpertsView& e, KvType type, const void* hi, const void* lo,
                               const DeviceInfo& dev, cudaStream_t stream);

// EXACT: to a few units of f32; otherwise to about 2^-20.
template <bool EXACT>
__device__ __forceinline__ float activate(float a, int kind) {
    if (kind == QM_ACT_NONE) return a;
    const float z = kind == QM_ACT_SILU ? a : 1.5957691216057308f * (a + 0.044715f * a * a * a);  // tanh(y) = 2 sigmoid(2 y) - 1
    // (The approximate division is off by 2 units, and 0 where the divisor is 2^126 and more.)
    return __fdividef(a, 1.f + (EXACT ? expf(-z) : __expf(-z)));
}

__device__ __forceinline__ bool warp_wait(uint64_t* a, uint32_t pa, unsigned int* err) {
    for (uint32_t i = 0; i < kMaxWaitPolls; ++i)
        if (__all_sync(kAll, mbar_try_wait(a, pa))) return true;
    atomicOr(err, kErrWaitTimeout);
    return false;
}
// A value (>= 0) that all lanes have, in a uniform register: what is computed from it, and the
// branches on it, stay warp-uniform for the compiler too.
__device__ __forceinline__ int uniform(int v) { return static_cast<int>(__reduce_max_sync(kAll, static_cast<unsigned>(v))); }

// What a CTA does, one piece after the other: tiles, each with a range of units.
struct Plan {
    int tiles, full, rest, ku, ctas, cta;
    int each, more;  // units of shared tiles that a CTA has, and how many CTAs have one more
    bool share;  // the tiles left over are shared by all CTAs
    __device__ __forceinline__ int unit_of(int c) const { return c * each + min(c, more); }  // (without a division: it is cold code)
};
struct Item {
    int tile, u0, u1;
};
struct Cursor {
    int next;     // of the whole tiles
    int at, end;  // units of shared tiles
};
__device__ __forceinline__ Cursor first_item(const Plan& p) {
    Cursor c{p.cta, 0, 0};
    if (p.share) c.at = p.unit_of(p.cta), c.end = p.unit_of(p.cta + 1);
    return c;
}
// Shared tiles first: the CTA that comes last to one has others to go on with.
__device__ __forceinline__ bool next_item(const Plan& p, Cursor& c, Item* item) {
    if (c.at < c.end) {
        const int t = c.at / p.ku;
        item->tile = uniform(p.full + t);
        item->u0 = uniform(c.at - t * p.ku);
        item->u1 = uniform(min(p.ku, item->u0 + (c.end - c.at)));
        c.at += item->u1 - item->u0;
        return true;
    }
    if (c.next >= (p.share ? p.full : p.tiles)) return false;
    *item = {uniform(c.next), 0, uniform(p.ku)};
    c.next += p.ctas;
    return true;
}

// What this thread, and those it has met at a barrier, have written before is seen by whoever finds the
// counter changed.  (A fence of every thread and a plain atomic take some 3 us more.)
__device__ __forceinline__ unsigned atom_add_acq_rel(unsigned* p, unsigned n) {
    unsigned before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(before) : "l"(p), "r"(n) : "memory");
    return before;
}

// Where a tile lies: its expert, its block of weight rows, its token rows.
struct Place {
    int expert, block, p0, n;
};

// A matrix tensor as groups of `together` rows (a multiple of 16 bytes), one box the rows of
// one number within 128 / together groups.
inline cudaError_t weight_map(CUtensorMap* map, const uint8_t* w, int64_t stride, int64_t row_bytes, int rows, int n, int together,
                       int pitch) {
    const int64_t dims[3] = {row_bytes * together, rows / together, n};
    const int64_t strides[2] = {row_bytes * together, stride};
    const int box[3] = {pitch, kExpertHalf / together, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, 3, dims, strides, box);
}

}  // namespace qm
