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

// One of the two products: rows of W (gate and up, or down) with the pieces of token
// rows, sorted by expert.
struct ExpertsMm {
    const int32_t* starts;  // [n + 1] sorted rows of each expert
    const float* unit;      // what a sorted row's pieces are to be multiplied by
    float* out;             // [sorted row][rows]
    float* split;           // partial sums of tiles that several CTAs share
    unsigned* counters;     // and how much of each is there
    unsigned int* err;
    const uint8_t* w[2];    // the matrices of a tile's two halves
    int64_t w_stride[2];    // bytes
    int n, K, rows;
    int activation;
    int split_cols;         // columns of a partial tile
    uint32_t k1024;         // 0x64006400
};

// Values of f16 pieces per row: the contraction's length, padded to whole 128-byte lines.
__host__ __device__ inline int64_t piece_pitch(int K) { return (K + 63) / 64 * 64; }

// The products: pieces `hi` (and `lo` for f32 rows) [n_pieces sorted rows][piece_pitch].
cudaError_t launch_experts_mm(const ExpertsMm& m, const ExpertsView& e, bool down, KvType type, const void* hi,
                              const void* lo, int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream);

// EXACT: to a few units of f32; otherwise to about 2^-20.
template <bool EXACT>
__device__ __forceinline__ float activate(float a, int kind) {
    if (kind == QM_ACT_NONE) return a;
    const float z = kind == QM_ACT_SILU ? a : 1.5957691216057308f * (a + 0.044715f * a * a * a);  // tanh(y) = 2 sigmoid(2 y) - 1
    // (The approximate division is off by 2 units, and 0 where the divisor is 2^126 and more.)
    return __fdividef(a, 1.f + (EXACT ? expf(-z) : __expf(-z)));
}

}  // namespace qm
