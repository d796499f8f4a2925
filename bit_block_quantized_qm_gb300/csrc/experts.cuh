// What the kernels of qm_experts_q4_0 share.
#pragma once

#include <cuda_bf16.h>

#include "qm_device.cuh"

namespace qm {

// The products run on at most this many CTAs (one per SM): a bound for the
// workspace, whose size the host gives without asking a device.
constexpr int kExpertCtas = 160;
// Most token rows of a tile of the products (f32 rows: half of it).
constexpr int kExpertTokens = 128;

// One of the two products: rows of W (gate and up, or down) with the pieces of token
// rows, sorted by expert.
struct ExpertsMm {
    const int32_t* starts;  // [n + 1] sorted rows of each expert
    const int32_t* order;   // the pair (token * top_k + j) of each sorted row
    const float* unit;      // what a sorted row's pieces are to be multiplied by
    float* out;             // inner [sorted row][rows], or part [pair][rows]
    float* split;           // partial sums of tiles that several CTAs share
    unsigned* counters;     // and how much of each is there
    unsigned int* err;
    const void* x;          // the token rows as they were, for sums done again
    int64_t x_stride;
    const uint8_t* w[2];    // the matrices of a tile's two halves
    int64_t w_stride[2];    // bytes
    int n, K, rows, top_k;
    int activation;
    int split_cols;         // columns of a partial tile
    uint32_t k1024;         // 0x64006400
};

// Values of f16 pieces per row: the contraction's length, padded to whole 128-byte lines.
__host__ __device__ inline int64_t piece_pitch(int K) { return (K + 63) / 64 * 64; }

// The products: pieces `hi` (and `lo` for f32 rows) [n_pieces sorted rows][piece_pitch].
cudaError_t launch_experts_mm(const ExpertsMm& m, const ExpertsView& e, bool down, KvType type, const void* hi,
                              const void* lo, int64_t n_pieces, const DeviceInfo& dev, cudaStream_t stream);

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

}  // namespace qm
