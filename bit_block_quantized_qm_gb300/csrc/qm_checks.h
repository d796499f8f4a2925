// Host-side argument checks that the C ABI's files share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "qm.h"

namespace qm {

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

inline bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    if (a_bytes <= 0 || b_bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(b_bytes) && b0 < a0 + static_cast<uintptr_t>(a_bytes);
}

// The pointer must be device-accessible memory of `device`: device or managed
// memory, or host memory registered/mapped with a device address.
inline int check_pointer(const void* p, int device) {
    cudaPointerAttributes attr;
    cudaError_t err = cudaPointerGetAttributes(&attr, p);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return QM_ERR_POINTER;
    }
    switch (attr.type) {
        case cudaMemoryTypeDevice:
            return attr.device == device ? QM_OK : QM_ERR_POINTER;
        case cudaMemoryTypeManaged:
            return QM_OK;
        case cudaMemoryTypeHost:
            return attr.devicePointer == p ? QM_OK : QM_ERR_POINTER;
        default:
            return QM_ERR_POINTER;
    }
}

inline int from_cuda(cudaError_t err) { return err == cudaSuccess ? QM_OK : QM_ERR_CUDA; }

}  // namespace qm
