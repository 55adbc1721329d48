// What the translation units of the C ABI (api.cu, rows_api.cu) share: alignment,
// statuses, the current device, and workspaces. Host code only.
#pragma once

#include "kernels.h"

namespace rmsn {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Maps a CUDA result to a status. A failure is also cleared from the
// runtime's last-error slot, so it does not surface in the caller's next,
// unrelated CUDA call.
inline int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return RMSNORM_OK;
    cudaGetLastError();
    return RMSNORM_ERR_CUDA;
}

inline int current_device(const DeviceInfo** out) {
    int dev = -1;
    if (cuda_status(cudaGetDevice(&dev)) != RMSNORM_OK) return RMSNORM_ERR_CUDA;
    *out = device_info(dev);
    return *out ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

// Workspace of a call: the caller's, or one from the stream-ordered allocator.
struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
    bool given = false;

    int take(size_t need, cudaStream_t s) {
        if (given) {
            if (need > 0 && (p == nullptr || bytes < need)) return RMSNORM_ERR_INVALID_ARG;
            return aligned(p, 16) ? RMSNORM_OK : RMSNORM_ERR_MISALIGNED;
        }
        if (need == 0) return RMSNORM_OK;
        return cuda_status(cudaMallocAsync(&p, need, s)) == RMSNORM_OK ? RMSNORM_OK : RMSNORM_ERR_NOMEM;
    }
    int give(int status, cudaStream_t s) {
        if (given || p == nullptr) return status;
        const int freed = cuda_status(cudaFreeAsync(p, s));
        return status != RMSNORM_OK ? status : freed;
    }
};

}  // namespace rmsn
