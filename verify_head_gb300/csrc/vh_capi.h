// What the C entry points share: checks of their arguments, of the device, and statuses of launches.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/verifyhead.h"

namespace vh {

constexpr int kMaxVocab = 2147483647 - 1023;  // vocabulary of the row operators: tile ends stay in 31 bits
inline bool known_dtype(int d) { return d == VH_F32 || d == VH_BF16 || d == VH_F16; }
inline uintptr_t dtype_size(int d) { return d == VH_F32 ? 4 : 2; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline vh_status check_device() {
    static std::atomic<int> ok_cache[64] = {};  // 1: device already checked
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
        cudaGetLastError();
        return VH_ERR_DEVICE;
    }
    if (dev < 64 && ok_cache[dev].load(std::memory_order_relaxed)) return VH_OK;
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess || major < 10) {
        cudaGetLastError();
        return VH_ERR_DEVICE;
    }
    if (dev < 64) ok_cache[dev].store(1, std::memory_order_relaxed);
    return VH_OK;
}

inline vh_status launch_status(cudaError_t e) {
    if (e == cudaSuccess) return VH_OK;
    cudaGetLastError();  // clear a non-sticky launch error
    return VH_ERR_LAUNCH;
}

}  // namespace vh
