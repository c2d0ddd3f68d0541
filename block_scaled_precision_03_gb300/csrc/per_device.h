// What has to be done once on each device a process uses.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace bsq {

// Allows a kernel more than 48 KB of dynamic shared memory.  The attribute
// belongs to the kernel on one device, so it is remembered per device; host
// threads may call at the same time (the attribute is then set twice).
class SharedMemory {
    std::atomic<uint64_t> done_{0};

public:
    cudaError_t allow(const void* kernel, int bytes) {
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        const uint64_t bit = device < 64 ? 1ull << device : 0;     // 64 and above: set at every call
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

}  // namespace bsq
