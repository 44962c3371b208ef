// smem_limit.h -- dynamic shared memory beyond 48 KB for a kernel, on every device it is launched on.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>

namespace w4 {

// The attribute belongs to the current device's copy of the kernel: raised before the
// first launch there, and known from then on (devices from 64 on: raised each time).  A
// failure is reported and not remembered.  One object for each kernel.
class SmemLimit {
public:
    cudaError_t raise(const void *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
        if (raised_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) raised_.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<uint64_t> raised_{0};
};

}  // namespace w4
