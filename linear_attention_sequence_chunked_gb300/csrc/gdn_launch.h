// What a launch sets up once per kernel and device.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gdn {

// Dynamic shared memory beyond 48 KB (and, `wide`, clusters of more than eight
// blocks) for a kernel, on the first call of each device: the attributes stay, and
// setting them again takes as long as a launch.  `done` belongs to the kernel.
template <typename K>
cudaError_t allow_once(K kernel, size_t smem, bool wide, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess && wide) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace gdn
