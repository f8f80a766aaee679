// rope_launch.cuh -- what a launch has to know of the current device (host code).
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace rope {

// Multiprocessors of the current device, looked up once per device.
static cudaError_t sm_count(int *sms, int *device)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    int n = known[dev].load(std::memory_order_acquire);
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        known[dev].store(n, std::memory_order_release);
    }
    *sms = n;
    *device = dev;
    return cudaSuccess;
}

// Raises a kernel's shared-memory limit, once per device.
static cudaError_t raise_smem(const void *kernel, int bytes, int device, std::atomic<uint64_t> &raised)
{
    const uint64_t bit = (uint64_t)1 << device;
    if (raised.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        raised.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

}  // namespace rope
