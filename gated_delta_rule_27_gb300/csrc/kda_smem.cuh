// kda_smem.cuh -- a kernel's limit of dynamic shared memory (host code, which a host compiler can take alone).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace kda {

// Lets a kernel use `bytes` of dynamic shared memory on the current device; the runtime is asked only when that is
// more than before.  (A device number past the table asks every time.)  The runtime's limit is what was set last, so
// asking and writing down go under one lock: a smaller size set behind a larger one would make every call between
// the two fail.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
    constexpr int kDevices = 64;
    static std::atomic<int> allowed[kDevices];
    static std::mutex setting;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess || (device < kDevices && allowed[device].load(std::memory_order_acquire) >= bytes)) return e;
    const std::lock_guard<std::mutex> lock(setting);
    if (device < kDevices && allowed[device].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && device < kDevices) allowed[device].store(bytes, std::memory_order_release);
    return e;
}

}  // namespace kda
