// tern_launch.h -- host-side helper of the launchers whose kernels take more
// than 64 KB of dynamic LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace tern {

// Raise a kernel's dynamic-LDS limit once per device and kernel (a per-process
// attribute; not a stream operation).
template <auto Kern>
inline hipError_t raise_lds_limit(size_t lds) {
    if (lds <= 64 * 1024) return hipSuccess;
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done_mask.load(std::memory_order_acquire) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(Kern), hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess) return e;
        done_mask.fetch_or(bit, std::memory_order_acq_rel);
    }
    return hipSuccess;
}

}  // namespace tern
