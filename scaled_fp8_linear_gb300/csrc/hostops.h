// hostops.h -- host-side helpers of the operators between the linears
// (norm.cu, gemm_act.cu, moe.cu): alignment checks, launch status, the
// shared-memory allowance of a kernel.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <mutex>

#include "internal.h"

namespace fp8 {
namespace host {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// FP8_OK, or the error of the launches since the last look.
inline int launch_status(const char* what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FP8_OK : set_error(FP8_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// How much dynamic shared memory one kernel has been allowed, per device (the
// last: any other device).
struct SmemAllowance {
    std::mutex mu;
    std::atomic<int> bytes[65] = {};
};

// Allows `kernel` this much dynamic shared memory on the current device.  The
// attribute is a setting, not a maximum, so it is raised with its record under
// one lock and never lowered: a launch of another thread may be on its way.
// `a`: the kernel's own static record.
template <typename Kernel>
int allow_smem(Kernel kernel, int bytes, SmemAllowance& a) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    const bool known = dev >= 0 && dev < 64;   // other devices: set at every call
    std::atomic<int>& allowed = a.bytes[known ? dev : 64];
    if (known && allowed.load(std::memory_order_acquire) >= bytes) return FP8_OK;
    std::lock_guard<std::mutex> lock(a.mu);
    const int was = allowed.load(std::memory_order_relaxed);
    if (known && was >= bytes) return FP8_OK;
    const int most = was > bytes ? was : bytes;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess)
        return set_error(FP8_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    allowed.store(most, std::memory_order_release);
    return FP8_OK;
}

}  // namespace host
}  // namespace fp8
