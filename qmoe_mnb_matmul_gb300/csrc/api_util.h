// api_util.h -- what the extern "C" entry points share: checks of dtypes,
// alignment and sizes, the device's SM count, status codes (host only).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <cstdlib>

#include "../../include/mnb.h"

namespace mnb {

inline bool valid_dtype(int d) { return d == MNB_F32 || d == MNB_F16 || d == MNB_BF16; }
inline size_t dsize(int d) { return d == MNB_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b without overflow past 2^62 (the largest byte count we accept).
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > (int64_t(1) << 62) / a) return false;
    *out = a * b;
    return true;
}

inline int sm_count_current() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Programmatic dependent launch is on unless MNB_DISABLE_PDL is set in the
// environment (for tools that replay kernels one by one).
inline bool pdl_enabled() {
    static const bool on = std::getenv("MNB_DISABLE_PDL") == nullptr;
    return on;
}

inline mnb_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return MNB_OK;
    if (e == cudaErrorNotSupported) return MNB_ERR_UNSUPPORTED;
    return MNB_ERR_CUDA;
}

}  // namespace mnb
