// pa_host.cuh -- host-side argument checks and device facts that several
// entry points share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "pa.h"

namespace pa {

// log2 of a supported pool block size (8 .. 256 tokens, a power of two), or -1
inline int pool_block_shift(int b) {
    for (int sh = 3; sh <= 8; ++sh)
        if (b == (1 << sh)) return sh;
    return -1;
}

inline bool is_aligned(const void *p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool is_16bit(pa_dtype_t t) { return t == PA_F16 || t == PA_BF16; }

inline bool head_dim_supported(int d) { return d == 64 || d == 128 || d == 256; }

inline size_t round_up_256(size_t x) { return (x + 255) / 256 * 256; }

// Streaming multiprocessors of the current device (cached), 0 on an error.
inline int device_sms() {
    constexpr int kMax = 64;
    static std::atomic<int> cached[kMax];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMax) return 0;
    int v = cached[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        cached[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

}  // namespace pa
