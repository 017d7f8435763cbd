// pa_q4_decode_launch.cuh -- launches of the 4-bit decode kernels, per head_dim.
#pragma once

#include <atomic>

#include "pa_q4_decode.cuh"

namespace pa {

constexpr int kMaxDevices = 64;

template <typename T, int D, int RT>
cudaError_t launch_q4_decode_rows(const Q4DecodeParams &P, int ctas, bool merge,
                                  cudaStream_t stream) {
    constexpr size_t smem = Q4Shape<D, RT>::kSmem;
    auto kern = q4_decode_kernel<T, D, RT>;
    static std::atomic<bool> set[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_relaxed);
    }
    e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kQ4Threads), smem, stream, P);
    if (e == cudaSuccess && merge)
        e = launch_pdl(q4_merge_kernel<T, D, RT>, dim3((unsigned)ctas * kQ4Warps / kQ4MergeTails),
                       dim3(kQ4MergeThreads), 0,
                       stream, P);
    return e;
}

template <int D>
cudaError_t launch_q4_decode(const Q4DecodeParams &P, int rows, pa_dtype_t dtype, int ctas,
                             bool merge, cudaStream_t stream) {
    auto go = [&](auto t) -> cudaError_t {
        using T = decltype(t);
        if constexpr (D <= 128)
            if (rows == 1) return launch_q4_decode_rows<T, D, 1>(P, ctas, merge, stream);
        if (rows == 2) return launch_q4_decode_rows<T, D, 2>(P, ctas, merge, stream);
        if (rows == 4) return launch_q4_decode_rows<T, D, 4>(P, ctas, merge, stream);
        if (rows == 8) return launch_q4_decode_rows<T, D, 8>(P, ctas, merge, stream);
        if constexpr (D <= 128) return launch_q4_decode_rows<T, D, 16>(P, ctas, merge, stream);
        return cudaErrorInvalidValue;
    };
    return dtype == PA_F16 ? go(__half()) : go(__nv_bfloat16());
}

}  // namespace pa
