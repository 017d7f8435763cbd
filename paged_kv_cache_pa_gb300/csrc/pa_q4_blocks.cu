// pa_q4_blocks.cu -- pa_unpack_blocks_q4: blocks of a 4-bit cache as blocks of a
// 16-bit one, every pair and layer in one launch.
//
// A thread turns one 4-byte word (eight elements of a token's head) into 16
// bytes, in the order of the 16-bit block, so a warp's stores are 512
// contiguous bytes and its loads whole 32-byte sectors.
//
// Bound: HBM, 36 bytes read and 128 written a group of 64 elements.  A thread
// has kUnpackBatch words in flight.  16 layers of 1021 blocks of 8 heads of 128: 219 us,
// 6.3 TB/s, 0.92 of the measured copy; 500 blocks of 8 heads of 64, one layer: 4.9 us, of
// which 3 are the bytes.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_nvtx.cuh"
#include "pa_ptx.cuh"
#include "pa_q4.cuh"

namespace pa {
namespace {

constexpr int kUnpackThreads = 256;
constexpr int kUnpackBatch = 4;

struct UnpackParams {
    const uint8_t *src_k[PA_MAX_LAYERS], *src_v[PA_MAX_LAYERS];
    uint4 *dst_k[PA_MAX_LAYERS], *dst_v[PA_MAX_LAYERS];
    const int64_t *pairs;
    int num_src_blocks, num_dst_blocks;
    unsigned chunks;  // 16-byte pieces of a 16-bit block
    int lg_cpr;       // log2 of a row's
    unsigned int *err;
};

// grid (pair, layer x {K, V}, piece of the block)
template <typename T>
__global__ void __launch_bounds__(kUnpackThreads)
    unpack_blocks_kernel(const __grid_constant__ UnpackParams P) {
    pdl_wait();  // earlier kernels on the stream may still read or write the pools
    pdl_trigger();  // (what follows waits for this grid's end before it writes anything)
    const int64_t src = P.pairs[2 * blockIdx.x], dst = P.pairs[2 * blockIdx.x + 1];
    if (src < 0 || src >= P.num_src_blocks || dst < 0 || dst >= P.num_dst_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && P.err)
            atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
        return;
    }
    const int layer = blockIdx.y >> 1;
    const bool value = blockIdx.y & 1;
    const int cells = 1 << (P.lg_cpr - 3);
    const size_t tile_bytes = (size_t)cells * kQ4CellBytes;
    const size_t tiles = (P.chunks >> P.lg_cpr) / kQ4Tokens;  // of a block
    const uint8_t *s = (value ? P.src_v[layer] : P.src_k[layer]) + (size_t)src * tiles * tile_bytes;
    uint4 *d = (value ? P.dst_v[layer] : P.dst_k[layer]) + (size_t)dst * P.chunks;
    const unsigned i0 = blockIdx.z * (kUnpackThreads * kUnpackBatch) + threadIdx.x;
    uint32_t w[kUnpackBatch], sz[kUnpackBatch];
#pragma unroll
    for (int u = 0; u < kUnpackBatch; ++u) {
        const unsigned i = i0 + u * kUnpackThreads;
        if (i >= P.chunks) break;
        const unsigned row = i >> P.lg_cpr, c = i & ((1u << P.lg_cpr) - 1);
        const uint8_t *cell = s + (row / kQ4Tokens) * tile_bytes + (c >> 3) * kQ4CellBytes;
        const int token = row % kQ4Tokens;
        w[u] = __ldcs(reinterpret_cast<const uint32_t *>(cell + q4_word(token, c & 7)));
        sz[u] = __ldcs(reinterpret_cast<const uint32_t *>(cell + kQ4CellParams + 4 * token));
    }
#pragma unroll
    for (int u = 0; u < kUnpackBatch; ++u) {
        const unsigned i = i0 + u * kUnpackThreads;
        if (i >= P.chunks) break;
        const float2 p = Pack<T>::up(sz[u]);
        d[i] = q4_values8<T>(w[u], p.x, p.y);
    }
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_unpack_blocks_q4(void *const *dst_k_caches, void *const *dst_v_caches,
                                           const void *const *src_k_caches,
                                           const void *const *src_v_caches, int num_layers,
                                           const int64_t *block_pairs, int num_pairs,
                                           int num_dst_blocks, int num_src_blocks, int block_size,
                                           int num_kv_heads, int head_dim, pa_dtype_t dtype,
                                           unsigned int *dev_error_word, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_unpack_blocks_q4");
    using namespace pa;
    if (num_layers <= 0 || num_pairs < 0 || num_dst_blocks <= 0 || num_src_blocks <= 0 ||
        num_kv_heads <= 0)
        return PA_ERR_INVALID_ARG;
    if (num_layers > PA_MAX_LAYERS || q4_block_shift(block_size) < 0) return PA_ERR_UNSUPPORTED;
    if (!is_16bit(dtype)) return PA_ERR_INVALID_ARG;
    if (!head_dim_supported(head_dim)) return PA_ERR_UNSUPPORTED;
    const long long chunks = (long long)num_kv_heads * block_size * head_dim / 8;
    const long long splits = (chunks + kUnpackThreads * kUnpackBatch - 1) / (kUnpackThreads * kUnpackBatch);
    if (splits > 65535) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PA_OK;
    if (!dst_k_caches || !dst_v_caches || !src_k_caches || !src_v_caches || !block_pairs)
        return PA_ERR_INVALID_ARG;
    UnpackParams P = {};
    for (int l = 0; l < num_layers; ++l) {
        for (const void *p : {dst_k_caches[l], dst_v_caches[l], const_cast<void *>(src_k_caches[l]),
                              const_cast<void *>(src_v_caches[l])})
            if (!p || !is_aligned(p, 16)) return PA_ERR_INVALID_ARG;
        P.src_k[l] = (const uint8_t *)src_k_caches[l];
        P.src_v[l] = (const uint8_t *)src_v_caches[l];
        P.dst_k[l] = (uint4 *)dst_k_caches[l];
        P.dst_v[l] = (uint4 *)dst_v_caches[l];
    }
    P.pairs = block_pairs;
    P.num_src_blocks = num_src_blocks;
    P.num_dst_blocks = num_dst_blocks;
    P.chunks = (unsigned)chunks;
    P.lg_cpr = head_dim == 64 ? 3 : head_dim == 128 ? 4 : 5;
    P.err = dev_error_word;
    const dim3 grid((unsigned)num_pairs, (unsigned)(2 * num_layers), (unsigned)splits);
    const cudaError_t e =
        dtype == PA_F16
            ? launch_pdl(unpack_blocks_kernel<__half>, grid, dim3(kUnpackThreads), 0, (cudaStream_t)stream, P)
            : launch_pdl(unpack_blocks_kernel<__nv_bfloat16>, grid, dim3(kUnpackThreads), 0, (cudaStream_t)stream, P);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
