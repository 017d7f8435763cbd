// pa_q4_write.cu -- pa_cache_write_q4 and pa_rotary_cache_write_q4: new keys
// (turned by their positions, or not) and values into a cache held in 4 bits.
// The kernel is that of pa_rotary.cuh, whose threads quantise their row together
// before they store it: no pass over the new rows of its own.
//
// Bound: instructions.  16384 tokens of 40 heads of 128, K and V turned and all in 4 bits:
// 165 us where the bytes alone would take 113 and the 16-bit write, with a third more
// bytes, takes 150.  K and V alone, not turned: 117 us, the bytes 64.
#include <cuda_runtime.h>

#include "pa.h"
#include "pa_nvtx.cuh"
#include "pa_rotary.cuh"

extern "C" pa_status_t pa_cache_write_q4(const void *key, int64_t key_stride, const void *value,
                                         int64_t value_stride, void *k_cache, void *v_cache,
                                         const int64_t *slot_mapping, int num_tokens,
                                         int num_blocks, int block_size, int num_kv_heads,
                                         int head_dim, pa_dtype_t dtype,
                                         unsigned int *dev_error_word, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_cache_write_q4");
    return pa::rotary_write<true>(nullptr, 0, nullptr, 0, key, key_stride, value, value_stride,
                                  nullptr, nullptr, k_cache, v_cache, slot_mapping, num_tokens,
                                  num_blocks, block_size, 0, num_kv_heads, head_dim, dtype,
                                  dev_error_word, stream);
}

extern "C" pa_status_t pa_rotary_cache_write_q4(
    void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
    const void *key, int64_t key_stride, const void *value, int64_t value_stride,
    const int64_t *positions, const pa_rotary_t *rotary, void *k_cache, void *v_cache,
    const int64_t *slot_mapping, int num_tokens, int num_blocks, int block_size, int num_heads,
    int num_kv_heads, int head_dim, pa_dtype_t dtype, unsigned int *dev_error_word,
    pa_stream_t stream) {
    PA_NVTX_RANGE("pa_rotary_cache_write_q4");
    if (!rotary) return PA_ERR_INVALID_ARG;
    return pa::rotary_write<true>(query_out, query_out_stride, query, query_stride, key,
                                  key_stride, value, value_stride, positions, rotary, k_cache,
                                  v_cache, slot_mapping, num_tokens, num_blocks, block_size,
                                  num_heads, num_kv_heads, head_dim, dtype, dev_error_word,
                                  stream);
}
