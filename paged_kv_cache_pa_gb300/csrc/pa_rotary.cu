// pa_rotary.cu -- pa_rotary_init and pa_rotary_cache_write: rotary positions
// on the query and the key, fused with the write of key and value into the
// paged cache (pa_rotary.cuh).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pa.h"
#include "pa_nvtx.cuh"
#include "pa_rotary.cuh"

namespace pa {
namespace {

// frac(|w| / 2 pi) 2^64, rounded to nearest, for |w| < 2^64: with |w| = m 2^e, m
// of 53 bits, and C = floor(2^256 / 2 pi), it is m C 2^(e - 192) modulo 2^64, off
// by |w| 2^-192 before the rounding.
uint64_t turn_fraction(double w) {
    static const uint64_t kC[4] = {0x7f9458eaf7aef158ull, 0x36d8a5664f10e410ull,  // least first
                                   0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};
    int e;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(w), &e), 53);
    const int shift = 192 - (e - 53);  // bits of m C behind the point; 181 or more
    uint64_t p[6] = {};                // m C, one word to spare
    unsigned __int128 carry = 0;
    for (int i = 0; i < 4; ++i) {
        carry += (unsigned __int128)m * kC[i];
        p[i] = (uint64_t)carry;
        carry >>= 64;
    }
    p[4] = (uint64_t)carry;
    auto word = [&](int bit) -> uint64_t {  // 64 bits from `bit` on
        const int i = bit >> 6, r = bit & 63;
        if (i > 4) return 0u;
        return r ? (p[i] >> r) | (p[i + 1] << (64 - r)) : p[i];
    };
    return word(shift) + (word(shift - 1) & 1u);
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_rotary_init(pa_rotary_t *rotary, const double *inv_freq,
                                      const int32_t *axes, int num_pairs, int interleaved,
                                      float scale) {
    if (!rotary || !inv_freq) return PA_ERR_INVALID_ARG;
    if (num_pairs <= 0 || num_pairs % 8 != 0 || num_pairs > PA_MAX_ROTARY_PAIRS)
        return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    pa_rotary_t r;
    std::memset(&r, 0, sizeof(r));
    r.rotary_dim = 2 * num_pairs;
    r.num_axes = 1;
    r.interleaved = interleaved ? 1 : 0;
    r.scale = scale;
    for (int i = 0; i < num_pairs; ++i) {
        if (!(std::fabs(inv_freq[i]) < 0x1p64)) return PA_ERR_INVALID_ARG;
        const int a = axes ? axes[i] : 0;
        if (a < 0 || a >= PA_MAX_ROTARY_AXES) return PA_ERR_INVALID_ARG;
        if (a + 1 > r.num_axes) r.num_axes = a + 1;
        r.axis[i] = (uint8_t)a;
        const uint64_t u = pa::turn_fraction(inv_freq[i]);
        r.turns[i] = inv_freq[i] < 0.0 ? 0u - u : u;
    }
    *rotary = r;
    return PA_OK;
}

extern "C" pa_status_t pa_rotary_cache_write(
    void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
    const void *key, int64_t key_stride, const void *value, int64_t value_stride,
    const int64_t *positions, const pa_rotary_t *rotary, void *k_cache, void *v_cache,
    const int64_t *slot_mapping, int num_tokens, int num_blocks, int block_size, int num_heads,
    int num_kv_heads, int head_dim, pa_dtype_t dtype, unsigned int *dev_error_word,
    pa_stream_t stream) {
    PA_NVTX_RANGE("pa_rotary_cache_write");
    return pa::rotary_write<false>(query_out, query_out_stride, query, query_stride, key,
                                   key_stride, value, value_stride, positions, rotary, k_cache,
                                   v_cache, slot_mapping, num_tokens, num_blocks, block_size,
                                   num_heads, num_kv_heads, head_dim, dtype, dev_error_word,
                                   stream);
}
