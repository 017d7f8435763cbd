// pa_rotary.cu -- pa_rotary_init and pa_rotary_cache_write: rotary positions
// on the query and the key, fused with the write of key and value into the
// paged cache.
//
// What it computes: pair i (of rotary_dim / 2) of a head has the angular
// frequency w_i and takes its position from axis a_i; token t turns it by
//     angle = position[a_i][t] * w_i,
//     (x, y) -> scale * (x cos - y sin, y cos + x sin),
// with (x, y) the elements (i, i + rotary_dim / 2) or, interleaved,
// (2i, 2i + 1) of the head; elements from rotary_dim on pass through.
//
// Angles.  Only the angle's fraction of a turn matters, and positions are
// whole numbers, so the frequency is kept as a 64-bit binary fraction of a
// turn, F = frac(w / 2 pi) 2^64: the product position * F modulo 2^64 (one
// wrapping integer multiply) is the fraction of a turn, where a 32-bit product
// w * position is off by 0.03 rad at position 10^6.  F is w / 2 pi rounded to 64
// bits once (turn_fraction: a double holds the quotient to 2^-53 of itself only,
// 2^-25 of a turn at position 2^30 already), so the fraction is off by
// |position| 2^-65 turns, less than the one rounding to 32 bits that follows up
// to positions of 2^40.  Read as a signed number, it goes to sincospi.
//
// Bound: HBM.  Every row is read once and written once.  A row of head_dim
// elements belongs to head_dim / 16 threads of two 16-byte chunks each, the
// two halves of its eight pairs (or two neighbouring chunks when interleaved
// or past rotary_dim), so a rotation never leaves its thread.  A token's
// sines and cosines are computed once a CTA, for all its heads, while its
// first rows are in flight.  A CTA takes as many tokens as give each thread
// four rows, unless that leaves fewer than two CTAs an SM: with few rows a
// token (grouped queries) one row a thread is one round trip to memory a CTA
// and half the rate (4099 tokens of 12 + 2 + 2 heads of 128: 12.4 us with four
// rows, 3.4 more with one).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_nvtx.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotBatch = 4;  // rows a thread has in flight

struct RotaryParams {
    const uint4 *q, *k, *v;
    uint4 *q_out, *k_cache, *v_cache;
    long long q_stride, k_stride, v_stride, q_out_stride;  // 16-byte chunks between tokens
    const int64_t *positions;                              // [num_axes][num_tokens]
    const int64_t *slot_mapping;
    long long num_slots;
    int num_tokens, num_heads, num_kv_heads, block_shift;
    int lg_lpr;        // log2 of a row's threads (head_dim / 16)
    int lg_rows;       // log2 of the rows a token's threads take at once
    int rounds;        // tokens a thread takes, one after the other
    unsigned int *err;
    pa_rotary_t rot;
};

template <typename T>
struct Pack;
template <>
struct Pack<__half> {
    static __device__ __forceinline__ float2 up(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Pack<__nv_bfloat16> {
    static __device__ __forceinline__ float2 up(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Eight pairs: x in chunk a and y in chunk b, element by element.
template <typename T>
__device__ __forceinline__ void turn_halves(uint4 &a, uint4 &b, const float2 (&cs)[8]) {
    uint32_t *pa_ = reinterpret_cast<uint32_t *>(&a), *pb = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = Pack<T>::up(pa_[i]), y = Pack<T>::up(pb[i]);
        const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
        pa_[i] = Pack<T>::down(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
        pb[i] = Pack<T>::down(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
    }
}

// Four pairs of neighbouring elements.
template <typename T>
__device__ __forceinline__ void turn_neighbours(uint4 &a, const float2 *cs) {
    uint32_t *p = reinterpret_cast<uint32_t *>(&a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = Pack<T>::up(p[i]);
        p[i] = Pack<T>::down(x.x * cs[i].x - x.y * cs[i].y, x.y * cs[i].x + x.x * cs[i].y);
    }
}

// A CTA takes `rounds` times 256 / (threads a row * rows at once) tokens; thread
// = (token, row, unit j of the row).  A token's rows are its query heads, its
// key heads and its value heads; a thread goes through its rows of all its
// tokens as one list, four at a time.
template <typename T, bool IL>
__global__ void __launch_bounds__(kRotThreads)
    rotary_cache_write_kernel(const __grid_constant__ RotaryParams P) {
    extern __shared__ __align__(16) float2 s_cs[];  // [token][pair]
    const int lpr = 1 << P.lg_lpr, rows_at_once = 1 << P.lg_rows;
    const int j = threadIdx.x & (lpr - 1);
    const int r0 = ((int)threadIdx.x >> P.lg_lpr) & (rows_at_once - 1);
    const int tl = (int)threadIdx.x >> (P.lg_lpr + P.lg_rows);
    const int lanes = kRotThreads >> (P.lg_lpr + P.lg_rows);  // tokens at once
    const int tokens = lanes * P.rounds;
    const long long t0 = (long long)blockIdx.x * tokens;
    const int H = P.num_heads, Hkv = P.num_kv_heads, rows = H + 2 * Hkv;
    const int pairs = P.rot.rotary_dim / 2, rot_units = pairs / 8;
    // The frequencies from shared memory: lanes that read different parameters
    // are served one after the other, which for several tokens a CTA is most of
    // the time until the angles are there (4099 tokens of 12 + 2 + 2 heads of
    // 128: 12.4 us, 14.4 without).
    __shared__ uint64_t s_turns[PA_MAX_ROTARY_PAIRS];
    __shared__ uint8_t s_axis[PA_MAX_ROTARY_PAIRS];
    const bool staged = tokens > 1;
    if (staged && threadIdx.x < pairs) {
        s_turns[threadIdx.x] = P.rot.turns[threadIdx.x];
        s_axis[threadIdx.x] = P.rot.axis[threadIdx.x];
    }
    pdl_wait();  // earlier kernels on the stream may still read or write what this touches
    pdl_trigger();  // (after the wait: what follows may start before this grid ends, not before those)

    // this thread's two chunks of a row
    int ca, cb;
    if (IL || j >= rot_units) {
        ca = 2 * j;
        cb = 2 * j + 1;
    } else {
        ca = j;
        cb = j + rot_units;
    }
    const int lg_cpr = P.lg_lpr + 1;  // log2 of a row's chunks
    // the thread's place in its list: token of the CTA and row
    struct At {
        int tok, r;
    };
    auto next = [&](At &p) {
        p.r += rows_at_once;
        if (p.r >= rows) {
            p.r = r0;
            p.tok += lanes;
        }
    };
    auto in_list = [&](const At &p) { return p.tok < tokens && t0 + p.tok < P.num_tokens; };
    uint4 a[kRotBatch], b[kRotBatch];
    int64_t slot[kRotBatch];
    auto load = [&](At p) {
#pragma unroll
        for (int u = 0; u < kRotBatch; ++u, next(p)) {
            if (!in_list(p)) break;
            const long long t = t0 + p.tok;
            const int r = p.r;
            slot[u] = r < H ? 0 : P.slot_mapping[t];
            const uint4 *src = r < H ? P.q + t * P.q_stride + ((size_t)r << lg_cpr)
                               : r < H + Hkv ? P.k + t * P.k_stride + ((size_t)(r - H) << lg_cpr)
                                             : P.v + t * P.v_stride + ((size_t)(r - H - Hkv) << lg_cpr);
            a[u] = __ldcs(src + ca);
            b[u] = __ldcs(src + cb);
        }
    };
    At at = {tl, r0};
    if (r0 >= rows) at.tok = tokens;  // more threads than rows
    load(at);

    // sines and cosines of the CTA's tokens, once each
    if (staged) __syncthreads();
    for (int i = threadIdx.x; i < tokens * pairs; i += kRotThreads) {
        const int tok = i / pairs, pr = i - tok * pairs;
        const long long t = t0 + tok;
        if (t < P.num_tokens) {
            const int axis = staged ? s_axis[pr] : P.rot.axis[pr];
            const int64_t pos = P.positions[(size_t)axis * P.num_tokens + t];
            const uint64_t turn =  // modulo one turn
                (uint64_t)pos * (staged ? s_turns[pr] : P.rot.turns[pr]);
            float s, c;
            sincospif(__ll2float_rn((long long)turn) * 0x1p-63f, &s, &c);
            s_cs[i] = make_float2(c * P.rot.scale, s * P.rot.scale);
        }
    }
    __syncthreads();
    const bool turns = j < rot_units;
    while (in_list(at)) {
        At p = at;
#pragma unroll
        for (int u = 0; u < kRotBatch; ++u, next(p)) {
            if (!in_list(p)) break;
            const long long t = t0 + p.tok;
            const int r = p.r;
            if (turns && r < H + Hkv) {
                float2 cs[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    *reinterpret_cast<float4 *>(&cs[e]) =
                        *reinterpret_cast<const float4 *>(&s_cs[p.tok * pairs + 8 * j + e]);
                if (IL) {
                    turn_neighbours<T>(a[u], cs);
                    turn_neighbours<T>(b[u], cs + 4);
                } else {
                    turn_halves<T>(a[u], b[u], cs);
                }
            }
            uint4 *dst;
            if (r < H) {
                dst = P.q_out + t * P.q_out_stride + ((size_t)r << lg_cpr);
            } else {
                if (slot[u] < 0) continue;  // padding
                if (slot[u] >= P.num_slots) {
                    if (r == H && j == 0 && P.err) atomicOr(P.err, PA_ERRBIT_SLOT_OOB);
                    continue;
                }
                const int h = r < H + Hkv ? r - H : r - H - Hkv;
                dst = (r < H + Hkv ? P.k_cache : P.v_cache) +
                      ((((((size_t)(slot[u] >> P.block_shift) * Hkv) + h) << P.block_shift) +
                        (size_t)(slot[u] & ((1 << P.block_shift) - 1)))
                       << lg_cpr);
            }
            dst[ca] = a[u];
            dst[cb] = b[u];
        }
        at = p;
        load(at);
    }
}

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

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
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
    using namespace pa;
    if (num_tokens < 0 || num_blocks <= 0 || num_heads <= 0 || num_kv_heads <= 0 || !rotary)
        return PA_ERR_INVALID_ARG;
    const int shift = pool_block_shift(block_size);
    if (shift < 0) return PA_ERR_UNSUPPORTED;
    if (!is_16bit(dtype)) return PA_ERR_INVALID_ARG;
    if (!head_dim_supported(head_dim)) return PA_ERR_UNSUPPORTED;
    if (rotary->rotary_dim <= 0 || rotary->rotary_dim % 16 != 0 || rotary->rotary_dim > head_dim ||
        rotary->num_axes < 1 || rotary->num_axes > PA_MAX_ROTARY_AXES)
        return PA_ERR_INVALID_ARG;
    for (int i = 0; i < rotary->rotary_dim / 2; ++i)
        if (rotary->axis[i] >= rotary->num_axes) return PA_ERR_INVALID_ARG;
    if ((long long)num_heads + 2ll * num_kv_heads > (1 << 20)) return PA_ERR_UNSUPPORTED;
    const long long q_row = (long long)num_heads * head_dim;
    const long long kv_row = (long long)num_kv_heads * head_dim;
    if (query_stride < q_row || query_out_stride < q_row || key_stride < kv_row ||
        value_stride < kv_row || query_stride % 8 || query_out_stride % 8 || key_stride % 8 ||
        value_stride % 8)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!query_out || !query || !key || !value || !positions || !k_cache || !v_cache ||
        !slot_mapping)
        return PA_ERR_INVALID_ARG;
    for (const void *p : {(const void *)query_out, query, key, value, (const void *)k_cache,
                          (const void *)v_cache})
        if (!is_aligned(p, 16)) return PA_ERR_INVALID_ARG;

    RotaryParams P;
    P.q = (const uint4 *)query;
    P.k = (const uint4 *)key;
    P.v = (const uint4 *)value;
    P.q_out = (uint4 *)query_out;
    P.k_cache = (uint4 *)k_cache;
    P.v_cache = (uint4 *)v_cache;
    P.q_stride = query_stride / 8;
    P.k_stride = key_stride / 8;
    P.v_stride = value_stride / 8;
    P.q_out_stride = query_out_stride / 8;
    P.positions = positions;
    P.slot_mapping = slot_mapping;
    P.num_slots = (long long)num_blocks << shift;
    P.num_tokens = num_tokens;
    P.num_heads = num_heads;
    P.num_kv_heads = num_kv_heads;
    P.block_shift = shift;
    P.lg_lpr = log2_of(head_dim / 16);
    // rows a token's threads take at once: all of them, up to the CTA
    const int max_rows = kRotThreads >> P.lg_lpr;
    const int rows = num_heads + 2 * num_kv_heads;
    P.lg_rows = log2_of(rows < max_rows ? rows : max_rows);
    P.err = dev_error_word;
    P.rot = *rotary;
    // tokens a CTA: enough for four rows a thread, while two CTAs an SM are left
    const int lanes = kRotThreads >> (P.lg_lpr + P.lg_rows);
    const int groups = (rows + (1 << P.lg_rows) - 1) >> P.lg_rows;  // rows a thread and token
    const int sms = device_sms();
    if (sms <= 0) return PA_ERR_CUDA;
    P.rounds = 1;
    while (P.rounds * groups < kRotBatch &&
           (long long)num_tokens >= 2ll * sms * lanes * (2 * P.rounds))
        P.rounds *= 2;
    const int tokens = lanes * P.rounds;
    const dim3 grid((unsigned)((num_tokens + tokens - 1) / tokens));
    // at most 256 / 4 units of 8 pairs at once (a token has three rows at
    // least), four rounds: 16 KB
    const size_t smem = (size_t)tokens * (rotary->rotary_dim / 2) * sizeof(float2);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (dtype == PA_F16)
        e = rotary->interleaved
                ? launch_pdl(rotary_cache_write_kernel<__half, true>, grid, dim3(kRotThreads), smem, st, P)
                : launch_pdl(rotary_cache_write_kernel<__half, false>, grid, dim3(kRotThreads), smem, st, P);
    else
        e = rotary->interleaved
                ? launch_pdl(rotary_cache_write_kernel<__nv_bfloat16, true>, grid, dim3(kRotThreads), smem, st, P)
                : launch_pdl(rotary_cache_write_kernel<__nv_bfloat16, false>, grid, dim3(kRotThreads), smem, st, P);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
