// pa_rotary.cuh -- the kernel that turns query and key by their positions and
// writes key and value into the paged cache, in 16 bits (pa_rotary.cu) or in 4
// (pa_q4_write.cu), and its host side.
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
// four rows (two with 4-bit pools), unless that leaves fewer than two CTAs an SM: with few rows a
// token (grouped queries) one row a thread is one round trip to memory a CTA
// and half the rate (4099 tokens of 12 + 2 + 2 heads of 128: 12.4 us with four
// rows, 3.4 more with one).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_ptx.cuh"
#include "pa_q4.cuh"

namespace pa {
namespace {


constexpr int kRotThreads = 256;
// Rows a thread has in flight.  Quantising takes registers and instructions: two rows
// and four CTAs an SM there (16384 tokens of 40 heads of 128: 176 us; four rows and
// three CTAs 195, one row and six 180; it takes 165 since a group's range comes from its
// own lanes).
template <bool Q4>
constexpr int kRotBatch = Q4 ? 2 : 4;
template <bool Q4>
constexpr int kRotCtas = Q4 ? 4 : 0;  // 0: not stated

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

// A row's two chunks of every thread, quantised, to token `token` of tile `tile`
// of a 4-bit pool.  Called by the D / 16 lanes of a row together (j: the lane's
// place among them).  How the chunks lie decides which lanes have a group:
//   IL: neighbouring chunks (interleaved pairs, or no rotation): four lanes;
//   halves of the whole head: eight lanes have a group of the one half and a group
//       of the other (D = 64: four lanes, both chunks);
//   halves of a part of it: spread unevenly, so every group is reduced over all lanes.
template <typename T, bool IL, int D>
__device__ __forceinline__ void store_q4(uint8_t *pool, size_t tile, int token, int j, int ca,
                                         int cb, bool whole, const uint4 &a, const uint4 &b) {
    constexpr int kLanes = D / 16, kCells = D / kQ4Group;
    const unsigned row = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(unsigned)(kLanes - 1));
    uint32_t ra = q4_range8<T>(a), rb = q4_range8<T>(b);
    uint8_t *cells = pool + tile * (size_t)(kCells * kQ4CellBytes);
    uint8_t *cell_a = cells + (ca >> 3) * kQ4CellBytes, *cell_b = cells + (cb >> 3) * kQ4CellBytes;
    auto reduce = [&](uint32_t x, int lanes) {
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1)
            if (o < lanes) x = Pack<T>::min2(x, __shfl_xor_sync(row, x, o));
        return x;
    };
    if (IL || kCells == 1) {
        const Q4Scale q = q4_scale<T>(reduce(Pack<T>::min2(ra, rb), 4));
        *reinterpret_cast<uint32_t *>(cell_a + q4_word(token, ca & 7)) = q4_codes8<T>(a, q);
        *reinterpret_cast<uint32_t *>(cell_b + q4_word(token, cb & 7)) = q4_codes8<T>(b, q);
        if ((j & 3) == 0)
            *reinterpret_cast<uint32_t *>(cell_a + kQ4CellParams + 4 * token) = q.params;
        return;
    }
    bool first_a, first_b;  // the lane writes its chunks' scales
    if (whole) {
        ra = reduce(ra, 8);
        rb = reduce(rb, 8);
        first_a = first_b = (j & 7) == 0;
    } else {
        uint32_t of_a = 0, of_b = 0;
        first_a = first_b = false;
#pragma unroll
        for (int g = 0; g < kCells; ++g) {
            const bool in_a = ca >> 3 == g, in_b = cb >> 3 == g;
            const uint32_t x = reduce(Pack<T>::min2(in_a ? ra : Pack<T>::kInf2, in_b ? rb : Pack<T>::kInf2), kLanes);
            if (in_a) of_a = x;
            if (in_b) of_b = x;
            // (the lane that has the group's first chunk)
            first_a |= ca == 8 * g;
            first_b |= cb == 8 * g;
        }
        ra = of_a;
        rb = of_b;
    }
    const Q4Scale qa = q4_scale<T>(ra);
    *reinterpret_cast<uint32_t *>(cell_a + q4_word(token, ca & 7)) = q4_codes8<T>(a, qa);
    if (first_a) *reinterpret_cast<uint32_t *>(cell_a + kQ4CellParams + 4 * token) = qa.params;
    const Q4Scale qb = q4_scale<T>(rb);
    *reinterpret_cast<uint32_t *>(cell_b + q4_word(token, cb & 7)) = q4_codes8<T>(b, qb);
    if (first_b) *reinterpret_cast<uint32_t *>(cell_b + kQ4CellParams + 4 * token) = qb.params;
}

// A CTA takes `rounds` times 256 / (threads a row * rows at once) tokens; thread
// = (token, row, unit j of the row).  A token's rows are its query heads, its
// key heads and its value heads; a thread goes through its rows of all its
// tokens as one list, four at a time (4-bit pools: two).  QD: 0 for 16-bit pools, else
// 4-bit pools of that head_dim.
template <typename T, bool IL, int QD>
__global__ void __launch_bounds__(kRotThreads, kRotCtas<(QD > 0)>)
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
    constexpr int kBatch = kRotBatch<(QD > 0)>;
    uint4 a[kBatch], b[kBatch];
    int64_t slot[kBatch];
    auto load = [&](At p) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u, next(p)) {
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
        for (int u = 0; u < kBatch; ++u, next(p)) {
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
                // the slot's row of its head in the pool
                const size_t at_row =
                    ((((size_t)(slot[u] >> P.block_shift) * Hkv) + h) << P.block_shift) +
                    (size_t)(slot[u] & ((1 << P.block_shift) - 1));
                if constexpr (QD > 0) {
                    store_q4<T, IL, QD>(reinterpret_cast<uint8_t *>(r < H + Hkv ? P.k_cache : P.v_cache),
                                        at_row / kQ4Tokens, (int)(at_row % kQ4Tokens), j, ca, cb,
                                        rot_units == lpr, a[u], b[u]);
                    continue;
                }
                dst = (r < H + Hkv ? P.k_cache : P.v_cache) + (at_row << lg_cpr);
            }
            dst[ca] = a[u];
            dst[cb] = b[u];
        }
        at = p;
        load(at);
    }
}


inline int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

// Checks and launch of the write, for 16-bit pools and (Q4) 4-bit ones.  Q4 without
// `rotary`: key and value alone, no query.
template <bool Q4>
inline pa_status_t rotary_write(void *query_out, int64_t query_out_stride, const void *query,
                                int64_t query_stride, const void *key, int64_t key_stride,
                                const void *value, int64_t value_stride, const int64_t *positions,
                                const pa_rotary_t *rotary, void *k_cache, void *v_cache,
                                const int64_t *slot_mapping, int num_tokens, int num_blocks,
                                int block_size, int num_heads, int num_kv_heads, int head_dim,
                                pa_dtype_t dtype, unsigned int *dev_error_word,
                                pa_stream_t stream) {
    const bool plain = Q4 && !rotary;
    if (num_tokens < 0 || num_blocks <= 0 || num_heads < (plain ? 0 : 1) || num_kv_heads <= 0 ||
        (!rotary && !plain))
        return PA_ERR_INVALID_ARG;
    const int shift = Q4 ? q4_block_shift(block_size) : pool_block_shift(block_size);
    if (shift < 0) return PA_ERR_UNSUPPORTED;
    if (!is_16bit(dtype)) return PA_ERR_INVALID_ARG;
    if (!head_dim_supported(head_dim)) return PA_ERR_UNSUPPORTED;
    if (!plain) {
        if (rotary->rotary_dim <= 0 || rotary->rotary_dim % 16 != 0 ||
            rotary->rotary_dim > head_dim || rotary->num_axes < 1 ||
            rotary->num_axes > PA_MAX_ROTARY_AXES)
            return PA_ERR_INVALID_ARG;
        for (int i = 0; i < rotary->rotary_dim / 2; ++i)
            if (rotary->axis[i] >= rotary->num_axes) return PA_ERR_INVALID_ARG;
    }
    if ((long long)num_heads + 2ll * num_kv_heads > (1 << 20)) return PA_ERR_UNSUPPORTED;
    const long long q_row = (long long)num_heads * head_dim;
    const long long kv_row = (long long)num_kv_heads * head_dim;
    if (query_stride < q_row || query_out_stride < q_row || key_stride < kv_row ||
        value_stride < kv_row || query_stride % 8 || query_out_stride % 8 || key_stride % 8 ||
        value_stride % 8)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!plain && (!query_out || !query || !positions)) return PA_ERR_INVALID_ARG;
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
    if (plain) std::memset(&P.rot, 0, sizeof(P.rot));
    else P.rot = *rotary;
    // tokens a CTA: enough for kRotBatch rows a thread, while two CTAs an SM are left
    const int lanes = kRotThreads >> (P.lg_lpr + P.lg_rows);
    const int groups = (rows + (1 << P.lg_rows) - 1) >> P.lg_rows;  // rows a thread and token
    const int sms = device_sms();
    if (sms <= 0) return PA_ERR_CUDA;
    P.rounds = 1;
    while (P.rounds * groups < kRotBatch<Q4> &&
           (long long)num_tokens >= 2ll * sms * lanes * (2 * P.rounds))
        P.rounds *= 2;
    const int tokens = lanes * P.rounds;
    const dim3 grid((unsigned)((num_tokens + tokens - 1) / tokens));
    // at most 256 / 4 units of 8 pairs at once (a token has three rows at
    // least), four rounds: 16 KB
    const size_t smem = (size_t)tokens * (P.rot.rotary_dim / 2) * sizeof(float2);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaErrorInvalidValue;
    auto go = [&](auto kern) { e = launch_pdl(kern, grid, dim3(kRotThreads), smem, st, P); };
    const bool neighbours = P.rot.interleaved || plain;
    auto dim = [&](auto d) {
        constexpr int QD = decltype(d)::value;
        if (dtype == PA_F16) {
            if (neighbours) go(rotary_cache_write_kernel<__half, true, QD>);
            else go(rotary_cache_write_kernel<__half, false, QD>);
        } else {
            if (neighbours) go(rotary_cache_write_kernel<__nv_bfloat16, true, QD>);
            else go(rotary_cache_write_kernel<__nv_bfloat16, false, QD>);
        }
    };
    if constexpr (!Q4) {
        dim(std::integral_constant<int, 0>());
    } else {
        if (head_dim == 64) dim(std::integral_constant<int, 64>());
        else if (head_dim == 128) dim(std::integral_constant<int, 128>());
        else dim(std::integral_constant<int, 256>());
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa
