// pa_q4.cuh -- the 4-bit cache: format, addresses, conversions.
//
// A token's head is cut into groups of 64 channels.  With T the 16-bit type of
// the keys and values, a group x_0 .. x_63 is held as
//     z = min x,  s = T((max x - z) / 15),  n_i = rint((x_i - z) / s) in 0 .. 15
// (n = 0 where s = 0) and read as s n_i + z.  z is one of the group's own values,
// so it is exact in T.  A group whose range is not finite has s = z = NaN, n = 0.
//
// A pool [num_blocks][num_kv_heads][block_size][36 head_dim / 64] bytes holds
// each (block, head) as tiles of 16 tokens, a tile as head_dim / 64 cells, one
// a group of channels.  A cell is 576 bytes:
//     32 bytes a token: channel c of the group in byte c / 2, low half first;
//         the two 16-byte halves change places in tokens 4-7 and 12-15
//     4 bytes a token: s, then z
// A cell's nibbles are then two 8 x 8 matrices of 16-bit units a half, which
// ldmatrix reads without bank conflicts as they lie (rows 0-3 and 4-7 of 32
// bytes fall on different halves of the banks), a token's group is one 32-byte
// sector, and a tile is one contiguous multiple of 64 bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"

namespace pa {

constexpr int kQ4Group = 64;       // channels of a group
constexpr int kQ4Tokens = 16;      // tokens of a tile
constexpr int kQ4CellBytes = 576;  // 16 x (32 + 4)
constexpr int kQ4CellParams = 512;

// log2 of a block size that a 4-bit pool can have (16 .. 256), or -1
inline int q4_block_shift(int b) {
    for (int sh = 4; sh <= 8; ++sh)
        if (b == (1 << sh)) return sh;
    return -1;
}

// Byte, in a cell, of the 4-byte word that holds channels 8 c .. 8 c + 7 of a
// token (both counted in the cell).
__host__ __device__ __forceinline__ int q4_word(int token, int c) {
    return token * 32 + ((((c >> 2) ^ (token >> 2)) & 1) << 4) + (c & 3) * 4;
}

// Two elements of a 16-bit type in one register, element 0 in the low half.
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
    // the lesser of each half; a NaN stays
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
        const __half2 h = __hmin2_nan(*reinterpret_cast<const __half2 *>(&a),
                                      *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static constexpr uint32_t kInf2 = 0x7c007c00u;
    static constexpr uint32_t kNan2 = 0x7fff7fffu;
};
template <>
struct Pack<__nv_bfloat16> {
    static __device__ __forceinline__ float2 up(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
        const __nv_bfloat162 h = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static constexpr uint32_t kInf2 = 0x7f807f80u;
    static constexpr uint32_t kNan2 = 0x7fff7fffu;
};

// (least, -greatest) of eight elements, packed: one comparison a step reduces both.
template <typename T>
__device__ __forceinline__ uint32_t q4_range8(const uint4 &v) {
    const uint32_t lo = Pack<T>::min2(Pack<T>::min2(v.x, v.y), Pack<T>::min2(v.z, v.w));
    const uint32_t hi = Pack<T>::min2(
        Pack<T>::min2(v.x ^ 0x80008000u, v.y ^ 0x80008000u),
        Pack<T>::min2(v.z ^ 0x80008000u, v.w ^ 0x80008000u));
    // halves of lo, and of hi, against each other
    return Pack<T>::min2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
}

// A group's scale and least value from its (least, -greatest).
struct Q4Scale {
    uint32_t params;  // s, z in T
    float s, z, inv;  // inv: 1 / s, or 0 (see q4_codes8)
};
template <typename T>
__device__ __forceinline__ Q4Scale q4_scale(uint32_t range) {
    const float2 r = Pack<T>::up(range);
    const float width = -r.y - r.x;
    Q4Scale q;
    if (width < INFINITY) {
        const uint32_t s16 = Pack<T>::down(__fdiv_rn(width, 15.0f), 0.0f);
        q.params = (s16 & 0xffffu) | (range << 16);
        q.s = Pack<T>::up(s16).x;
    } else {  // an infinity or a NaN among them, or a range past fp32
        q.params = Pack<T>::kNan2;
        q.s = 0.0f;
    }
    q.z = r.x;
    q.inv = q.s >= 0x1p-100f ? __frcp_rn(q.s) : 0.0f;
    return q;
}

// n of eight elements.  The quotient is rounded to fp32 once (a product with
// the reciprocal, corrected by its exact remainder), then to a whole number by
// adding 1.5 2^23, whose low bits then hold it; the words' constant parts are
// taken off together.  Scales whose reciprocal or remainders leave fp32's normal
// range (bf16 groups a hair wide) are divided by.
template <typename T>
__device__ __forceinline__ uint32_t q4_codes8(const uint4 &v, const Q4Scale &q) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t acc = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = Pack<T>::up(u[i / 2]);
        const float d = (i & 1 ? x.y : x.x) - q.z;
        float t = d * q.inv;
        t = fmaf(fmaf(-t, q.s, d), q.inv, t);
        if (q.inv == 0.0f) t = __fdiv_rn(d, q.s);
        acc += __float_as_uint(fminf(t, 15.0f) + 12582912.0f) << (4 * i);
    }
    return q.s > 0.0f ? acc - 0x4b400000u * 0x11111111u : 0u;
}

// Eight elements from their word, as T.
template <typename T>
__device__ __forceinline__ uint4 q4_values8(uint32_t w, float s, float z) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(0x4b000000u | ((w >> (8 * i)) & 15u)) - 8388608.0f;
        const float b = __uint_as_float(0x4b000000u | ((w >> (8 * i + 4)) & 15u)) - 8388608.0f;
        o[i] = Pack<T>::down(fmaf(a, s, z), fmaf(b, s, z));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace pa
