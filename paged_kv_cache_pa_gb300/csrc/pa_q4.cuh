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
    // the same with the largest finite number past it (a NaN stays)
    static __device__ __forceinline__ uint32_t down_finite(float a, float b) {
        uint32_t d;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
        return d;
    }
    // the lesser of each half; a NaN stays
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
        const __half2 h = __hmin2_nan(*reinterpret_cast<const __half2 *>(&a),
                                      *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        const __half2 h = __hmax2_nan(*reinterpret_cast<const __half2 *>(&a),
                                      *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static constexpr float kLeastScale = 0x1p-14f;  // the least that is not subnormal
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
    // the same with the largest finite number past it (a NaN stays)
    static __device__ __forceinline__ uint32_t down_finite(float a, float b) {
        uint32_t d;
        asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
        return d;
    }
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
        const __nv_bfloat162 h = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        const __nv_bfloat162 h = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static constexpr float kLeastScale = 0x1p-100f;
    static constexpr uint32_t kInf2 = 0x7f807f80u;
    static constexpr uint32_t kNan2 = 0x7fff7fffu;
};

// (least, -greatest) of eight elements, packed: one comparison a step reduces both.
template <typename T>
__device__ __forceinline__ uint32_t q4_range8(const uint4 &v) {
    const uint32_t lo = Pack<T>::min2(Pack<T>::min2(v.x, v.y), Pack<T>::min2(v.z, v.w));
    const uint32_t hi = Pack<T>::max2(Pack<T>::max2(v.x, v.y), Pack<T>::max2(v.z, v.w));
    // halves of lo, and of -hi, against each other
    return Pack<T>::min2(__byte_perm(lo, hi, 0x5410) ^ 0x80000000u,
                         __byte_perm(lo, hi, 0x7632) ^ 0x80000000u);
}

// Out of line: few groups are this narrow.
static __device__ __noinline__ float q4_fifteenth(float width) { return __fdiv_rn(width, 15.0f); }

// Reciprocal to one step (MUFU).
__device__ __forceinline__ float q4_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A group's scale and least value from its (least, -greatest).
struct Q4Scale {
    uint32_t params;  // s, z in T
    float s, z, inv;  // inv: 1 / s to 2^-22, or 0 (see q4_codes8)
};
template <typename T>
__device__ __forceinline__ Q4Scale q4_scale(uint32_t range) {
    const float2 r = Pack<T>::up(range);
    const float width = -r.y - r.x;
    Q4Scale q;
    // width / 15, rounded once: a product with the reciprocal and its exact
    // remainder's (right for every fp32 width above 2^-100; the type's rounding takes
    // what is below)
    float f = width * (1.0f / 15.0f);
    f = fmaf(fmaf(-15.0f, f, width), 1.0f / 15.0f, f);
    if (width < 0x1p-100f) f = q4_fifteenth(width);
    const uint32_t s16 = Pack<T>::down(f, 0.0f);
    q.z = r.x;
    q.s = Pack<T>::up(s16).x;
    q.params = (s16 & 0xffffu) | (range << 16);
    if (!(width < INFINITY)) {  // an infinity or a NaN among them, or a range past fp32
        q.params = Pack<T>::kNan2;
        q.s = 0.0f;
    }
    q.inv = q.s >= Pack<T>::kLeastScale ? q4_rcp(q.s) : 0.0f;
    return q;
}

// The same by division, for scales that are subnormal in T (then 15 s may be
// well below the range) or whose reciprocal or remainders leave fp32's normal range.
template <typename T>
__device__ __noinline__ uint32_t q4_codes8_small(uint4 v, float s, float z) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t w = 0;
    if (!(s > 0.0f)) return 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = Pack<T>::up(u[i / 2]);
        const float t = __fdiv_rn((i & 1 ? x.y : x.x) - z, s);
        w |= (uint32_t)__float2int_rn(fminf(t, 15.0f)) << (4 * i);
    }
    return w;
}

// n of eight elements.  The quotient is a product with the reciprocal, corrected by
// its exact remainder, which leaves ties where they are; adding 1.5 2^23 rounds it to
// a whole number, in the low bits; the words' constant parts are taken off
// together.  (s is at least range / 15 less half a step of T, so n stays below 15.5.)
template <typename T>
__device__ __forceinline__ uint32_t q4_codes8(const uint4 &v, const Q4Scale &q) {
    if (q.inv == 0.0f) return q4_codes8_small<T>(v, q.s, q.z);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    const float2 nz = make_float2(-q.z, -q.z), ns = make_float2(-q.s, -q.s);
    const float2 inv = make_float2(q.inv, q.inv), whole = make_float2(12582912.0f, 12582912.0f);
    uint32_t acc = 0u - 0x4b400000u * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // two at once
        const float2 d = __fadd2_rn(Pack<T>::up(u[i]), nz);
        float2 t = __fmul2_rn(d, inv);
        t = __ffma2_rn(__ffma2_rn(t, ns, d), inv, t);
        t = __fadd2_rn(t, whole);
        acc += (__float_as_uint(t.x) << (8 * i)) + (__float_as_uint(t.y) << (8 * i + 4));
    }
    return acc;
}

// Eight elements from their word, as T.  A group's top may be past the type's largest number,
// its scale having been rounded up (by 2^-12 and 15 s + z: 65520 for 0 .. 65504 in fp16): that
// reads as the largest, where it would round to an infinity.  A NaN stays.
template <typename T>
__device__ __forceinline__ uint4 q4_values8(uint32_t w, float s, float z) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(0x4b000000u | ((w >> (8 * i)) & 15u)) - 8388608.0f;
        const float b = __uint_as_float(0x4b000000u | ((w >> (8 * i + 4)) & 15u)) - 8388608.0f;
        o[i] = Pack<T>::down_finite(fmaf(a, s, z), fmaf(b, s, z));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace pa
