// pa_q4_decode.cuh -- attention of a sequence's newest tokens over a cache held in
// 4 bits (pa_decode_attention_q4), one instantiation per (T, head_dim, rows).
//
// The mathematics.  A cached key is s n + z per group of 64 channels, so with n
// whole numbers of 4 bits
//     <q, k> = sum_groups s <q_group, n_group> + z sum q_group,
// and with weights p_j = 2^(x_j - m)
//     sum_j p_j v_j = sum_j (p_j s_j) n_j + sum_j p_j z_j   (per group).
// The two sums over channels and tokens are matrix products with a factor of
// whole numbers below 16; scales and least values touch one number a token and
// group.
//
// Operands without conversion.  Read as fp16, the bits 0x000n are n 2^-24 (a
// subnormal, which the tensor cores multiply exactly) and 0x00n0 are 16 n 2^-24.
// Two nibbles of a 32-bit word become a pair of fp16 factors by one AND, eight by
// a shift and four: no subtraction, no conversion.  The other factor takes up
// the powers of two: odd nibbles' queries are divided by 16 ahead, odd channels
// of the output at the end.  It works in fp16 only (bf16 has no such
// subnormals), so a bf16 query goes to fp16, each row scaled by the power of two
// that brings its largest element to 2^13: exact, but for elements 2^-28 of the
// largest, where fp16 itself ends.
//
// The weights p s go to fp16 in two parts (their rounding, and its remainder), so
// their error is 2^-22 of them; a running power of two keeps them in range
// (below).  With at most four rows the two parts are two columns of one product,
// which has eight, at no cost.
//
// Softmax in one pass.  Each warp keeps a maximum m per row which it moves only
// when a weight has outgrown 2^8 (the first chunk, then rarely): the check is
// one comparison and a vote instead of three exchanges between the lanes, and
// any m gives the same quotient.
//
// Work.  A warp works on its own, without barriers: it has a range of chunks (16
// tokens of a sequence's KV head) of the batch's, all laid end to end and cut
// into equal parts, and a ring of kStages chunks that it fills itself by
// asynchronous copies.  A (sequence, head, rows) that is cut leaves partial
// results, which the merge kernel puts together.
//
// Bound: HBM, 72 bytes a group and token of K and V.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_launch.cuh"
#include "pa_ptx.cuh"
#include "pa_q4.cuh"

namespace pa {

constexpr int kQ4Warps = 4;  // of a CTA
constexpr int kQ4Threads = 32 * kQ4Warps;
constexpr int kQ4Sms = 152;  // that the workers are sized for (right for any number)
constexpr float kQ4NoMax = -1e30f;   // m before any token: below every logit that counts
// A weight (2^6 where the maximum was last taken) and a scale (below 2^5 then) beyond
// which both are taken anew: their product stays below fp16's 2^16.
constexpr float kQ4TopP = 1024.f, kQ4TopS = 32.f;

struct Q4DecodeParams {
    void *out;
    const void *query;
    const uint8_t *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens, *query_start_loc;  // the last: or null
    float *part;    // [workers][2][rows][head_dim]
    float2 *part_ml;  // [workers][2][rows]: m, l
    int4 *tails;    // [workers]: what the worker's last unit leaves to be merged
    unsigned int *err;
    int out_f32;
    int max_blocks_per_seq, max_context_len, max_query_len, num_seqs, num_tokens;
    int num_heads, num_kv_heads, G, num_blocks;
    int sub_shift;      // log2 of a block's tiles
    int whole;          // no unit is cut
    int workers;
    float scale_log2;
};

// A sequence's share of the work.
struct Q4Seq {
    int q0, n;      // its query tokens
    int len;        // of its context
    int chunks, tiles;  // 16-token chunks; tiles of query rows (0 work: chunks = 0)
    bool bad;       // breaks the rules
};

template <int RT>
__device__ __forceinline__ Q4Seq q4_seq(const Q4DecodeParams &P, int s) {
    Q4Seq r;
    r.len = P.context_lens[s];
    if (P.query_start_loc) {
        r.q0 = P.query_start_loc[s];
        r.n = P.query_start_loc[s + 1] - r.q0;
        r.bad = r.q0 < 0 || r.n < 0 || r.q0 > P.num_tokens || r.n > P.num_tokens - r.q0 ||
                r.n > P.max_query_len;
    } else {
        r.q0 = s;
        r.n = 1;
        r.bad = false;
    }
    r.bad |= r.len < 0 || r.len > P.max_context_len || (r.len > 0 && r.n > r.len);
    const bool work = !r.bad && r.n > 0;
    r.chunks = work ? (r.len + kQ4Tokens - 1) / kQ4Tokens : 0;
    r.tiles = work ? (r.n * P.G + RT - 1) / RT : 0;
    return r;
}

__device__ __forceinline__ void q4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit units, spread as ldmatrix gives it, transposed.
__device__ __forceinline__ uint32_t q4_transpose(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t q4_fma2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b),
                              *reinterpret_cast<const __half2 *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ void q4_copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void q4_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void q4_copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int RT>
struct Q4Shape {
    static constexpr int kCells = D / kQ4Group;
    static constexpr int kTileBytes = kCells * kQ4CellBytes;
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = D == 64 ? 6 : 4;
    static constexpr int kTiles8 = RT <= 8 ? 1 : RT / 8;  // groups of eight columns
    static constexpr bool kDouble = RT == 4;  // columns 4-7: the weights' remainders
    static constexpr int kCtas = D <= 128 && RT <= 8 ? 4 : 3;  // an SM
    static constexpr int kWorkers = kQ4Sms * kCtas * kQ4Warps;
    static constexpr size_t kSmem = (size_t)kQ4Warps * kStages * kStageBytes;
};

// Where a warp is in the batch's chunks: sequence, KV head, tile of its query rows,
// chunk, from the slowest to the fastest (a head's tiles read the same chunks: the
// later ones find them in L2).
struct Q4Cursor {
    int s, head, tile, chunk;
    Q4Seq q;
};

// The next sequence with work; past the last one s = num_seqs.
template <int RT>
__device__ __forceinline__ void q4_next_seq(const Q4DecodeParams &P, Q4Cursor &c) {
    c.head = c.tile = c.chunk = 0;
    while (++c.s < P.num_seqs) {
        c.q = q4_seq<RT>(P, c.s);
        if (c.q.chunks) break;
    }
}

// The next (sequence, head, tile); true where that is another sequence's.
template <int RT>
__device__ __forceinline__ bool q4_next_unit(const Q4DecodeParams &P, Q4Cursor &c) {
    c.chunk = 0;
    if (++c.tile < c.q.tiles) return false;
    c.tile = 0;
    if (++c.head < P.num_kv_heads) return false;
    q4_next_seq<RT>(P, c);
    return true;
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kQ4Threads, (Q4Shape<D, RT>::kCtas))
    q4_decode_kernel(const __grid_constant__ Q4DecodeParams P) {
    using S = Q4Shape<D, RT>;
    constexpr int NT = S::kTiles8, C = S::kCells;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ long long s_base[kQ4Threads];  // chunks of the batch before a thread's sequences
    __shared__ long long s_warp[kQ4Warps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    pdl_wait();  // earlier kernels on the stream may still write what this reads

    // The batch's chunks, laid end to end: thread i's sequences are i * each ..
    const int each = (P.num_seqs + kQ4Threads - 1) / kQ4Threads;
    long long mine = 0;
    for (int s = tid * each; s < min(P.num_seqs, (tid + 1) * each); ++s) {
        const Q4Seq q = q4_seq<RT>(P, s);
        mine += (long long)q.chunks * q.tiles * P.num_kv_heads;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kQ4Warps; ++i) {
        if (i == warp) before = total;
        total += s_warp[i];
    }
    s_base[tid] = before + incl - mine;
    __syncthreads();

    const int worker = blockIdx.x * kQ4Warps + warp;
    const long long per = max((total + P.workers - 1) / P.workers, 1ll);
    const long long start = min(worker * per, total), end = min(start + per, total);
    int4 tail = make_int4(-1, 0, 0, 0);

    if (start < end) {
        // the sequence that holds `start`
        int lo = 0;
#pragma unroll
        for (int i = 0; i < kQ4Threads; i += 32)
            lo += __popc(__ballot_sync(0xffffffffu, s_base[i + lane] <= start));
        lo -= 1;  // the last thread whose sequences begin at or before it; where they are
                  // empty, those behind them have it
        long long off = start - s_base[lo];
        Q4Cursor at;  // the next chunk to ask for
        at.s = lo * each - 1;
        for (;;) {
            q4_next_seq<RT>(P, at);
            if (at.s >= P.num_seqs) break;
            const long long n = (long long)at.q.chunks * at.q.tiles * P.num_kv_heads;
            if (off < n) break;
            off -= n;
        }
        const int count = (int)(end - start);  // chunks of the range
        int pos = 0;                           // of `at` in it
        if (at.s < P.num_seqs) {
            const int unit = (int)off / at.q.chunks;
            at.chunk = (int)off - unit * at.q.chunks;
            at.head = unit / at.q.tiles;
            at.tile = unit - at.head * at.q.tiles;
            if (P.whole && at.chunk > 0) {  // that unit is the worker's in whose range it begins
                pos = at.q.chunks - at.chunk;
                q4_next_unit<RT>(P, at);
            }
        }
        Q4Cursor cu = at;  // the chunk at hand
        uint8_t *ring = s_ring + (size_t)warp * S::kStages * S::kStageBytes;
        const uint32_t ring_u32 = smem_u32(ring);

        // ---- asking for chunks ----
        // A stage is the K tile and the V tile, 16 bytes a lane and step; one step has the end
        // of the one and the beginning of the other.
        constexpr int kPieces = S::kTileBytes / 16, kMixed = kPieces / 32 * 32;
        const uint8_t *k_lane = P.k_cache + lane * 16;
        const uint8_t *v_lane = P.v_cache + lane * 16 - S::kTileBytes;
        const uint8_t *m_lane = kMixed + lane < kPieces ? k_lane : v_lane;
        const uint32_t dst_lane = ring_u32 + lane * 16;
        const uint32_t block_bytes = (uint32_t)(P.num_kv_heads << P.sub_shift) * S::kTileBytes;
        const int sub_mask = (1 << P.sub_shift) - 1;
        int asked = 0, used = 0;
        uint32_t bad = 0;       // bit i & 31: the i-th chunk's block is outside the pool
        int ids = 0;            // the lane's block id, of chunk (at.chunk & ~31) + lane
        bool load_ids = true;
        uint32_t head_off = (uint32_t)(at.head << P.sub_shift) * S::kTileBytes;
        auto ask = [&](uint32_t slot) {
            if (at.s < P.num_seqs && (pos < count || (P.whole && at.chunk > 0))) {
                if (load_ids) {
                    const int c = (at.chunk & ~31) + lane;
                    ids = c < at.q.chunks ? P.block_tables[(size_t)at.s * P.max_blocks_per_seq +
                                                           (c >> P.sub_shift)]
                                          : 0;
                    load_ids = false;
                }
                const int id = __shfl_sync(0xffffffffu, ids, at.chunk & 31);
                if ((unsigned)id < (unsigned)P.num_blocks) {
                    const size_t o = (size_t)(uint32_t)id * block_bytes +
                                     (head_off + (uint32_t)(at.chunk & sub_mask) * S::kTileBytes);
#pragma unroll
                    for (int i = 0; i < 2 * kPieces; i += 32) {
                        const uint8_t *src = i < kMixed ? k_lane : i == kMixed ? m_lane : v_lane;
                        if (i + 32 <= 2 * kPieces || i + lane < 2 * kPieces)
                            q4_copy16(dst_lane + slot + i * 16, src + o + i * 16);
                    }
                } else {
                    bad |= 1u << (asked & 31);
                    if (lane == 0 && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
                }
                ++pos;
                ++asked;
                if (++at.chunk == at.q.chunks) {
                    // (a table of at most 32 chunks is all in the lanes, for every head)
                    load_ids = at.q.chunks > 32;
                    if (q4_next_unit<RT>(P, at)) load_ids = true;
                    head_off = (uint32_t)(at.head << P.sub_shift) * S::kTileBytes;
                } else if ((at.chunk & 31) == 0) {
                    load_ids = true;
                }
            }
            q4_copy_commit();
        };
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) ask(i * S::kStageBytes);

        // ---- the unit at hand ----
        float O[NT][C][4][4];           // [rows of 16 channels: cell, nibble j][fragment]
        float m[NT][2], l[NT][2], za[NT][C][2];  // columns 2t, 2t + 1
        uint32_t qf[NT][C][2][2][2];    // the query's fragments: cell, half, nibble pair
        float c1[NT][2], qz[NT][C][2];
        int lim[NT][2], lim_min = 0;    // tokens a column sees; the fewest of any
        float vs = 0.f;                 // power of two on the weights times scales
        int first_chunk = 0, rows = 0, row0 = 0;
        bool fresh = true;              // the chunk at hand begins a unit, or the range

        auto begin_unit = [&]() {
            first_chunk = cu.chunk;
            row0 = cu.tile * RT;
            rows = min(RT, cu.q.n * P.G - row0);
            lim_min = cu.q.len - cu.q.n + 1 + row0 / P.G;
            vs = 0x1p60f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int col = S::kDouble ? (g & 3) : nt * 8 + g;
                const int r = row0 + col;
                float f[C][2][8];
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (col < rows) {
                            const size_t row = (size_t)(cu.q.q0 + r / P.G) * P.num_heads +
                                               (size_t)cu.head * P.G + r % P.G;
                            w = *reinterpret_cast<const uint4 *>(
                                static_cast<const T *>(P.query) + row * D + c * 64 + h * 32 + 8 * t);
                        }
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x = Pack<T>::up(u[i]);
                            f[c][h][2 * i] = x.x;
                            f[c][h][2 * i + 1] = x.y;
                            top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                        }
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int eb = (__float_as_int(top) >> 23) & 255;
                // 2^13 over the largest element's power of two; as it is for a row of
                // zeros or with an infinity
                const int nb = eb == 0 || eb == 255 ? 127 : max(1, min(250, 267 - eb));
                const float norm = __int_as_float(nb << 23);
                const float back = __int_as_float((254 - nb) << 23) * (0x1p24f * P.scale_log2);
                float sum[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    sum[c] = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum[c] += f[c][h][i];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float *x = f[c][h] + 2 * i;
                            qf[nt][c][h][i][0] = Pack<__half>::down(x[0] * norm, x[4] * norm);
                            qf[nt][c][h][i][1] =
                                Pack<__half>::down(x[1] * norm * 0.0625f, x[5] * norm * 0.0625f);
                        }
                    }
                    sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 1);
                    sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 2);
                    sum[c] *= P.scale_log2;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // column 2t + e of this group: its row is that of lanes 4 (2t + e) ..
                    const int src = 4 * (2 * t + e);
                    c1[nt][e] = __shfl_sync(0xffffffffu, back, src);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        qz[nt][c][e] = __shfl_sync(0xffffffffu, sum[c], src);
                        za[nt][c][e] = 0.f;
                    }
                    const int cc = S::kDouble ? ((2 * t + e) & 3) : nt * 8 + 2 * t + e;
                    lim[nt][e] = cu.q.len - cu.q.n + 1 + (row0 + cc) / P.G;
                    m[nt][e] = kQ4NoMax;
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) O[nt][c][j][i] = 0.f;
            }
        };

        // What the unit's chunks so far give, to the output or, where it is cut, to
        // the workspace: slot 0 of a worker is its first unit's if that began
        // before, slot 1 its last one's.
        auto end_unit = [&]() {
            const bool all = first_chunk == 0 && cu.chunk + 1 == cu.q.chunks;
            const int slot = 2 * worker + (first_chunk == 0 ? 1 : 0);
            if (!all && first_chunk == 0) {
                const int rest = cu.q.chunks - cu.chunk - 1;
                tail = make_int4(cu.s, cu.head, cu.tile, (int)((rest + per - 1) / per));
            }
            const float unscale = 0x1p24f / vs;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float ls = l[nt][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
                    const int col = nt * 8 + 2 * t + e;
                    const bool in = col < rows && (!S::kDouble || col < 4);
                    const int r = row0 + col;
                    const size_t out_row = (size_t)(cu.q.q0 + r / P.G) * P.num_heads +
                                           (size_t)cu.head * P.G + r % P.G;
                    const float inv = !all ? 1.f : ls == 0.f ? 0.f : 1.f / ls;
                    if (!all && in && g == 0)
                        P.part_ml[(size_t)slot * RT + col] = make_float2(m[nt][e], ls);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float z = za[nt][c][e];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float x = O[nt][c][j][2 * h + e];
                                if (S::kDouble) x += __shfl_xor_sync(0xffffffffu, x, 2);
                                v[j] = fmaf(x, j & 1 ? unscale * 0.0625f : unscale, z) * inv;
                            }
                            const int d0 = c * 64 + h * 32 + 4 * g;
                            if (!in) continue;
                            if (!all) {
                                *reinterpret_cast<float4 *>(P.part + ((size_t)slot * RT + col) * D + d0) =
                                    make_float4(v[0], v[1], v[2], v[3]);
                            } else if (P.out_f32) {
                                *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + out_row * D + d0) =
                                    make_float4(v[0], v[1], v[2], v[3]);
                            } else {
                                *reinterpret_cast<uint2 *>(static_cast<T *>(P.out) + out_row * D + d0) =
                                    make_uint2(Pack<T>::down(v[0], v[1]), Pack<T>::down(v[2], v[3]));
                            }
                        }
                    }
                }
        };

        // lane's row of the 8 x 8 matrices that ldmatrix takes from a cell
        const int lm_token = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t lm_off = q4_word(lm_token, (lane >> 4) * 4);

        auto chunk_step = [&](uint32_t slot) {
            const uint32_t kb = ring_u32 + slot, vb = kb + S::kTileBytes;
            const uint8_t *kp = ring + slot, *vp = kp + S::kTileBytes;
            // x = scale <q, k> in units of log2: rows g, g + 8 (tokens) of columns 2t, 2t + 1
            float x[NT][4];
            {
                float acc[NT][C][4];
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[nt][c][i] = 0.f;
                    uint32_t r[4];
                    ldsm_x4(r[0], r[1], r[2], r[3], kb + c * kQ4CellBytes + lm_off);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t lo = r[2 * h] >> (8 * i), hi = r[2 * h + 1] >> (8 * i);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                q4_mma(acc[nt][c], lo & 0x000f000fu, hi & 0x000f000fu,
                                       lo & 0x00f000f0u, hi & 0x00f000f0u, qf[nt][c][h][i][0],
                                       qf[nt][c][h][i][1]);
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[nt][i] = 0.f;
                float y[NT][4];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint8_t *pp = kp + c * kQ4CellBytes + kQ4CellParams;
                    const float2 p0 = Pack<T>::up(*reinterpret_cast<const uint32_t *>(pp + 4 * g));
                    const float2 p1 = Pack<T>::up(*reinterpret_cast<const uint32_t *>(pp + 4 * g + 32));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 p = i < 2 ? p0 : p1;
                            y[nt][i] = c == 0 ? p.x * acc[nt][c][i] : fmaf(p.x, acc[nt][c][i], y[nt][i]);
                            x[nt][i] = fmaf(p.y, qz[nt][c][i & 1], x[nt][i]);
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[nt][i] = fmaf(y[nt][i], c1[nt][i & 1], x[nt][i]);
            }
            // the values' scales and least values
            float sv[C][2], zv[C][2];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint8_t *pp = vp + c * kQ4CellBytes + kQ4CellParams;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 p = Pack<T>::up(*reinterpret_cast<const uint32_t *>(pp + 4 * g + 32 * i));
                    sv[c][i] = p.x;
                    zv[c][i] = p.y;
                }
            }
            const bool skip = (bad >> (used & 31)) & 1u;
            if (skip || (cu.chunk + 1) * kQ4Tokens > lim_min) {
                // past the context, past a column's own token, or a block that was skipped:
                // whatever lies there must not meet a weight, not even one of zero
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int p = skip ? 0x7fffffff : cu.chunk * kQ4Tokens + g + 8 * i;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (p >= lim[nt][e]) x[nt][2 * i + e] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const bool nan = !(sv[c][i] + zv[c][i] == sv[c][i] + zv[c][i]);
                        if (p < cu.q.len && nan)  // of the columns that see it alone
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (p < lim[nt][e]) za[nt][c][e] = NAN;
                        if (p >= cu.q.len || nan) sv[c][i] = zv[c][i] = 0.f;
                    }
                }
                bad &= ~(1u << (used & 31));
            }
            float p[NT][4], top;
            auto weights = [&]() {
                top = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[nt][i] = ex2(x[nt][i] - m[nt][i & 1]);
                        top = fmaxf(top, p[nt][i]);
                    }
            };
            weights();
            float s_top = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) s_top = fmaxf(s_top, fmaxf(sv[c][0], sv[c][1]));
            if (__any_sync(0xffffffffu, fmaxf(top, s_top * vs * (kQ4TopP / kQ4TopS)) > kQ4TopP)) {
                // new maxima, and a new power of two on the scales
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float a = fmaxf(x[nt][e], x[nt][2 + e]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                        a = fmaxf(a - 6.f, m[nt][e]);
                        const float f = ex2(m[nt][e] - a);
                        m[nt][e] = a;
                        l[nt][e] *= f;
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            za[nt][c][e] *= f;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                O[nt][c][j][e] *= f;
                                O[nt][c][j][2 + e] *= f;
                            }
                        }
                    }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    s_top = fmaxf(s_top, __shfl_xor_sync(0xffffffffu, s_top, o));
                const int sb = (__float_as_int(s_top) >> 23) & 255;
                const float nv = fminf(vs, __int_as_float(max(1, min(187, 258 - sb)) << 23));
                if (nv != vs) {
                    const float f = nv / vs;
                    vs = nv;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < C; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i) O[nt][c][j][i] *= f;
                }
                weights();
            }
            // the weights in two parts of fp16, tokens g and g + 8
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float p0 = p[nt][2 * i], p1 = p[nt][2 * i + 1];
                    l[nt][0] += p0;
                    l[nt][1] += p1;
                    ph[nt][i] = Pack<__half>::down(p0, p1);
                    const float2 h = Pack<__half>::up(ph[nt][i]);
                    pl[nt][i] = Pack<__half>::down(p0 - h.x, p1 - h.y);
                }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uint32_t r[4];
                ldsm_x4_trans(r[0], r[1], r[2], r[3], vb + c * kQ4CellBytes + lm_off);
                uint32_t s2[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v = sv[c][i] * vs;
                    s2[i] = Pack<__half>::down(v, v);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t b[2], bl[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        za[nt][c][0] = fmaf(p[nt][2 * i], zv[c][i], za[nt][c][0]);
                        za[nt][c][1] = fmaf(p[nt][2 * i + 1], zv[c][i], za[nt][c][1]);
                        // times the scale: rounded, and what that and the weight left
                        const uint32_t hi = q4_mul2(ph[nt][i], s2[i]);
                        const uint32_t lo =
                            q4_fma2(pl[nt][i], s2[i], q4_fma2(ph[nt][i], s2[i], hi ^ 0x80008000u));
                        b[i] = q4_transpose(S::kDouble && t >= 2 ? lo : hi);
                        if (!S::kDouble) bl[i] = q4_transpose(lo);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t mask = j & 1 ? 0x00f000f0u : 0x000f000fu;
                        const int sh = j >> 1 ? 8 : 0;
                        const uint32_t a0 = (r[0] >> sh) & mask, a1 = (r[2] >> sh) & mask;
                        const uint32_t a2 = (r[1] >> sh) & mask, a3 = (r[3] >> sh) & mask;
                        q4_mma(O[nt][c][j], a0, a1, a2, a3, b[0], b[1]);
                        if (!S::kDouble) q4_mma(O[nt][c][j], a0, a1, a2, a3, bl[0], bl[1]);
                    }
                }
            }
        };

        uint32_t slot = 0, prev = (S::kStages - 1) * S::kStageBytes;
        while (used < asked) {
            q4_copy_wait<S::kStages - 2>();
            __syncwarp();  // the stage is whole, and nothing reads the one before any more
            ask(prev);
            if (fresh) begin_unit();
            chunk_step(slot);
            prev = slot;
            slot = slot == (S::kStages - 1) * S::kStageBytes ? 0 : slot + S::kStageBytes;
            fresh = ++used == asked || cu.chunk + 1 == cu.q.chunks;
            if (fresh) {
                end_unit();
                q4_next_unit<RT>(P, cu);
            } else {
                ++cu.chunk;
            }
        }
        q4_copy_wait<0>();
    }
    if (!P.whole) {
        if (lane == 0) P.tails[worker] = tail;
        pdl_trigger();
    }

    // rows without anything to attend over
    for (int s = blockIdx.x; s < P.num_seqs; s += gridDim.x) {
        const Q4Seq q = q4_seq<RT>(P, s);
        if (q.bad && tid == 0 && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
        if (q.chunks) continue;
        const int r0 = max(0, min(q.q0, P.num_tokens));
        const int r1 = max(r0, (int)min((long long)q.q0 + q.n, (long long)P.num_tokens));
        const size_t row = (size_t)P.num_heads * D * (P.out_f32 ? 4 : 2) / 16;
        uint4 *o = static_cast<uint4 *>(P.out);
        for (size_t i = r0 * row + tid; i < r1 * row; i += kQ4Threads) o[i] = make_uint4(0, 0, 0, 0);
    }
}

// Puts together the units that the main kernel's ranges cut.  CTA = the worker
// in whose range a unit begins; its parts are slot 1 of that worker and slot 0
// of the ones behind it.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(256) q4_merge_kernel(const __grid_constant__ Q4DecodeParams P) {
    constexpr int kLanes = D / 4;               // threads of a row, four channels each
    constexpr int kRowsAtOnce = 256 / kLanes;
    pdl_wait();
    const int worker = blockIdx.x;
    const int4 tail = P.tails[worker];
    if (tail.x < 0) return;
    const Q4Seq q = q4_seq<RT>(P, tail.x);
    const int head = tail.y, row0 = tail.z * RT;
    const int parts = 1 + tail.w, rows = min(RT, q.n * P.G - row0);
    const int d0 = (threadIdx.x % kLanes) * 4;
    for (int col = threadIdx.x / kLanes; col < rows; col += kRowsAtOnce) {
        float M = kQ4NoMax, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) {
            const size_t slot = i == 0 ? 2 * (size_t)worker + 1 : 2 * (size_t)(worker + i);
            const float2 ml = __ldcg(P.part_ml + slot * RT + col);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(P.part + (slot * RT + col) * D + d0));
            const float mn = fmaxf(M, ml.x);
            const float fa = ex2(M - mn), fb = ex2(ml.x - mn);
            M = mn;
            L = L * fa + ml.y * fb;
            acc.x = acc.x * fa + v.x * fb;
            acc.y = acc.y * fa + v.y * fb;
            acc.z = acc.z * fa + v.z * fb;
            acc.w = acc.w * fa + v.w * fb;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int r = row0 + col;
        const size_t out_row =
            (size_t)(q.q0 + r / P.G) * P.num_heads + (size_t)head * P.G + r % P.G;
        if (P.out_f32)
            *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + out_row * D + d0) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        else
            *reinterpret_cast<uint2 *>(static_cast<T *>(P.out) + out_row * D + d0) =
                make_uint2(Pack<T>::down(acc.x * inv, acc.y * inv), Pack<T>::down(acc.z * inv, acc.w * inv));
    }
}

}  // namespace pa
