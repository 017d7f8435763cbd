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
// subnormal, which the tensor cores multiply exactly), 0x00n0 are 16 n 2^-24 and a
// byte 0x00hl is (l + 16 h) 2^-24.  A 32-bit word's eight nibbles become the pairs
// l and l + 16 h by two ANDs, a byte permute and an AND; no subtraction, no
// conversion.  The other side of the product makes up for it: a value's two
// sums are subtracted at the end; a key's factors are q_1 / 16 for l + 16 h and q_0 - q_1 / 16
// for l, in two parts of fp16 in the two columns that a row has (with more than
// four rows, one column each: l and 16 h, by another shift, for q_0 and q_1 / 16).  It
// works in fp16 only (bf16 has no such subnormals), so a query row is scaled by
// the power of two that brings its largest element to 2^13; what fp16 then
// cannot hold of an element is below 2^-34 of the largest.
//
// Sums.  The tensor cores cut what does not fit a sum off, always towards zero: a sum
// of many terms of one sign, as n >= 0 makes it, loses half a step a product, the
// same way every time.  Over two documents of 131072 tokens, whose terms cancel to 1 / 200
// of their size, that was 1.6 10^-3 of the output.  So
//   - the weights p s, in fp32, go to fp16 as their first 8 bits and the rest (2^-19 of
//     them is rounded off that): products of 8 bits with l + 16 h below 256 fit the sum
//     of a chunk, and of most pairs of chunks, without being cut.  (A first part of 11
//     bits: 2^-22, but 8 10^-5 of the output.)
//   - the parts are summed apart: in columns, or in products, of their own;
//   - a sum is of one pack of chunks, or two; then it is added to the row's in fp32 with
//     ordinary rounding.
// 6 10^-6 of the output now.  (Sums that go on, and are brought back to their middle every
// eight chunks: 1.2 10^-4, and 142 us where this takes 139 for 256 sequences of 40 heads;
// whole numbers around 0, a subtraction for every operand: 1 10^-6, 156 us.)
// A power of two for every group of channels, moved now and then, keeps the largest of
// the weights p s between 2^10 and 2^15: what is below 2^-34 of that is rounded off.
// It follows the weights, not the scales: a token of huge values without weight does
// not move it, and other groups' scales do not.
//
// Few rows.  The products have eight columns.  With at most four rows a column is
// (chunk of 16 tokens, row, part of the weight): a step of 4 / rows chunks fills
// them, and each lane has two logits of one row, all different ones, instead of
// repeating a row's softmax in idle columns.  With more rows a column is a row, and
// the second parts have a product of their own.
//
// Softmax in one pass.  Each warp keeps a maximum m per row which it moves only
// when a weight has outgrown 2^4 (the first chunk, then rarely): the check is
// one comparison and a vote instead of exchanges between the lanes, and any m
// gives the same quotient.
//
// Work.  A warp works on its own, without barriers: it has a range of chunks (16
// tokens of a sequence's KV head) of the batch's, all laid end to end and cut
// into equal parts, and a ring of kStages stages of kStep chunks that it fills
// itself by bulk copies, one a lane for every K and V tile.  A (sequence, head,
// rows) that is cut leaves partial results, which the merge kernel puts together.
//
// Bound: HBM, 72 bytes a group and token of K and V.  256 sequences of 40 heads of
// 128, one row each: 139 us, 5.95 TB/s, 0.88 of the measured copy (an early form, of 137 us:
// 123 without the copies, 131 without the products).  With more rows the products and
// the softmax bound it (64 heads on 8, 125000 tokens: 49 us; the early form 48, 39 without
// the values' products, 27 without any and without copies): the warps that the
// registers leave (8 an SM) do not hide each other's latencies.
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
constexpr float kQ4NoMax = -0x1.fffffep127f;  // m before any token: no finite logit is below it
constexpr float kQ4NoRow = 0x1.fffffep127f;   // m of a tile's idle rows, whose weights are zero
// A weight, 2^-26 where the maximum was last taken, is taken anew beyond 2^-22 (so that
// the sum of 2^22 tokens' values is in range wherever the values are); weight times scale,
// 2^10 where the power of two was last taken, beyond 2^15 (fp16 ends at 2^16).
constexpr int kQ4HalfLog = 12;  // (of the logits' unit: half of the codes' 2^24)
constexpr float kQ4Half = 0x1p12f;
constexpr float kQ4Lift = 26.f, kQ4TopP = 0x1p-22f, kQ4TopW = 0x1p15f;

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
    float scale_log2, inv_G;
};

// Query token and head of row r of a sequence's rows, [token][G]: r / G of a number
// below 2^16 by a product in fp32 (a half is far more than its rounding).
__device__ __forceinline__ int q4_token_of(const Q4DecodeParams &P, int r) {
    return __float2int_rz(((float)r + 0.5f) * P.inv_G);
}
// The row of [num_tokens][num_heads] that has row r of the sequence from token q0 on.
__device__ __forceinline__ size_t q4_out_row(const Q4DecodeParams &P, int q0, int head, int r) {
    const int i = q4_token_of(P, r);
    return (size_t)(q0 + i) * P.num_heads + (size_t)(head * P.G + r - i * P.G);
}

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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same on a zeroed accumulator.
__device__ __forceinline__ void q4_mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// An 8 x 8 matrix of 16-bit units, spread as ldmatrix gives it, transposed.
__device__ __forceinline__ uint32_t q4_transpose(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// A weight's first part: its first 8 bits.
__device__ __forceinline__ float q4_first(float w) {
    return __int_as_float(__float_as_int(w) & 0xffff0000);
}

template <int D, int R>
struct Q4Shape {
    static constexpr int kCells = D / kQ4Group;
    static constexpr int kTileBytes = kCells * kQ4CellBytes;
    static constexpr int kChunkBytes = 2 * kTileBytes;
    // Chunks of a stage: what asking for them costs is shared by more where shared memory
    // has room.
    static constexpr int kStep = D == 256 ? 2 : R < 8 ? 4 : D == 64 ? 8 : 6;
    static constexpr int kStages = D == 64 && R < 8 ? 3 : 2;
    static constexpr bool kPacked = R <= 4;
    static constexpr int kPack = kPacked ? 4 / R : 1;        // chunks at once
    static constexpr int kUnroll = R >= 4 ? 2 : 1;           // packs at once
    static_assert(kStep % (kPack * kUnroll) == 0, "packs are of one stage");
    static constexpr int kTiles8 = kPacked ? 1 : R / 8;      // groups of eight columns
    static constexpr int kRows = kPacked ? 1 : 2 * kTiles8;  // rows of a lane
    // What a unit costs beside its chunks, in chunks: its query, the first maxima, its
    // output, half a pack that is not full.  The warps' shares count it.
    static constexpr int kUnitCost = 3 + kPack;
    static constexpr int kStageBytes = kStep * kChunkBytes;
    // CTAs an SM: what the registers allow without spills, which cost more than warps bring
    // (drafts of five tokens, 32 heads on 8 of 128: 87 us with two, 105 with three; 12 heads
    // on 2 of 256: 35 and 45; but 40 heads of 128, one row each: 166 with two, 143 with three)
    static constexpr int kCtas = D == 256 || (D == 128 && R >= 8) ? 2 : D == 64 && R < 8 ? 4 : 3;
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

template <typename T, int D, int R>
__global__ void __launch_bounds__(kQ4Threads, (Q4Shape<D, R>::kCtas))
    q4_decode_kernel(const __grid_constant__ Q4DecodeParams P) {
    using S = Q4Shape<D, R>;
    constexpr int NT = S::kTiles8, C = S::kCells, NR = S::kRows, kPack = S::kPack;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ long long s_base[kQ4Threads];  // length of the batch before a thread's sequences
    __shared__ long long s_warp[kQ4Warps];
    __shared__ uint64_t s_full[kQ4Warps][S::kStages];
    __shared__ uint32_t s_lost[kQ4Warps][S::kStages];  // tiles of a stage that were not copied
    __shared__ int s_never;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    if (tid == 0) s_never = 0;
    if (lane == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&s_full[warp][i], 1);
            s_lost[warp][i] = 0;
        }
        fence_mbar_init();
    }
    // (Lengths and tables are read before the wait, as the other decode calls read
    // them: the search below and the first block ids overlap the kernel ahead.)

    // The batch's units, laid end to end, each its chunks' number and S::kUnitCost
    // long; thread i's sequences are i * each ..
    const int each = (P.num_seqs + kQ4Threads - 1) / kQ4Threads;
    long long mine = 0;
    for (int s = tid * each; s < min(P.num_seqs, (tid + 1) * each); ++s) {
        const Q4Seq q = q4_seq<R>(P, s);
        if (q.chunks) mine += (long long)(q.chunks + S::kUnitCost) * q.tiles * P.num_kv_heads;
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
    // (a 64-bit division takes longer than the rest of the search)
    const long long per =
        total <= 0x7fffffffll - P.workers
            ? max(((int)total + P.workers - 1) / P.workers, 1)
            : (total + P.workers - 1) / P.workers;
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
            q4_next_seq<R>(P, at);
            if (at.s >= P.num_seqs) break;
            const long long n =
                (long long)(at.q.chunks + S::kUnitCost) * at.q.tiles * P.num_kv_heads;
            if (off < n) break;
            off -= n;
        }
        // A range that begins in what a unit costs beside its chunks has its first chunk.
        const int count = (int)(end - start);  // length of the range
        int pos = 0;                           // of `at` in it
        if (at.s < P.num_seqs) {
            const int length = at.q.chunks + S::kUnitCost;
            const int unit = (int)off / length, o = (int)off - unit * length;
            at.chunk = max(0, o - S::kUnitCost);
            pos = max(0, S::kUnitCost - o);
            at.head = unit / at.q.tiles;
            at.tile = unit - at.head * at.q.tiles;
            if (P.whole && at.chunk > 0) {  // that unit is the worker's in whose range it begins
                pos = length - o + S::kUnitCost;
                q4_next_unit<R>(P, at);
            }
        }
        Q4Cursor cu = at;  // the chunk at hand
        const int pos0 = pos;
        uint8_t *ring = s_ring + (size_t)warp * S::kStages * S::kStageBytes;
        const uint32_t ring_u32 = smem_u32(ring);

        // ---- asking for chunks ----
        const uint32_t block_bytes = (uint32_t)(P.num_kv_heads << P.sub_shift) * S::kTileBytes;
        const int sub_mask = (1 << P.sub_shift) - 1;
        const uint8_t *lane_pool = lane & 1 ? P.v_cache : P.k_cache;
        const uint64_t policy = l2_evict_first_policy();
        int asked = 0, used = 0;  // steps
        bool any_lost = false;    // a block was outside the pool: s_lost counts from then on
        int ids = 0;              // the lane's block id, of chunk ids_c + lane
        int ids_c = 1 << 30;
        // chunks of the step at a cursor that has `left` chunks of the range before it
        auto step_chunks = [&](const Q4Cursor &c, int left) {
            const int n = min(S::kStep, c.q.chunks - c.chunk);
            return P.whole ? n : min(n, left);
        };
        // What the next step needs, on its way while the one before is worked on: the block
        // ids, and for a unit's first step its query rows (128 bytes a lane).
        auto look_ahead = [&]() {
            if (at.s >= P.num_seqs) return;
            if (at.chunk < ids_c || at.chunk + S::kStep > ids_c + 32) {
                ids_c = at.chunk;
                const int c = ids_c + lane;
                ids = c < at.q.chunks ? P.block_tables[(size_t)at.s * P.max_blocks_per_seq +
                                                       (c >> P.sub_shift)]
                                      : 0;
            }
            const int r = at.tile * R + lane / C;
            if (at.chunk == 0 && lane < R * C && r < at.q.n * P.G) {
                const size_t row = q4_out_row(P, at.q.q0, at.head, r);
                prefetch_l2(static_cast<const T *>(P.query) + row * D + lane % C * kQ4Group);
            }
        };
        auto ask = [&]() {
            if (at.s >= P.num_seqs || !(pos < count || (P.whole && at.chunk > 0))) return;
            const int n = step_chunks(at, count - pos);
            const int stage = asked % S::kStages;
            // lane 2j: K tile of chunk j, lane 2j + 1: its V tile
            const int c = at.chunk + (lane >> 1);
            const int id = __shfl_sync(0xffffffffu, ids, (c - ids_c) & 31);
            const bool mine = lane < 2 * n, good = (unsigned)id < (unsigned)P.num_blocks;
            const uint32_t copies = __ballot_sync(0xffffffffu, mine && good);
            const uint32_t lost = ~copies & (uint32_t)((1ull << (2 * n)) - 1ull);
            any_lost |= lost != 0;
            if (lane == 0) {
                mbar_arrive_expect_tx(&s_full[warp][stage], __popc(copies) * S::kTileBytes);
                if (any_lost) s_lost[warp][stage] = lost;
                if (lost && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
            }
            __syncwarp();
            if (mine && good) {
                const size_t o = (size_t)(uint32_t)id * block_bytes +
                                 (size_t)((uint32_t)(at.head << P.sub_shift) + (uint32_t)(c & sub_mask)) *
                                     S::kTileBytes;
                bulk_g2s(ring + stage * S::kStageBytes + lane * S::kTileBytes, lane_pool + o,
                         S::kTileBytes, &s_full[warp][stage], policy);
            }
            ++asked;
            pos += n;
            at.chunk += n;
            if (at.chunk == at.q.chunks) {
                pos += S::kUnitCost;
                if (q4_next_unit<R>(P, at)) ids_c = 1 << 30;
            }
            look_ahead();
        };
        look_ahead();
        pdl_wait();  // earlier kernels on the stream may still write the query and the cache
        pdl_trigger();  // (what follows waits for this kernel's end before it touches its data)
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) ask();

        // Whether the next step's chunks are here.  The warp goes on or gives up as a whole: one
        // lane's wait may give up where another's just ends, and those that go on would
        // exchange data with lanes that are gone, with copies in flight when the CTA has ended.
        auto arrived = [&]() {
            const bool mine = mbar_wait(&s_full[warp][used % S::kStages], (used / S::kStages) & 1u, &s_never);
            return __all_sync(0xffffffffu, mine) != 0;
        };
        bool gone = false;  // a wait gave up
        // (the test build's few polls: right behind the copies, before these can have come)
        if constexpr (kShortWaits) gone = used < asked && !arrived();

        // ---- the unit at hand ----
        // A lane's rows: packed, row t % R of chunk t / R of a pack; else 2t and 2t + 1 of
        // every eight.
        float O[NT][C][4][4];     // [rows of 16 channels: cell, nibble][fragment]
        float m[NR], l[NR], za[NR][C];
        uint32_t qf[NT][C][2][2][2];  // the query's fragments: cell, half, nibble pair
        float c1[NR], qz[NR][C];
        int lim[NR], lim_min = 0;     // tokens a row sees; the fewest of any
        float vs[C];                  // power of two on the values' scales, by group of channels
        int first_chunk = 0, rows = 0, row0 = 0, upos = pos0;
        // (a tile of at most eight rows leaves the second eight columns out)
        auto empty = [&](int nt) { return nt > 0 && rows <= 8 * nt; };
        bool fresh = true;            // the step at hand begins a unit, or the range
        const int jl = S::kPacked ? t / R : 0;  // the lane's chunk of a pack

        // 1 where chunk j of a pack is the lane's: its logits, its columns of the weights.
        float own_f[kPack];
        uint32_t own_c[kPack];
#pragma unroll
        for (int j = 0; j < kPack; ++j) {
            own_f[j] = S::kPacked && t / R == j ? 1.f : 0.f;
            own_c[j] = S::kPacked && (g >> 1) / R == j ? 1u : 0u;
            asm volatile("" : "+f"(own_f[j]), "+r"(own_c[j]));
        }

        auto begin_unit = [&]() {
            first_chunk = cu.chunk;
            row0 = cu.tile * R;
            rows = min(R, cu.q.n * P.G - row0);
            const int seen0 = cu.q.len - cu.q.n + 1;
            lim_min = seen0 + q4_token_of(P, row0);
#pragma unroll
            for (int c = 0; c < C; ++c) vs[c] = 1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int col = S::kPacked ? (g >> 1) % R : nt * 8 + g;
                const size_t row = q4_out_row(P, cu.q.q0, cu.head, row0 + col);
                float f[C][2][8];
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (col < rows) {
                            // (from L2: what this SM has read of its line before the wait for
                            // the kernel ahead may be older than what that has written)
                            w = __ldcg(reinterpret_cast<const uint4 *>(
                                static_cast<const T *>(P.query) + row * D + c * 64 + h * 32 + 8 * t));
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
                // a product's factor (the codes' 2^24 in two halves, here and with the maxima:
                // in one the factor may overflow where no logit does)
                const float back = __int_as_float((254 + kQ4HalfLog - nb) << 23) * P.scale_log2;
                float sum[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    sum[c] = 0.f;
                    float sum16 = 0.f;  // of the odd elements, a sixteenth
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // elements 2i (+ 4) and 2i + 1 (+ 4) of the word's eight
                            const float e0 = f[c][h][2 * i] * norm, e4 = f[c][h][2 * i + 4] * norm;
                            const float o0 = f[c][h][2 * i + 1] * (norm * 0.0625f);
                            const float o4 = f[c][h][2 * i + 5] * (norm * 0.0625f);
                            sum[c] += e0 + e4;
                            sum16 += o0 + o4;
                            uint32_t(&q)[2] = qf[nt][c][h][i];
                            if (!S::kPacked) {
                                q[0] = Pack<__half>::down(e0, e4);
                                q[1] = Pack<__half>::down(o0, o4);
                            } else {
                                // for n_0 and n_0 + 16 n_1: even columns the factors, odd ones
                                // what their rounding left
                                q[0] = Pack<__half>::down(e0 - o0, e4 - o4);
                                q[1] = Pack<__half>::down(o0, o4);
                                const float2 h0 = Pack<__half>::up(q[0]), h1 = Pack<__half>::up(q[1]);
                                if (g & 1) {
                                    q[0] = Pack<__half>::down(e0 - o0 - h0.x, e4 - o4 - h0.y);
                                    q[1] = Pack<__half>::down(o0 - h1.x, o4 - h1.y);
                                }
                            }
                        }
                    }
                    sum[c] = fmaf(16.f, sum16, sum[c]);
                    sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 1);
                    sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 2);
                    sum[c] = sum[c] * 0x1p-24f * back;
                }
#pragma unroll
                for (int e = 0; e < (S::kPacked ? 1 : 2); ++e) {
                    const int i = 2 * nt + e;
                    const int mine = S::kPacked ? t % R : 2 * t + e;  // row of the eight
                    const int src = S::kPacked ? 8 * mine : 4 * mine;  // a lane that has its sums
                    c1[i] = __shfl_sync(0xffffffffu, back, src);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        qz[i][c] = __shfl_sync(0xffffffffu, sum[c], src);
                        za[i][c] = 0.f;
                    }
                    lim[i] = seen0 + q4_token_of(P, row0 + nt * 8 + mine);
                    m[i] = nt * 8 + mine < rows ? kQ4NoMax : kQ4NoRow;
                    l[i] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) O[nt][c][j][i] = 0.f;
            }
        };

        // Sum over the lanes that have a row's other tokens.
        auto row_sum = [&](float v) {
#pragma unroll
            for (int o = S::kPacked ? R : 4; o < 32; o <<= 1)
                v += __shfl_xor_sync(0xffffffffu, v, o);
            return v;
        };

        // What the unit's chunks so far give, up to chunk `stop`, to the output or, where it
        // is cut, to the workspace: slot 0 of a worker is its first unit's if that began
        // before, slot 1 its last one's.
        auto end_unit = [&](int stop) {
            const bool all = first_chunk == 0 && stop == cu.q.chunks;
            const int slot = 2 * worker + (first_chunk == 0 ? 1 : 0);
            if (!all && first_chunk == 0)
                tail = make_int4(cu.q.q0, cu.head, row0,
                                 (cu.q.chunks - stop + (int)per - 1) / (int)per << 5 | rows);
            float unscale[C];  // 1 / vs (2^24, of the codes as fp16, apart: together they may overflow)
#pragma unroll
            for (int c = 0; c < C; ++c) unscale[c] = __int_as_float((254 << 23) - __float_as_int(vs[c]));
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int nt = i / 2, e = i % 2;
                const int row = S::kPacked ? t % R : nt * 8 + 2 * t + e;  // of the tile
                const bool in = row < rows && (!S::kPacked || t < R);
                const size_t out_row = q4_out_row(P, cu.q.q0, cu.head, row0 + row);
                const float ls = row_sum(l[i]);
                const float inv = !all ? 1.f : ls == 0.f ? 0.f : __fdividef(1.f, ls);
                if (!all && in && g == 0) P.part_ml[(size_t)slot * R + row] = make_float2(m[i], ls);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float z = row_sum(za[i][c]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (S::kPacked) {  // both parts, and the pack's chunks
                                v[j] = O[nt][c][j][2 * h] + O[nt][c][j][2 * h + 1];
#pragma unroll
                                for (int o = R; o < 4; o <<= 1)
                                    v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
                            } else {
                                v[j] = O[nt][c][j][2 * h + e];
                            }
                        }
                        v[1] = (v[1] - v[0]) * 0x1p20f;  // n_0 + 16 n_1 -> n_1
                        v[3] = (v[3] - v[2]) * 0x1p20f;
                        v[0] *= 0x1p24f;
                        v[2] *= 0x1p24f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = fmaf(v[j], unscale[c], z) * inv;
                        const int d0 = c * 64 + h * 32 + 4 * g;
                        if (!in) continue;
                        if (!all) {
                            *reinterpret_cast<float4 *>(P.part + ((size_t)slot * R + row) * D + d0) =
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

        // The products of a K tile's cell with the query.
        auto keys = [&](uint32_t cell, int c, float (&acc)[NT][4]) {
            uint32_t r[4];
            ldsm_x4(r[0], r[1], r[2], r[3], cell + lm_off);
#pragma unroll
            for (int nt = 1; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t a0, a1, a2, a3;
                    if (S::kPacked) {
                        a2 = i ? __byte_perm(r[2 * h], 0, 0x4341) : r[2 * h] & 0x00ff00ffu;
                        a3 = i ? __byte_perm(r[2 * h + 1], 0, 0x4341) : r[2 * h + 1] & 0x00ff00ffu;
                        a0 = a2 & 0x000f000fu;
                        a1 = a3 & 0x000f000fu;
                    } else {
                        const uint32_t lo = r[2 * h] >> (8 * i), hi = r[2 * h + 1] >> (8 * i);
                        a0 = lo & 0x000f000fu, a1 = hi & 0x000f000fu;
                        a2 = lo & 0x00f000f0u, a3 = hi & 0x00f000f0u;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (empty(nt)) break;
                        const uint32_t(&q)[2] = qf[nt][c][h][i];
                        if (nt == 0 && h == 0 && i == 0) q4_mma_first(acc[nt], a0, a1, a2, a3, q[0], q[1]);
                        else q4_mma(acc[nt], a0, a1, a2, a3, q[0], q[1]);
                    }
                }
        };
        // The products of a V tile's cell (its words in r) with weights; first: no sums yet.
        auto values = [&](const uint32_t (&r)[4], float (&o)[4][4], uint32_t b0, uint32_t b1, bool first) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = j ? __byte_perm(r[i], 0, 0x4341) : r[i] & 0x00ff00ffu;
                const uint32_t n[4] = {w[0] & 0x000f000fu, w[1] & 0x000f000fu, w[2] & 0x000f000fu,
                                       w[3] & 0x000f000fu};
                if (first) {
                    q4_mma_first(o[2 * j], n[0], n[2], n[1], n[3], b0, b1);
                    q4_mma_first(o[2 * j + 1], w[0], w[2], w[1], w[3], b0, b1);
                } else {
                    q4_mma(o[2 * j], n[0], n[2], n[1], n[3], b0, b1);
                    q4_mma(o[2 * j + 1], w[0], w[2], w[1], w[3], b0, b1);
                }
            }
        };

        // U packs of chunks from chunk `chunk` on, `n` of them there, in the stage at `at_pack`;
        // lost: bits of the tiles that were not copied.  (Two packs, where the registers
        // allow: one's products run while the other's logits are worked on.)
        constexpr int U = S::kUnroll;
        auto pack_step = [&](uint32_t at_pack, int chunk, int n, uint32_t lost) {
            const uint32_t base = ring_u32 + at_pack;
            // the scales of the lane's chunk
            const uint8_t *pk = ring + at_pack + jl * (S::kPacked ? S::kChunkBytes : 0) +
                                kQ4CellParams + 4 * g;
            constexpr int kPackBytes = kPack * S::kChunkBytes;
            // x = scale <q, k> in units of 2^12 log2, tokens g and g + 8 of the lane's rows
            float x[U][NR][2];
            float a[U][C][NR][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < kPack; ++j)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float acc[NT][4];
                        keys(base + u * kPackBytes + j * S::kChunkBytes + c * kQ4CellBytes, c, acc);
                        if constexpr (S::kPacked) {
                            // the lane's chunk, by a factor of 0 or 1: not another
                            // instruction for the integer pipe
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float v = acc[0][2 * k], w = acc[0][2 * k + 1];
                                float &o = a[u][c][0][k];
                                if (kPack == 1) o = v + w;
                                else o = fmaf(w, own_f[j], j == 0 ? v * own_f[j] : fmaf(v, own_f[j], o));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < NR; ++i) {
                                a[u][c][i][0] = acc[i / 2][i % 2];
                                a[u][c][i][1] = acc[i / 2][2 + i % 2];
                            }
                        }
                    }
            // the values' scales and least values
            float sv[U][C][2], zv[U][C][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint8_t *pu = pk + u * kPackBytes;
                float y[NR][2];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float2 p0 = Pack<T>::up(*reinterpret_cast<const uint32_t *>(pu + c * kQ4CellBytes));
                    const float2 p1 = Pack<T>::up(*reinterpret_cast<const uint32_t *>(pu + c * kQ4CellBytes + 32));
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        y[i][0] = c == 0 ? p0.x * a[u][c][i][0] : fmaf(p0.x, a[u][c][i][0], y[i][0]);
                        y[i][1] = c == 0 ? p1.x * a[u][c][i][1] : fmaf(p1.x, a[u][c][i][1], y[i][1]);
                        x[u][i][0] = c == 0 ? p0.y * qz[i][c] : fmaf(p0.y, qz[i][c], x[u][i][0]);
                        x[u][i][1] = c == 0 ? p1.y * qz[i][c] : fmaf(p1.y, qz[i][c], x[u][i][1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) x[u][i][k] = fmaf(y[i][k], c1[i], x[u][i][k]);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 p = Pack<T>::up(*reinterpret_cast<const uint32_t *>(
                            pu + S::kTileBytes + c * kQ4CellBytes + 32 * k));
                        sv[u][c][k] = p.x;
                        zv[u][c][k] = p.y;
                    }
            }
            if (n < U * kPack || lost || (chunk + U * kPack) * kQ4Tokens > lim_min) {
                // past the context or the range, past a row's own token, or a block that was
                // skipped: whatever lies there must not meet a weight, not even one of zero
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = u * kPack + jl;
                    const bool there = j < n && !((lost >> (2 * j)) & 3u);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int tok = (chunk + j) * kQ4Tokens + g + 8 * k;
#pragma unroll
                        for (int i = 0; i < NR; ++i)
                            if (!there || tok >= lim[i]) x[u][i][k] = -INFINITY;
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            float &s = sv[u][c][k], &z = zv[u][c][k];
                            const bool in = there && tok < cu.q.len;
                            const bool nan = !(s + z == s + z);
                            if (in && nan)  // of the rows that see it alone
#pragma unroll
                                for (int i = 0; i < NR; ++i)
                                    if (tok < lim[i]) za[i][c] = NAN;
                            if (!in || nan) s = z = 0.f;
                        }
                    }
                }
            }
            // Weights, and what is to be multiplied out: packed, weight times scale (the power of
            // two first: finite whatever the scale, and zero where the weight is); else the
            // scales times the power of two, below.  A token's largest weight and largest
            // scale bound its products.
            float p[U][NR][2], pm[U][2], w[U][C][2], top;
            auto weights = [&]() {
                top = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pm[u][k] = 0.f;
#pragma unroll
                        for (int i = 0; i < NR; ++i) {
                            p[u][i][k] = ex2(fmaf(x[u][i][k], kQ4Half, -m[i]));
                            pm[u][k] = fmaxf(pm[u][k], p[u][i][k]);
                        }
                        if constexpr (S::kPacked) {
                            top = fmaxf(top, p[u][0][k] * (kQ4TopW / kQ4TopP));
#pragma unroll
                            for (int c = 0; c < C; ++c) {
                                w[u][c][k] = p[u][0][k] * vs[c] * sv[u][c][k];
                                top = fmaxf(top, w[u][c][k]);
                            }
                        } else {
                            float s = kQ4TopW / kQ4TopP;
#pragma unroll
                            for (int c = 0; c < C; ++c) s = fmaxf(s, sv[u][c][k] * vs[c]);
                            top = fmaxf(top, pm[u][k] * s);
                        }
                    }
            };
            weights();
            if (__any_sync(0xffffffffu, top > kQ4TopW)) {
                // new maxima, and new powers of two on the scales
                float kept = 0.f;  // what stays of a row's sums, of the row with the most
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    float a = fmaxf(x[0][i][0], x[0][i][1]);
#pragma unroll
                    for (int u = 1; u < U; ++u) a = fmaxf(a, fmaxf(x[u][i][0], x[u][i][1]));
#pragma unroll
                    for (int o = S::kPacked ? R : 4; o < 32; o <<= 1)
                        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                    a = fmaxf(fmaf(a, kQ4Half, kQ4Lift), m[i]);
                    const float f = ex2(m[i] - a);
                    m[i] = a;
                    if (l[i] > 0.f) kept = fmaxf(kept, f);
                    l[i] *= f;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        za[i][c] *= f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (S::kPacked) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) O[0][c][j][k] *= f;
                            } else {
                                O[i / 2][c][j][i % 2] *= f;
                                O[i / 2][c][j][2 + i % 2] *= f;
                            }
                        }
                    }
                }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    kept = fmaxf(kept, __shfl_xor_sync(0xffffffffu, kept, o));
                weights();  // (for the maxima alone)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float e = -INFINITY;  // log2 of the largest weight times scale of the packs
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) e = fmaxf(e, lg2(pm[u][k]) + lg2(sv[u][c][k]));
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1)
                        e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
                    // up by no more than the sums have just come down, so that they stay in range
                    const int was = (__float_as_int(vs[c]) >> 23) - 127;
                    const int now = __float2int_rd(
                        fmaxf(-126.f, fminf(126.f, fminf(10.f - e, (float)was - lg2(kept)))));
                    const float f = __int_as_float((max(-126, min(127, now - was)) + 127) << 23);
                    vs[c] = __int_as_float((now + 127) << 23);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) O[nt][c][j][i] *= f;
                }
                weights();
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // (finite beside a weight of zero)
                        if constexpr (!S::kPacked) w[u][c][k] = fminf(sv[u][c][k] * vs[c], 0x1p127f);
                    }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    l[i] += p[u][i][0] + p[u][i][1];
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        za[i][c] = fmaf(p[u][i][0], zv[u][c][0], fmaf(p[u][i][1], zv[u][c][1], za[i][c]));
                }
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (empty(nt)) break;
                    float o[4][4], ol[4][4];  // this step's sums; ol: not packed, of the second parts
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint32_t v_at = base + u * kPackBytes + S::kTileBytes + lm_off + c * kQ4CellBytes;
                        uint32_t b[2], bl[2];
                        if constexpr (S::kPacked) {
                            // both parts of a weight side by side: columns 2t and 2t + 1
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float hi = q4_first(w[u][c][k]);
                                b[k] = q4_transpose(Pack<__half>::down(hi, w[u][c][k] - hi));
                            }
#pragma unroll
                            for (int j = 0; j < kPack; ++j) {
                                uint32_t r[4];
                                ldsm_x4_trans(r[0], r[1], r[2], r[3], v_at + j * S::kChunkBytes);
                                // a chunk's weights are in its own columns
                                if (kPack == 1) values(r, o, b[0], b[1], u == 0 && j == 0);
                                else values(r, o, b[0] * own_c[j], b[1] * own_c[j], u == 0 && j == 0);
                            }
                        } else {
                            uint32_t r[4];
                            ldsm_x4_trans(r[0], r[1], r[2], r[3], v_at);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {  // tokens g and g + 8, of two columns
                                const float w0 = p[u][2 * nt % NR][k] * w[u][c][k];
                                const float w1 = p[u][(2 * nt + 1) % NR][k] * w[u][c][k];
                                const float h0 = q4_first(w0), h1 = q4_first(w1);
                                b[k] = q4_transpose(Pack<__half>::down(h0, h1));
                                bl[k] = q4_transpose(Pack<__half>::down(w0 - h0, w1 - h1));
                            }
                            values(r, ol, bl[0], bl[1], u == 0);
                            values(r, o, b[0], b[1], u == 0);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            O[nt][c][j][i] += S::kPacked ? o[j][i] : o[j][i] + ol[j][i];
                }
            }
        };

        while (used < asked) {
            const int stage = used % S::kStages;
            if (gone || !arrived()) {
                gone = true;
                break;
            }
            __syncwarp();  // nothing reads the stage before this one any more
            ask();
            if (fresh) begin_unit();
            const int n = step_chunks(cu, count - upos);
            const uint32_t lost = any_lost ? s_lost[warp][stage] : 0u;
            for (int j = 0; j < n; j += U * kPack)
                pack_step(stage * S::kStageBytes + j * S::kChunkBytes, cu.chunk + j, n - j, lost >> (2 * j));
            ++used;
            upos += n;
            cu.chunk += n;
            fresh = used == asked || cu.chunk == cu.q.chunks;
            if (fresh) {
                end_unit(cu.chunk);
                if (cu.chunk == cu.q.chunks) {
                    upos += S::kUnitCost;
                    q4_next_unit<R>(P, cu);
                }
            }
        }
        if (gone) {
            if (lane == 0 && P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
            for (; used < asked; ++used)  // the warp's copies in flight
                mbar_drain_wait(&s_full[warp][used % S::kStages], (used / S::kStages) & 1u, &s_never);
        }
    }
    pdl_wait();  // (the warps without work)
    pdl_trigger();
    if (!P.whole && lane == 0) P.tails[worker] = tail;

    // rows without anything to attend over
    for (int s = blockIdx.x; s < P.num_seqs; s += gridDim.x) {
        const Q4Seq q = q4_seq<R>(P, s);
        if (q.bad && tid == 0 && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
        if (q.chunks) continue;
        const int r0 = max(0, min(q.q0, P.num_tokens));
        const int r1 = max(r0, (int)min((long long)q.q0 + q.n, (long long)P.num_tokens));
        const size_t row = (size_t)P.num_heads * D * (P.out_f32 ? 4 : 2) / 16;
        uint4 *o = static_cast<uint4 *>(P.out);
        for (size_t i = r0 * row + tid; i < r1 * row; i += kQ4Threads) o[i] = make_uint4(0, 0, 0, 0);
    }
}

// Puts together the units that the main kernel's ranges cut: the unit that
// begins in a worker's range and goes on has its parts in slot 1 of that worker
// and slot 0 of the ones behind it.  A CTA takes kQ4MergeTails neighbouring workers,
// a quarter of its warps each; where one of their units has many parts, all warps
// take one after the other.  A warp sums some of the parts of a row with many
// loads in flight (what takes time here is the chain of loads); shared memory joins
// the warps of a row.  64 sequences of up to 4096 tokens, 12 heads on 2 of 128: 4 of 20 us.
constexpr int kQ4MergeThreads = 512;
constexpr int kQ4MergeTails = 4;
constexpr int kQ4MergeMany = 12;  // parts
template <typename T, int D, int R>
__global__ void __launch_bounds__(kQ4MergeThreads)
    q4_merge_kernel(const __grid_constant__ Q4DecodeParams P) {
    constexpr int kWarps = kQ4MergeThreads / 32, kVec = D / 32;  // channels of a lane
    __shared__ float s_acc[kWarps][D];
    __shared__ float2 s_ml[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    int most = 0;
    int4 tails[kQ4MergeTails];
#pragma unroll
    for (int i = 0; i < kQ4MergeTails; ++i) {
        tails[i] = __ldcg(P.tails + blockIdx.x * kQ4MergeTails + i);
        if (tails[i].x >= 0) most = max(most, (tails[i].w >> 5) + 1);
    }
    if (most == 0) return;
    const bool together = most > kQ4MergeMany;
    const int group = together ? kWarps : kWarps / kQ4MergeTails;  // warps of a unit
    const int in_group = warp % group;
    // rows at once, and the warps of each (the same in every group of the CTA, whatever
    // rows its unit has: the barriers below are the CTA's)
    const int at_once = min(R, group), share = group / at_once;
    const int mine = in_group % share;
    for (int turn = 0; turn < (together ? kQ4MergeTails : 1); ++turn) {
        const int which = together ? turn : warp / group;
        int4 tail = tails[0];
#pragma unroll
        for (int i = 1; i < kQ4MergeTails; ++i)
            if (which == i) tail = tails[i];
        const int rows = tail.x >= 0 ? tail.w & 31 : 0, row0 = tail.z;
        const int parts = 1 + (tail.w >> 5);
        const size_t worker = (size_t)blockIdx.x * kQ4MergeTails + which;
        auto slot = [&](int i) { return i == 0 ? 2 * worker + 1 : 2 * (worker + i); };
        for (int first = 0; first < R; first += at_once) {
            const int row = first + in_group / share;
            const bool in = row < rows;
            float M = kQ4NoMax, L = 0.f, acc[kVec] = {};
            auto add = [&](float m, float l, const float (&x)[kVec]) {
                const float mn = fmaxf(M, m);
                const float fa = ex2(M - mn), fb = ex2(m - mn);
                M = mn;
                L = L * fa + l * fb;
#pragma unroll
                for (int k = 0; k < kVec; ++k) acc[k] = acc[k] * fa + x[k] * fb;
            };
            if (in) {
                constexpr int kBatch = D == 256 ? 6 : D == 128 ? 10 : 16;
                for (int i0 = mine; i0 < parts; i0 += kBatch * share) {
                    float2 ml[kBatch];
                    float x[kBatch][kVec];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int i = i0 + j * share;
                        if (i >= parts) break;
                        ml[j] = __ldcg(P.part_ml + slot(i) * R + row);
                        const float *v = P.part + (slot(i) * R + row) * D + lane * kVec;
                        if constexpr (kVec == 2) {
                            *reinterpret_cast<float2 *>(x[j]) = __ldcg(reinterpret_cast<const float2 *>(v));
                        } else {
#pragma unroll
                            for (int k = 0; k < kVec; k += 4)
                                *reinterpret_cast<float4 *>(x[j] + k) =
                                    __ldcg(reinterpret_cast<const float4 *>(v + k));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        if (i0 + j * share >= parts) break;
                        add(ml[j].x, ml[j].y, x[j]);
                    }
                }
            }
            // (behind the loads: 64 sequences of 2000 tokens, 64 heads on 8, take 49.8 us a
            // layer's write and attention, 52.2 where what follows is let in at the start)
            if (first + at_once >= R && (!together || turn + 1 == kQ4MergeTails)) pdl_trigger();
            if (mine > 0) {
#pragma unroll
                for (int k = 0; k < kVec; ++k) s_acc[warp][lane * kVec + k] = acc[k];
                if (lane == 0) s_ml[warp] = make_float2(M, L);
            }
            __syncthreads();
            if (mine == 0 && in) {
                for (int i = 1; i < share; ++i) {
                    float x[kVec];
#pragma unroll
                    for (int k = 0; k < kVec; ++k) x[k] = s_acc[warp + i][lane * kVec + k];
                    add(s_ml[warp + i].x, s_ml[warp + i].y, x);
                }
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const size_t o = q4_out_row(P, tail.x, tail.y, row0 + row) * D + lane * kVec;
                if (P.out_f32) {
#pragma unroll
                    for (int k = 0; k < kVec; k += 2)
                        *reinterpret_cast<float2 *>(static_cast<float *>(P.out) + o + k) =
                            make_float2(acc[k] * inv, acc[k + 1] * inv);
                } else {
#pragma unroll
                    for (int k = 0; k < kVec; k += 2)
                        *reinterpret_cast<uint32_t *>(static_cast<T *>(P.out) + o + k) =
                            Pack<T>::down(acc[k] * inv, acc[k + 1] * inv);
                }
            }
            __syncthreads();
        }
    }
}

}  // namespace pa
