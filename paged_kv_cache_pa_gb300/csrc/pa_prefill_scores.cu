// pa_prefill_scores.cu -- the attention weight that the new tokens of a batch
// give to every cached token, added to the tokens' scores, on the
// 5th-generation tensor cores.
//
// What it computes: with p_ij = exp(scale <q_i, k_j> - lse_i) for new token i
// at position c + i and key j <= c + i (lse_i from pa_prefill_attention_lse),
//     scores[s][hk][j] += sum over the group's heads and the rows i of p_ij.
//
// Because lse is known, a weight needs no running maximum and no second pass,
// and the sum over queries is taken with the keys on the rows: S = K Q^T puts
// key j in tensor-memory lane j and the queries in the columns, so one thread
// reads a key's whole row of S and adds it up alone -- no shuffles, no atomics,
// a fixed order.
//
// How.  A work item is 256 keys of one (sequence, KV head): two tiles of 128
// keys that share every query tile, which halves the query traffic from L2.  A
// query tile is up to 128 (token, head) rows, NH heads of the group times NQ
// tokens, one TMA box.  The kernel is persistent, one CTA per SM; items are
// numbered from the first keys on (with whole prompts those see the most
// queries) and dealt out forth and back, so every CTA's share is about as
// heavy.  Each CTA works the numbering out for itself in shared memory, from
// the lengths: only ranges that hold keys are numbered (sequences ordered by
// their number of ranges, so range k's are the first of them), and an item's
// sequence is at hand without a trip to memory.  Batches past kMaxTableSeqs
// sequences or kMaxTableRanges ranges number every range up to the longest and
// pass over the empty ones.
// Twenty warps:
//   * warp 0: K tiles into a ring of 128-key slots, block by block (tiled bulk
//     copies, TMA, one for a block's share: a warp issues one in about 60
//     cycles, which counts with small blocks); it runs ahead into the next
//     items;
//   * warps 1 and 2: S_t = K_t Q^T (M = 128 keys, N = the tile's rows,
//     K = head_dim) for key tile 0 and 1 into one of two tensor-memory buffers
//     each (two issuers: the waits of one fall into the other's products; both
//     pass through every tile of both rings, their own or not);
//     causal: a key tile starts with the query tile that holds the first token
//     to see its first key, so the second tile's copy has time while the first
//     one works alone.  Warp 1 allocates tensor memory;
//   * warp 3: query tiles into another ring, and beside them the rows' lse
//     (base 2, negated), with a flag for tiles that hold rows without a weight;
//   * warps 4..19: four groups of four, group (t, b) for the products of key
//     tile t in buffer b, one key a thread (the lanes a warp may read go by
//     its number modulo 4).  Each loads S from tensor memory 32 columns at a
//     time and sums 2^(x scale log2 e - lse) over the columns it may see -- a
//     range [lo, hi) of the tile, from its key's position.  At the item's end
//     group (t, 1) hands its sums to group (t, 0), which adds them and writes.
// Sums are fp32 in levels: the columns of a tile in pairs of chains, tiles,
// groups, CTAs.
//
// Few items (one prompt) leave most SMs idle and end with the longest, so a
// cluster of 2, 4 or 8 CTAs shares each: the query tiles in equal parts one
// after the other, and the first CTA's group (t, 0) adds the others' sums, in
// their order, through distributed shared memory.  One prompt, 32 heads on 8 of
// 128, with clusters and without: 4096 tokens 70 and 119 us, 1024 tokens 21 and
// 39 us.
//
// Bound: 2 prompts of 4096 tokens, 32 heads on 8 of 128, bf16, take 120 us; the
// products are 73 us at the rate of a large bf16 matrix product, and the sums 80
// at the 5.5 cycles a column that four busy warps of a scheduler take (four of
// them the exponential).  What keeps the two from overlapping is a buffer's
// turn: product, hand-over, the sums of all but its last columns, hand-over
// back, about 3500 cycles for two query tiles whose sums take 2800; tensor
// memory is full with two buffers a key tile.  (Query tiles of 256 rows with
// one buffer: 134 to 151 us.)  Windows of few queries are bound by the steps of
// an item one after the other: 8 of 32 queries on 3000 to 16384 tokens, 12
// heads on 2, take 18.5 us for 39 MB.
//
// A wait that gives up sets the abort flag; the groups then go through the
// rest of their items without waiting or writing, so that their named barriers
// always meet.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_nvtx.cuh"
#include "pa_ptx.cuh"
#include "pa_tmap.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace {

constexpr int kKeys = 128;    // keys of a tile (tensor-memory lanes)
constexpr int kTiles = 2;     // key tiles of an item
constexpr int kItemKeys = kKeys * kTiles;
constexpr int kChunk = 32;    // columns a thread holds at once
constexpr int kMaxCols = 128; // rows of a query tile
constexpr int kGroups = 4;    // of four warps: key tile and buffer
constexpr int kThreadsS = 128 + 128 * kGroups;
// registers a thread: 96 at launch (640 threads), then 104 for the groups and
// 64 for the other four warps -- no more than the same total
constexpr int kRegsLaunch = 96, kRegsSums = 104, kRegsOther = 64;
static_assert(128 * kGroups * kRegsSums + 128 * kRegsOther <= kThreadsS * kRegsLaunch,
              "register reallocation within the launch's registers");
constexpr uint32_t kTmemColsS = 512;  // S of tile t, buffer b at 128 (2 t + b)
constexpr uint32_t kKSlice = kKeys * 128;  // bytes of a 64-element slice of a K tile
constexpr int kMaxRing = 8;   // slots of the K and the query ring at most
constexpr uint32_t kTileBytes = 6 * 32768;  // shared memory of both tile rings
constexpr int kMaxParts = 8;  // CTAs that share one item at most (a cluster)
constexpr int kMaxTableSeqs = 512, kMaxTableRanges = 2047;  // sizes of the items' table

struct ScoreParams {
    CUtensorMap tmap_q;  // query as [head_dim/64][tokens][heads][64], box NQ x NH rows
    // pool rows as [rows/8][head_dim/64][8][64], box min(block, 64) rows: the two
    // 64-element slices of eight keys lie one after the other in a K tile
    CUtensorMap tmap_k;
    const float *lse;
    const int32_t *block_tables, *query_start_loc, *context_lens;
    float *scores;
    long long score_stride;
    int max_blocks_per_seq, block_shift, num_blocks;
    int max_query_len, max_context_len, num_seqs, num_tokens, num_heads, num_kv_heads, G;
    int nh, lg_nq;        // heads and log2 of the tokens of a query tile
    int head_groups;      // G / NH
    int rk, rq;           // slots of the K and the query ring
    unsigned rq_inv, kv_inv;  // small_inverse of rq and num_kv_heads
    unsigned num_items;   // 256-key ranges x num_seqs x num_kv_heads
    int ranges;           // 256-key ranges of the longest context
    int table;            // 1: items are numbered by the table in shared memory
    int lg_parts;         // log2 of the CTAs that share an item
    float scale_log2;
    unsigned int *err;
};

// The numbering of the items in shared memory.
struct STable {
    int tok0[kMaxTableSeqs], n[kMaxTableSeqs], L[kMaxTableSeqs];  // of each sequence
    unsigned short ranges[kMaxTableSeqs];  // its 256-key ranges (0: no work)
    unsigned short order[kMaxTableSeqs];   // sequences by ranges, most first
    unsigned first[kMaxTableRanges + 1];   // first item of range k; [ranges]: all items
};

// Shared memory: lse [slot][128], its flags [slot], the sums handed over
// [tile][128], barriers, the items' table; then, 1024-byte aligned, the K ring
// of rk tiles [16][slice][8 keys][64] and the query ring of rq tiles
// [slice][rows][64].
struct SLayout {
    static constexpr size_t dead_off = kMaxRing * kMaxCols * 4;
    static constexpr size_t part_off = dead_off + kMaxRing * 4;
    static constexpr size_t bar_off = part_off + kTiles * kKeys * 4;
    // k_full, k_free, q_full, q_free, l_full, l_free [kMaxRing], s_full[2][2],
    // s_free[2][2], done[2], c_full[2], c_free[2]
    static constexpr int kBars = 6 * kMaxRing + 8 + 2 + 4;
    static constexpr size_t tmem_off = bar_off + 8 * kBars;
    static constexpr size_t flag_off = tmem_off + 4;
    static constexpr size_t table_off = (flag_off + 4 + 15) / 16 * 16;
    // an item shared by a cluster: in its first CTA the sums of the others
    static constexpr size_t comb_off = (table_off + sizeof(STable) + 15) / 16 * 16;
    static constexpr size_t small =
        (comb_off + (kMaxParts - 1) * kItemKeys * 4 + 1023) / 1024 * 1024;
    static constexpr size_t bytes = small + kTileBytes;
    static_assert(bar_off % 8 == 0, "barrier alignment");
    static_assert(bytes <= 232448, "dynamic shared memory of one CTA");
};

struct SBars {
    uint64_t *k_full, *k_free, *q_full, *q_free, *l_full, *l_free, *s_full, *s_free, *done, *c_full,
        *c_free;
};

// A place in a ring: slot and the parity of its current phase.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// x / d for x below 2^31, by a multiplication: with inv = floor(2^32 / d) the
// high word of x inv is the quotient or one less.  (Every role works out every
// item.)
inline unsigned small_inverse(unsigned d) { return d == 1u ? 0xffffffffu : (unsigned)((1ull << 32) / d); }
__device__ __forceinline__ unsigned small_div(unsigned x, unsigned d, unsigned inv) {
    const unsigned q = __umulhi(x, inv);
    return x - q * d >= d ? q + 1u : q;
}

// One work item, worked out by every role for itself.
struct SItem {
    int s, hk;
    int n, L, c, tok0;  // new tokens, context length, cached before, first query row
    int k0;             // first key
    int tt0, tt1;       // token tiles that see some key of the item
    bool ok, any, run;  // lengths in order; work in the item; in this CTA's part
};

__device__ __forceinline__ bool lengths_ok(const ScoreParams &P, int a, int b, int L) {
    const int n = b - a;
    return a >= 0 && b <= P.num_tokens && n >= 0 && n <= P.max_query_len && L >= n &&
           L <= P.max_context_len;
}

// Fill the table (every thread of the CTA; ready after a barrier).  Up to 32
// sequences: every warp reads the lengths, a lane a sequence, and no step waits
// for another warp's (done after 1700 cycles instead of 3400).
__device__ __forceinline__ void number_items(const ScoreParams &P, STable &T) {
    const int tid = threadIdx.x, S = P.num_seqs;
    if (S <= 32) {
        const int s = tid & 31;
        int a = 0, b = 0, L = 0;
        if (s < S) {
            a = __ldg(&P.query_start_loc[s]);
            b = __ldg(&P.query_start_loc[s + 1]);
            L = __ldg(&P.context_lens[s]);
        }
        const bool ok = lengths_ok(P, a, b, L);
        const int mine = s < S && ok && b > a ? (L + kItemKeys - 1) / kItemKeys : 0;
        if (tid < S) {
            if (!ok && blockIdx.x == 0 && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
            T.tok0[s] = a;
            T.n[s] = b - a;
            T.L[s] = L;
        }
        int place = 0;
        unsigned before = 0u;  // items of the ranges before range tid
        for (int j = 0; j < S; ++j) {
            const int r = __shfl_sync(0xffffffffu, mine, j);
            place += r > mine || (r == mine && j < s);
            before += (unsigned)min(r, tid);
        }
        if (tid < S) T.order[place] = (unsigned short)s;
        if (tid <= P.ranges) T.first[tid] = before * (unsigned)P.num_kv_heads;
        for (int k0 = kThreadsS; k0 <= P.ranges; k0 += kThreadsS) {  // (whole warps)
            before = 0u;
            for (int j = 0; j < S; ++j)
                before += (unsigned)min(__shfl_sync(0xffffffffu, mine, j), k0 + tid);
            if (k0 + tid <= P.ranges) T.first[k0 + tid] = before * (unsigned)P.num_kv_heads;
        }
        return;
    }
    for (int s = tid; s < S; s += kThreadsS) {
        const int a = __ldg(&P.query_start_loc[s]), b = __ldg(&P.query_start_loc[s + 1]);
        const int L = __ldg(&P.context_lens[s]);
        const bool ok = lengths_ok(P, a, b, L);
        if (!ok && blockIdx.x == 0 && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
        T.tok0[s] = a;
        T.n[s] = b - a;
        T.L[s] = L;
        T.ranges[s] = ok && b > a ? (unsigned short)((L + kItemKeys - 1) / kItemKeys) : 0;
    }
    __syncthreads();
    for (int s = tid; s < S; s += kThreadsS) {
        const int mine = T.ranges[s];
        int place = 0;
        for (int j = 0; j < S; ++j) {
            const int r = T.ranges[j];
            place += r > mine || (r == mine && j < s);
        }
        T.order[place] = (unsigned short)s;
    }
    __syncthreads();
    for (int k = tid; k < P.ranges; k += kThreadsS) {  // sequences with more than k ranges
        int lo = 0, hi = S;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (T.ranges[T.order[mid]] > k) lo = mid + 1;
            else hi = mid;
        }
        T.first[k + 1] = (unsigned)lo * (unsigned)P.num_kv_heads;
    }
    __syncthreads();
    if (tid < 32) {
        unsigned carry = 0u;
        if (tid == 0) T.first[0] = 0u;
        for (int k0 = 1; k0 <= P.ranges; k0 += 32) {
            const int k = k0 + tid;
            unsigned v = k <= P.ranges ? T.first[k] : 0u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned u = __shfl_up_sync(0xffffffffu, v, o);
                if (tid >= o) v += u;
            }
            v += carry;
            if (k <= P.ranges) T.first[k] = v;
            carry = __shfl_sync(0xffffffffu, v, 31);
        }
    }
}

// A role's way through the CTA's items, round by round: forth and back over the
// CTAs, in ascending numbers.  SPLIT: the CTAs of a cluster go the same way,
// each with a part of every item's query tiles.
template <bool SPLIT>
struct Items {
    const ScoreParams &P;
    const STable &T;
    unsigned total;
    int range = 0;  // of the last item taken from the table
    __device__ __forceinline__ Items(const ScoreParams &params, const STable &table)
        : P(params), T(table), total(params.table ? table.first[params.ranges] : params.num_items) {}
    __device__ __forceinline__ unsigned id(unsigned r) const {
        const unsigned ways = SPLIT ? gridDim.x >> P.lg_parts : gridDim.x;
        const unsigned way = SPLIT ? blockIdx.x >> P.lg_parts : blockIdx.x;
        return r * ways + ((r & 1u) ? ways - 1u - way : way);
    }
    __device__ __forceinline__ bool has(unsigned r) const { return id(r) < total; }
    // the item of round r (rounds in ascending order; the whole warp)
    __device__ __forceinline__ SItem get(unsigned r) {
        SItem it;
        const unsigned i = id(r), Hkv = (unsigned)P.num_kv_heads;
        if (P.table) {
            for (int n = 32; n == 32;) {  // on by the ranges that end at or before i
                const int k = range + 1 + (int)(threadIdx.x & 31);
                n = __popc(__ballot_sync(0xffffffffu, k <= P.ranges && T.first[k] <= i));
                range += n;
            }
            const unsigned rest = i - T.first[range], place = small_div(rest, Hkv, P.kv_inv);
            it.s = T.order[place];
            it.hk = (int)(rest - place * Hkv);
            it.tok0 = T.tok0[it.s];
            it.n = T.n[it.s];
            it.L = T.L[it.s];
            it.ok = true;
        } else {
            const unsigned per = (unsigned)P.num_seqs * Hkv;
            range = (int)(i / per);
            const unsigned rest = i - (unsigned)range * per;
            it.s = (int)(rest / Hkv);
            it.hk = (int)(rest - (unsigned)it.s * Hkv);
            const int a = __ldg(&P.query_start_loc[it.s]), b = __ldg(&P.query_start_loc[it.s + 1]);
            it.L = __ldg(&P.context_lens[it.s]);
            it.n = b - a;
            it.tok0 = a;
            it.ok = lengths_ok(P, a, b, it.L);
        }
        it.c = it.L - it.n;
        it.k0 = range * kItemKeys;
        it.any = it.run = it.ok && it.n > 0 && it.k0 < it.L;
        it.tt0 = max(0, it.k0 - it.c) >> P.lg_nq;
        it.tt1 = (it.n + (1 << P.lg_nq) - 1) >> P.lg_nq;
        if (SPLIT) {
            const int tiles = it.tt1 - it.tt0, part = (int)blockIdx.x & ((1 << P.lg_parts) - 1);
            it.tt1 = it.tt0 + ((tiles * (part + 1)) >> P.lg_parts);
            it.tt0 += (tiles * part) >> P.lg_parts;
            it.run = it.run && it.tt0 < it.tt1;
        }
        return it;
    }
};

// First token tile that key tile t has a product with (the tile that holds the
// first token to see the tile's first key); tt1 if there is none.
template <bool SPLIT>
__device__ __forceinline__ int first_tile(const ScoreParams &P, const SItem &it, int t) {
    const int key = it.k0 + t * kKeys;
    const int tile = key < it.L ? max(0, key - it.c) >> P.lg_nq : it.tt1;
    return SPLIT ? min(max(tile, it.tt0), it.tt1) : tile;
}

// ---------------------------------------------------------------------------
// warp 0: K copies
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
__device__ __forceinline__ void run_score_producer(const ScoreParams &P, Items<SPLIT> items, unsigned char *sk,
                                                   const SBars &B, volatile int *abort_flag, int lane) {
    constexpr int KB = D / 64;
    constexpr uint32_t ktile = KB * kKSlice;
    const int lg_tbr = min(P.block_shift, 6);  // a copy: one block's share, 8 .. 64 keys
    const int units = kItemKeys >> lg_tbr;     // of an item, 4 .. 32: a lane each
    const uint64_t policy = l2_evict_first_policy();
    // this lane's unit of an item: the block it lies in, -1 past the last key
    auto entry = [&](const SItem &it) {
        const int tok = it.k0 + (lane << lg_tbr);
        return it.run && lane < units && tok < it.L
                   ? __ldg(&P.block_tables[(size_t)it.s * P.max_blocks_per_seq + (tok >> P.block_shift)])
                   : -1;
    };
    Ring kr;
    int kn = 0;  // slots armed so far
    bool ok = true;
    SItem it, nx;
    int e = -1, en = -1;
    auto ahead = [&](unsigned r) {
        if (!items.has(r)) return;
        nx = items.get(r);
        en = entry(nx);
    };
    ahead(0);
    for (unsigned r = 0; ok && items.has(r); ++r) {
        it = nx;
        e = en;
        if (!it.ok && it.k0 == 0 && it.hk == 0 && lane == 0 && P.err)
            atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
        if (!it.run) {
            ahead(r + 1);
            continue;
        }
        const int tok = it.k0 + (lane << lg_tbr);
        const int row = lane << lg_tbr;  // of the item's 256
        const bool use = lane < units && tok < it.L;
        const bool bad = use && (e < 0 || e >= P.num_blocks);
        const unsigned good = __ballot_sync(0xffffffffu, use && !bad);
        if (__any_sync(0xffffffffu, bad) && lane == 0 && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
        // lanes whose units belong to key tile 0
        const unsigned low = units >= 32 ? 0xffffu : (1u << (units / 2)) - 1u;
        auto load_k = [&](int t) {
            if (lane == 0) ok = mbar_wait(&B.k_free[kr.slot], kr.phase ^ 1u, abort_flag);
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            if (!ok) return;
            if (lane == 0)
                mbar_arrive_expect_tx(&B.k_full[kr.slot],
                                      ((uint32_t)__popc(good & (t ? ~low : low)) << lg_tbr) * 128u * KB);
            __syncwarp();
            if (use && !bad && (row >> 7) == t) {
                const int y = ((e * P.num_kv_heads + it.hk) << P.block_shift) +
                              (tok & ((1 << P.block_shift) - 1));
                tma_load_4d(sk + (size_t)kr.slot * ktile + (size_t)(row & 127) * (128 * KB),
                            &P.tmap_k, 0, 0, 0, y >> 3, &B.k_full[kr.slot], policy);
            }
            __syncwarp();
            kr.next(P.rk);
            ++kn;
        };
        load_k(0);
        ahead(r + 1);  // its table entries arrive during the second tile's copies
        if (ok && first_tile<SPLIT>(P, it, 1) < it.tt1) load_k(1);
    }
    if (lane == 0) {
        if (!ok) {
            *abort_flag = 1;
            if (P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
        }
        // every copy issued lands before the CTA can exit: the last phase armed
        // of every slot
        volatile int never = 0;
        for (int i = max(0, kn - P.rk); i < kn; ++i)
            mbar_drain_wait(&B.k_full[i % P.rk], (uint32_t)(i / P.rk) & 1u, &never);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// warps 1 and 2: S = K Q^T for key tile t.  The whole warp goes through the
// waits and one elected lane issues: an issuer's own instructions, each behind
// the one before, take longer than the products if they are many, and values
// that are the same in the warp stay in uniform registers, where the products
// want their descriptors.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

template <int D, bool SPLIT>
__device__ __forceinline__ void run_score_mma(const ScoreParams &P, Items<SPLIT> items, int t, uint32_t fmt,
                                              unsigned char *sk, unsigned char *sq, uint32_t tmem,
                                              const SBars &B, volatile int *abort_flag) {
    constexpr int KB = D / 64;
    constexpr uint32_t ktile = KB * kKSlice;
    const uint32_t cols = (uint32_t)P.nh << P.lg_nq;
    const uint32_t idesc = umma_idesc_f16(fmt, 0, 0, kKeys, cols);
    const uint32_t q_bytes = cols * 128u * KB;
    const uint64_t dk0 = umma_desc_sw128(smem_u32(sk), 16, 1024 * KB);
    const uint64_t dq0 = umma_desc_sw128(smem_u32(sq), 16, 1024);
    const uint32_t q_slice16 = cols * 128u / 16u;  // (head_dim 128: one further slice)
    Ring kr, qr, sr;
    bool ok = true;
    // a whole warp's wait
    auto wait = [&](uint64_t *bar, uint32_t phase) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar, phase, abort_flag));
        return ok;
    };
    // Both issuers pass through every K tile and every query tile in order, and
    // give back at once what is the other's alone: a wait by parity must never
    // be a whole ring ahead or behind.  (Copies land in any order, so that an
    // issuer's own tile is there says nothing about the one before it.)
    auto pass_k = [&]() {  // the other issuer's key tile
        if (!wait(&B.k_full[kr.slot], kr.phase)) return false;
        if (elect_one()) mbar_arrive(&B.k_free[kr.slot]);
        __syncwarp();
        kr.next(P.rk);
        return true;
    };
    unsigned r = 0;
    auto next_item = [&]() {  // the next item with work, from round r on; not run: none left
        SItem it;
        it.run = false;
        while (items.has(r)) {
            it = items.get(r++);
            if (it.run) break;
        }
        return it;
    };
    SItem nx = next_item();
    while (ok && nx.run) {
        const SItem it = nx;
        const bool two = first_tile<SPLIT>(P, it, 1) < it.tt1;
        if (t == 1 && !pass_k()) break;
        const int first = first_tile<SPLIT>(P, it, t);
        int n = (first - it.tt0) * P.head_groups;  // query tiles without a product here
        for (; n > 0; --n) {
            if (!wait(&B.q_full[qr.slot], qr.phase) || !wait(&B.l_full[qr.slot], qr.phase)) break;
            if (elect_one()) {
                mbar_arrive(&B.q_free[qr.slot]);
                for (int i = 0; i < 4; ++i) mbar_arrive(&B.l_free[qr.slot]);
            }
            qr.next(P.rq);
        }
        const int total = (it.tt1 - first) * P.head_groups;
        n = total;
        if (!ok || n == 0) {
            nx = next_item();
            continue;
        }
        if (!wait(&B.k_full[kr.slot], kr.phase)) break;
        const uint32_t dk = uniform((uint32_t)dk0 + (uint32_t)kr.slot * (ktile / 16u));
        for (; n > 0; --n) {
            if (!wait(&B.q_full[qr.slot], qr.phase)) break;
            if (!wait(&B.s_free[2 * t + sr.slot], sr.phase ^ 1u)) break;
            tc_fence_after();
            const uint32_t dq = uniform((uint32_t)dq0 + (uint32_t)qr.slot * (q_bytes / 16u));
            const uint32_t ts = uniform(tmem + (uint32_t)(128 * (2 * t + sr.slot)));
            if (elect_one()) {
                // a step of 16 elements is 32 bytes inside a slice; the offsets
                // (16-byte units) never carry out of the address field
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_f16(ts,
                             (dk0 & 0xffffffff00000000ull) |
                                 (dk + (uint32_t)((kk >> 2) * (1024 / 16) + (kk & 3) * 2)),
                             (dq0 & 0xffffffff00000000ull) |
                                 (dq + (uint32_t)((kk & 3) * 2) + ((kk >> 2) ? q_slice16 : 0u)),
                             idesc, kk > 0 ? 1u : 0u);
                umma_commit(&B.s_full[2 * t + sr.slot]);
                umma_commit(&B.q_free[qr.slot]);
                if (n == 1) umma_commit(&B.k_free[kr.slot]);
            }
            __syncwarp();
            if (n == 1) nx = next_item();  // while the products run
            sr.next(2);
            qr.next(P.rq);
        }
        if (!ok) break;
        kr.next(P.rk);
        if (t == 0 && two && !pass_k()) break;
    }
    if (!ok) {
        *abort_flag = 1;
        if (P.err && elect_one()) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
    }
    // after every product issued (by the same lane): the teardown
    if (elect_one()) umma_commit(&B.done[t]);
    __syncwarp();
}

// ---------------------------------------------------------------------------
// warp 3: query copies and the rows' lse
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
__device__ __forceinline__ void run_score_rows(const ScoreParams &P, Items<SPLIT> items,
                                              unsigned char *sq, float *s_lse,
                                              volatile int *s_dead, const SBars &B,
                                              volatile int *abort_flag, int lane) {
    const int cols = P.nh << P.lg_nq;
    const uint32_t q_bytes = (uint32_t)cols * (2u * D);
    constexpr int kPer = kMaxCols / 32;
    Ring lr;
    int qn = 0;  // query slots armed so far
    bool ok = true;
    // the next query tile, whose lse is on its way
    unsigned r = 0;
    SItem it;
    int tt = 0, hg = 0;
    auto next_item = [&]() {  // the first item with work from round r on
        for (; items.has(r); ++r) {
            it = items.get(r);
            if (it.run) {
                tt = it.tt0;
                hg = 0;
                return true;
            }
        }
        return false;
    };
    float l[kPer];
    int tok[kPer], head[kPer];  // of this lane's rows in a tile
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        tok[k] = (32 * k + lane) / P.nh;
        head[k] = 32 * k + lane - tok[k] * P.nh;
    }
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = (tt << P.lg_nq) + tok[k];
            l[k] = -INFINITY;  // no such row, or one without a weight
            if (32 * k + lane < cols && i < it.n)
                l[k] = __ldg(&P.lse[(size_t)(it.tok0 + i) * P.num_heads + it.hk * P.G + hg * P.nh +
                                    head[k]]);
        }
    };
    Ring qr;
    auto copy = [&]() {  // the tile's rows; false if the wait for its slot gave up
        if (lane == 0) {
            ok = mbar_wait(&B.q_free[qr.slot], qr.phase ^ 1u, abort_flag);
            if (ok) {
                mbar_arrive_expect_tx(&B.q_full[qr.slot], q_bytes);
                asm volatile(
                    "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                    " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                        smem_u32(sq + (size_t)qr.slot * q_bytes)),
                    "l"(&P.tmap_q), "r"(0), "r"(it.hk * P.G + hg * P.nh),
                    "r"(it.tok0 + (tt << P.lg_nq)), "r"(0), "r"(smem_u32(&B.q_full[qr.slot]))
                    : "memory");
                ++qn;
            }
        }
        qr.next(P.rq);
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        return ok;
    };
    // a tile's rows are on their way before the slot of the tile before it has
    // its lse (that slot's sums may still be at work)
    bool live = next_item();
    if (live) {
        load();
        copy();
    }
    while (live && ok) {
        float v[kPer];
        bool any_dead = false;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            v[k] = l[k] == -INFINITY ? -INFINITY : -l[k] * 1.4426950408889634f;
            any_dead |= 32 * k + lane < cols && l[k] == -INFINITY;
        }
        any_dead = __any_sync(0xffffffffu, any_dead);
        if (++hg == P.head_groups) {
            hg = 0;
            if (++tt == it.tt1) {
                ++r;
                live = next_item();
            }
        }
        if (live) {
            load();
            if (!copy()) break;
        }
        if (lane == 0) ok = mbar_wait(&B.l_free[lr.slot], lr.phase ^ 1u, abort_flag);
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < kPer; ++k) s_lse[lr.slot * kMaxCols + 32 * k + lane] = v[k];
        if (lane == 0) s_dead[lr.slot] = any_dead;
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.l_full[lr.slot]);
        lr.next(P.rq);
    }
    if (lane == 0) {
        if (!ok) {
            *abort_flag = 1;
            if (P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
        }
        // every copy issued lands before the CTA can exit: the last phase armed
        // of every slot
        volatile int never = 0;
        for (int i = max(0, qn - P.rq); i < qn; ++i)
            mbar_drain_wait(&B.q_full[i % P.rq], (uint32_t)(i / P.rq) & 1u, &never);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// warps 4..19: weights and sums of group (t, b), one key a thread
// ---------------------------------------------------------------------------
// Two fp32 values in a 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// One product of this thread's key: the weights of `cols` columns of tensor
// memory (a multiple of CH) in four chains of pairs.  CH columns at a time are
// loaded into registers, and the buffer is given back through `bar` with the
// last load, so the next product runs while their weights are worked out.  (2
// prompts of 4096 tokens with 32 heads on 8, 64 windows of 16 queries on 2048
// tokens: 120 and 52 us with 32 columns, 130 and 52 with 16; with the last 48
// at once, so that the buffer is free earlier, 121 and 97: more code.)  ALL:
// every column is visible; else those in [lo, hi) whose row has a weight at all
// (a row without has nl = -inf).  nl: the rows' negated lse.
template <bool ALL, int CH>
__device__ __forceinline__ float sum_product(uint32_t taddr, int cols, const float *nl, int lo,
                                             int hi, uint64_t sc2, uint64_t *bar) {
    uint64_t a[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
    for (int c = 0; c < cols; c += CH) {
        uint32_t u[CH];
#pragma unroll
        for (int i = 0; i < CH; i += 16)
            tmem_ld16(taddr + (uint32_t)(c + i), *reinterpret_cast<uint32_t(*)[16]>(&u[i]));
        tmem_wait_ld();
        if (c + CH >= cols) {
            tc_fence_before();
            mbar_arrive(bar);
        }
#pragma unroll
        for (int i = 0; i < CH; i += 4) {
            const float4 l4 = *reinterpret_cast<const float4 *>(nl + c + i);
            const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const float2 x =
                    unpair(fma2(pair(__uint_as_float(u[i + k]), __uint_as_float(u[i + k + 1])),
                                sc2, pair(l[k], l[k + 1])));
                float p0 = ex2(x.x), p1 = ex2(x.y);
                if (!ALL) {
                    const int col = c + i + k;
                    if (col < lo || col >= hi || l[k] == -INFINITY) p0 = 0.f;
                    if (col + 1 < lo || col + 1 >= hi || l[k + 1] == -INFINITY) p1 = 0.f;
                }
                a[(i + k) / 2 % 4] = add2(a[(i + k) / 2 % 4], pair(p0, p1));
            }
        }
    }
    const float2 v = unpair(add2(add2(a[0], a[1]), add2(a[2], a[3])));
    return v.x + v.y;
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Another CTA of the cluster's copy of a place in shared memory; a store to one,
// an arrival at one, and the wait for such arrivals.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster(float *p, uint32_t rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint64_t *bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     cluster_addr(bar, rank))
                 : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (!mbar_wait(bar, parity, abort)) return false;
    uint32_t done;  // (the phase has completed: seen once more, for the cluster's order)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0u;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

template <bool SPLIT>
__device__ __forceinline__ void run_score_sums(const ScoreParams &P, Items<SPLIT> items, int t, int b,
                                               const float *s_lse, const volatile int *s_dead,
                                               float *s_part, float *comb, uint32_t tmem,
                                               const SBars &B, volatile int *abort_flag, int wq,
                                               int lane) {
    const int rk = 32 * wq + lane;  // this thread's key of the tile
    const int cols = P.nh << P.lg_nq;
    const uint32_t tb = tmem + (uint32_t)(128 * (2 * t + b)) + ((uint32_t)(32 * wq) << 16);
    float *part = s_part + t * kKeys;
    const int bar_full = 1 + t, bar_free = 3 + t;
    const uint64_t sc2 = pair(P.scale_log2, P.scale_log2);
    // the next item with keys for this tile, from round r on; `skipped`: query
    // tiles of the items before it that have none
    auto next_item = [&](unsigned &r, SItem &it, int &skipped) {
        for (; items.has(r); ++r) {
            it = items.get(r);
            if (!it.any) continue;  // (a part without a product hands over zeros)
            if (it.k0 + t * kKeys < it.L) return true;
            skipped += (it.tt1 - it.tt0) * P.head_groups;
        }
        return false;
    };
    unsigned r = 0;
    SItem nx;
    int q0 = 0;           // query tiles before the item
    bool live = next_item(r, nx, q0);
    int cnt = 0;          // products of the key tile before the item
    int taken = 0;        // products of this group
    bool gave = false;    // group (t, 1): sums handed over and not yet taken
    const unsigned part_id = SPLIT ? blockIdx.x & ((1u << P.lg_parts) - 1u) : 0u;
    unsigned shared = 0u;  // items put together in the cluster
    bool ok = true;
    float old = 0.f;      // the key's score before (group (t, 0))
    int blk = -1;         // and its block
    auto prefetch = [&]() {  // of item nx
        const int key = nx.k0 + t * kKeys + rk;
        if (b == 0 && part_id == 0u && key < nx.L) {
            blk = __ldg(&P.block_tables[(size_t)nx.s * P.max_blocks_per_seq + (key >> P.block_shift)]);
            old = P.scores[((long long)nx.s * P.num_kv_heads + nx.hk) * P.score_stride + key];
        }
    };
    if (live) prefetch();
    while (live) {
        const SItem it = nx;
        const int first = first_tile<SPLIT>(P, it, t), np = (it.tt1 - first) * P.head_groups;
        const int key = it.k0 + t * kKeys + rk;
        const float old_now = old;
        const int blk_now = blk;
        const int qp = q0 + (first - it.tt0) * P.head_groups;  // query tile of product 0
        q0 += (it.tt1 - it.tt0) * P.head_groups;
        float acc = 0.f;
        int tt = first, hg = 0, p = (cnt ^ b) & 1;
        auto step = [&](int by) {
            for (hg += by; hg >= P.head_groups; hg -= P.head_groups) ++tt;
        };
        step(p);
        cnt += np;
        // the ring's slot of its query tile
        const unsigned turn = small_div((unsigned)(qp + p), (unsigned)P.rq, P.rq_inv);
        int slot = qp + p - (int)turn * P.rq;
        uint32_t phase = turn & 1u;
        auto slot_step = [&]() {
            slot += 2;
            if (slot >= P.rq) {
                slot -= P.rq;
                phase ^= 1u;
            }
        };
        const int p_first = p;
        for (; ok && p < np; p += 2, step(2), slot_step()) {
            // The lse is there by now or soon; waiting for it first hides that
            // wait behind the product's.  That its slot's phase before has
            // completed is known where this group has read the tile before
            // last; at the start of key tile 1's part of an item it is known
            // with the product, whose issuer has seen the last tile staged.
            const bool late = t == 1 && p == p_first;
            if (!late) ok = mbar_wait(&B.l_full[slot], phase, abort_flag);
            ok = ok && mbar_wait(&B.s_full[2 * t + b], (uint32_t)taken & 1u, abort_flag);
            if (late) ok = ok && mbar_wait(&B.l_full[slot], phase, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {  // at once: no sum that lacks this product is written or sent
                *abort_flag = 1;
                break;
            }
            ++taken;
            tc_fence_after();
            const float *nl = s_lse + slot * kMaxCols;
            const int tok = tt << P.lg_nq;  // the tile's first token
            const int lo = max(0, key - it.c - tok) * P.nh;
            const int hi = (it.n - tok) * P.nh;
            const bool all = __all_sync(0xffffffffu, lo == 0) && hi >= cols && !s_dead[slot];
            acc += all ? sum_product<true, kChunk>(tb, cols, nl, lo, hi, sc2, &B.s_free[2 * t + b])
                       : sum_product<false, kChunk>(tb, cols, nl, lo, hi, sc2, &B.s_free[2 * t + b]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.l_free[slot]);
        }
        // the item's sums
        if (b == 1) {
            if (gave) bar_sync(bar_free, 256);
            part[rk] = acc;
            bar_arrive(bar_full, 256);
            gave = true;
        } else {
            bar_sync(bar_full, 256);
            acc += part[rk];
            bar_arrive(bar_free, 256);
            // (group (t, 1) sets the flag before it hands over a sum that lacks a
            // product: such a sum is neither written nor sent on)
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (SPLIT && part_id) {  // to the cluster's first CTA
                if (shared) ok = ok && wait_cluster(&B.c_free[t], (shared - 1u) & 1u, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    st_cluster(comb + (part_id - 1u) * kItemKeys + t * kKeys + rk, 0u, acc);
                    __syncwarp();
                    if (lane == 0) arrive_cluster(&B.c_full[t], 0u);
                }
                ++shared;
            } else if (SPLIT) {
                ok = ok && wait_cluster(&B.c_full[t], shared & 1u, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    const unsigned parts = 1u << P.lg_parts;
                    for (unsigned i = 0; i + 1u < parts; ++i) acc += comb[i * kItemKeys + t * kKeys + rk];
                    __syncwarp();
                    if (lane > 0 && lane < (int)parts) arrive_cluster(&B.c_free[t], (uint32_t)lane);
                }
                ++shared;
            }
            if (part_id == 0u && ok && key < it.L && blk_now >= 0 &&
                blk_now < P.num_blocks)
                P.scores[((long long)it.s * P.num_kv_heads + it.hk) * P.score_stride + key] =
                    old_now + acc;
        }
        ++r;
        live = next_item(r, nx, q0);
        if (live) prefetch();
    }
    if (!ok) {
        *abort_flag = 1;
        if (lane == 0 && P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
    }
}

// SPLIT: the CTAs of a cluster share one item.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreadsS, 1)
    prefill_scores_kernel(const __grid_constant__ ScoreParams P, uint32_t fmt) {
    using L = SLayout;
    extern __shared__ __align__(1024) unsigned char smem[];
    // the swizzled tiles need 1024-byte alignment, which the start of dynamic
    // shared memory has
    if (smem_u32(smem) & 1023u) {
        pdl_wait();
        if (threadIdx.x == 0 && P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
        return;
    }
    float *s_lse = reinterpret_cast<float *>(smem);
    volatile int *s_dead = reinterpret_cast<volatile int *>(smem + L::dead_off);
    float *s_part = reinterpret_cast<float *>(smem + L::part_off);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bar_off);
    unsigned char *sk = smem + L::small, *sq = sk + (size_t)P.rk * (D / 64) * kKSlice;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::tmem_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::flag_off);
    SBars B;
    B.k_full = bars;
    B.k_free = B.k_full + kMaxRing;
    B.q_full = B.k_free + kMaxRing;
    B.q_free = B.q_full + kMaxRing;
    B.l_full = B.q_free + kMaxRing;
    B.l_free = B.l_full + kMaxRing;
    B.s_full = B.l_free + kMaxRing;
    B.s_free = B.s_full + 4;
    B.done = B.s_free + 4;
    B.c_full = B.done + 2;
    B.c_free = B.c_full + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&P.tmap_q);
        prefetch_tmap(&P.tmap_k);
        for (int b = 0; b < L::kBars; ++b) mbar_init(&bars[b], 1);
        for (int b = 0; b < 4; ++b) mbar_init(&B.s_free[b], kKeys);
        // a slot is given back by both issuers (or by the completion of their
        // products), the lse by the four warps of each key tile's group
        for (int b = 0; b < kMaxRing; ++b) {
            mbar_init(&B.k_free[b], 2);
            mbar_init(&B.q_free[b], 2);
            mbar_init(&B.l_free[b], 8);
        }
        for (int t = 0; SPLIT && t < kTiles; ++t) {  // (a warp arrives once)
            mbar_init(&B.c_full[t], 4u * ((1u << P.lg_parts) - 1u));
            mbar_init(&B.c_free[t], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemColsS);
    STable &table = *reinterpret_cast<STable *>(smem + L::table_off);
    float *comb = reinterpret_cast<float *>(smem + L::comb_off);
    if (P.table) number_items(P, table);  // (from the lengths alone: before the wait)
    tc_fence_before();
    __syncthreads();
    if (SPLIT) cluster_sync();  // every CTA has started, its barriers set up
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();     // the kernels before may still write what this reads
    pdl_trigger();  // (after the wait: what follows may start before this grid ends, not before those)
    const Items<SPLIT> items(P, table);
    // each role's code follows its own register reallocation (code after a
    // join of the two would be held to the smaller count)
    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
        run_score_sums<SPLIT>(P, items, (warp - 4) >> 3, ((warp - 4) >> 2) & 1, s_lse, s_dead, s_part,
                              comb, tmem, B, abort_flag, warp & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 0) {
            run_score_producer<D, SPLIT>(P, items, sk, B, abort_flag, lane);
        } else if (warp <= 2) {
            run_score_mma<D, SPLIT>(P, items, warp - 1, fmt, sk, sq, tmem, B, abort_flag);
            // every product has completed before tensor memory is released
            volatile int never = 0;
            mbar_drain_wait(&B.done[warp - 1], 0, &never);
            __syncwarp();
        } else {
            run_score_rows<D, SPLIT>(P, items, sq, s_lse, s_dead, B, abort_flag, lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemColsS);
    if (SPLIT) cluster_sync();  // no CTA leaves while another may still write to it
}

constexpr int kMaxLgParts = 3;
static_assert(1 << kMaxLgParts == kMaxParts, "parts of an item");

// A launch of either form; lg: log2 of the CTAs of a cluster.
struct ScoreLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    ScoreLaunch(unsigned grid, int lg, cudaStream_t stream) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kThreadsS);
        cfg.dynamicSmemBytes = SLayout::bytes;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1u << lg;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = lg ? 2 : 1;
    }
};

template <int D, bool SPLIT>
pa_status_t set_up_scores() {
    // the register reallocation inside the kernel assumes exactly kRegsLaunch
    // registers a thread at launch; anything else is refused
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, prefill_scores_kernel<D, SPLIT>) != cudaSuccess) return PA_ERR_CUDA;
    if (fa.numRegs != kRegsLaunch) return PA_ERR_UNSUPPORTED;
    return cudaFuncSetAttribute(prefill_scores_kernel<D, SPLIT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)SLayout::bytes) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

// tiles: token tiles of the longest sequence of queries.
template <int D>
pa_status_t launch_scores(ScoreParams &P, uint32_t fmt, int tiles, int sms, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> ready[kMaxDevices];
    static std::atomic<int> clusters[kMaxDevices][kMaxLgParts + 1];  // that run at once
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PA_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        pa_status_t e = set_up_scores<D, false>();
        if (e == PA_OK) e = set_up_scores<D, true>();
        if (e != PA_OK) return e;
        for (int lg = 1; lg <= kMaxLgParts; ++lg) {
            const ScoreLaunch one(1u << lg, lg, stream);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, prefill_scores_kernel<D, true>, &one.cfg) != cudaSuccess)
                return PA_ERR_CUDA;
            clusters[dev][lg].store(n, std::memory_order_relaxed);
        }
        ready[dev].store(true, std::memory_order_release);
    }
    // Few items are shared, while the GPU then has at most two parts a CTA and a
    // part two token tiles of the longest.  (One prompt of 4096 tokens, 32 heads
    // on 8: 67 us; with up to four parts a CTA 76, without clusters 119.  Two
    // prompts: 118 without clusters, 125 with.)
    P.lg_parts = 0;
    for (int lg = 1; lg <= kMaxLgParts; ++lg)
        if (tiles >= 2 << lg && (unsigned long long)P.num_items << lg <= 2ull * (unsigned)sms &&
            clusters[dev][lg].load(std::memory_order_relaxed) > 0)
            P.lg_parts = lg;
    const unsigned ways = P.lg_parts ? (unsigned)clusters[dev][P.lg_parts].load(std::memory_order_relaxed)
                                     : (unsigned)sms;
    const ScoreLaunch l((P.num_items < ways ? P.num_items : ways) << P.lg_parts, P.lg_parts, stream);
    const cudaError_t e = P.lg_parts ? cudaLaunchKernelEx(&l.cfg, prefill_scores_kernel<D, true>, P, fmt)
                                     : cudaLaunchKernelEx(&l.cfg, prefill_scores_kernel<D, false>, P, fmt);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_prefill_scores_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                                   int head_dim, int max_query_len,
                                                   int max_context_len) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128) || max_query_len < 0 || max_context_len < 0)
        return 0;
    return 256;
}

extern "C" pa_status_t pa_prefill_scores(
    const void *query, const float *lse, const void *k_cache, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *query_start_loc, const int32_t *context_lens,
    int max_query_len, int max_context_len, int num_seqs, int num_tokens, int num_heads,
    int num_kv_heads, int head_dim, int num_blocks, int block_size, float scale, pa_dtype_t dtype,
    float *scores, int64_t score_stride, void *workspace, size_t workspace_bytes,
    unsigned int *dev_error_word, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_prefill_scores");
    const int shift = pool_block_shift(block_size);
    if (shift < 0) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        max_query_len < 0 || max_context_len < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0 || !is_16bit(dtype)) return PA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)block_size * max_blocks_per_seq ||
        score_stride < max_context_len)
        return PA_ERR_INVALID_ARG;
    const unsigned long long pool_rows = (unsigned long long)num_blocks * num_kv_heads * block_size;
    if (pool_rows >= (1ull << 31) || (long long)num_tokens * num_heads >= (1ll << 31) ||
        num_kv_heads > 65535 || num_seqs > 65535)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0 || max_context_len == 0) return PA_OK;
    const bool no_workspace = !workspace && workspace_bytes == 0;  // (the kernel needs none)
    if (!query || !lse || !k_cache || !block_tables || !query_start_loc || !context_lens || !scores ||
        (!workspace && !no_workspace))
        return PA_ERR_INVALID_ARG;
    if (!is_aligned(query, 16) || !is_aligned(k_cache, 16) || !is_aligned(lse, 4) ||
        !is_aligned(scores, 4))
        return PA_ERR_INVALID_ARG;
    if (!no_workspace &&
        (!is_aligned(workspace, 256) ||
         workspace_bytes < pa_prefill_scores_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                            head_dim, max_query_len, max_context_len)))
        return PA_ERR_WORKSPACE;
    const int sms = device_sms();
    if (sms <= 0) return PA_ERR_CUDA;
    ScoreParams P;
    std::memset(&P, 0, sizeof(P));
    const int G = num_heads / num_kv_heads;
    // A query tile: NH heads, a divisor of the group, and NQ tokens, a power of
    // two; 32 to 128 rows in steps of 32, a thread's loads.  The fewest columns
    // for the longest sequence of queries, a tile's fixed cost counted as 32
    // (8 windows of 32 queries, 12 heads on 2: 18.6 us with two tiles of 16
    // tokens by 6 heads, 20.2 with three of 32 by 2).
    long long best = -1;
    for (int nh = G < kMaxCols ? G : kMaxCols; nh >= 1; --nh) {
        if (G % nh) continue;
        for (int lg = 7; lg >= 0; --lg) {
            const int cols = nh << lg;
            if (cols > kMaxCols || cols % kChunk) continue;
            const long long cost = ((max_query_len + (1ll << lg) - 1) >> lg) * (G / nh) * (cols + 32);
            if (best >= 0 && cost >= best) continue;
            best = cost;
            P.nh = nh;
            P.lg_nq = lg;
        }
    }
    P.head_groups = G / P.nh;
    // The rings (counted at head_dim 128; 64 has twice the slots): three K tiles and
    // what is left in query tiles, three of 128 rows, four of 96; four K tiles where
    // a query tile has at most 64 rows, which leaves four of those and more.  (96
    // rows with four K tiles and two query tiles: 14.6 us for 8 windows of 32
    // queries, 12 heads on 2, and 20.4 for 8 of 40, 24 heads on 2; 14.4 and 19.2
    // so.)  The waits for a tile's lse need two query slots at least.
    static_assert((kTileBytes - 3 * 32768) / 32768 >= 2 && (kTileBytes - 4 * 32768) / 16384 >= 2,
                  "query slots");
    const uint32_t kbytes = (uint32_t)head_dim * 256u, qbytes = (uint32_t)head_dim * 2u * P.nh << P.lg_nq;
    P.rk = 2 * qbytes <= kbytes ? 4 : 3;
    if (head_dim == 64) P.rk *= 2;
    P.rq = (int)((kTileBytes - (uint32_t)P.rk * kbytes) / qbytes);
    if (P.rq > kMaxRing) P.rq = kMaxRing;
    P.rq_inv = small_inverse((unsigned)P.rq);
    P.kv_inv = small_inverse((unsigned)num_kv_heads);
    const cuuint64_t KB = (cuuint64_t)head_dim / 64;
    {
        const cuuint64_t dims[4] = {64u, (cuuint64_t)num_heads, (cuuint64_t)num_tokens, KB};
        const cuuint64_t strides[3] = {(cuuint64_t)head_dim * 2,
                                       (cuuint64_t)num_heads * head_dim * 2, 128u};
        const cuuint32_t box[4] = {64u, (cuuint32_t)P.nh, 1u << P.lg_nq, (cuuint32_t)KB};
        if (!encode_tiled(&P.tmap_q, query, dtype, 4, dims, strides, box)) return PA_ERR_CUDA;
    }
    {
        const cuuint64_t dims[4] = {64u, 8u, KB, (cuuint64_t)pool_rows / 8};
        const cuuint64_t strides[3] = {(cuuint64_t)head_dim * 2, 128u, (cuuint64_t)head_dim * 16};
        const cuuint32_t box[4] = {64u, 8u, (cuuint32_t)KB, (cuuint32_t)(block_size < 64 ? block_size : 64) / 8};
        if (!encode_tiled(&P.tmap_k, k_cache, dtype, 4, dims, strides, box)) return PA_ERR_CUDA;
    }
    P.lse = lse;
    P.block_tables = block_tables;
    P.query_start_loc = query_start_loc;
    P.context_lens = context_lens;
    P.scores = scores;
    P.score_stride = score_stride;
    P.max_blocks_per_seq = max_blocks_per_seq;
    P.block_shift = shift;
    P.num_blocks = num_blocks;
    P.max_query_len = max_query_len;
    P.max_context_len = max_context_len;
    P.num_seqs = num_seqs;
    P.num_tokens = num_tokens;
    P.num_heads = num_heads;
    P.num_kv_heads = num_kv_heads;
    P.G = G;
    P.scale_log2 = scale * 1.4426950408889634f;
    P.err = dev_error_word;
    const unsigned long long items =
        (unsigned long long)((max_context_len + (long long)kItemKeys - 1) / kItemKeys) * num_seqs *
        num_kv_heads;
    if (items >= (1ull << 31)) return PA_ERR_UNSUPPORTED;
    P.num_items = (unsigned)items;
    P.ranges = (int)((max_context_len + (long long)kItemKeys - 1) / kItemKeys);
    P.table = num_seqs <= kMaxTableSeqs && P.ranges <= kMaxTableRanges ? 1 : 0;
    const int tiles = (int)((max_query_len + (1ll << P.lg_nq) - 1) >> P.lg_nq);
    const uint32_t fmt = dtype == PA_BF16 ? 1u : 0u;
    cudaStream_t st = (cudaStream_t)stream;
    return head_dim == 64 ? launch_scores<64>(P, fmt, tiles, sms, st)
                          : launch_scores<128>(P, fmt, tiles, sms, st);
}
