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
// query tile is up to 128 (token, head) rows: NH heads of the group (the
// largest power of two that divides it) times NQ tokens, one TMA box.  The
// kernel is persistent, one CTA per SM; items are numbered from the first keys
// on (with whole prompts those see the most queries) and dealt out forth and
// back, so every CTA's share is about as heavy and no list is needed.
// Twelve warps:
//   * warp 0 (producer): the item's K tiles into one of two K buffers, block
//     by block (tiled bulk copies, TMA), then its query tiles into a ring.  It
//     runs ahead into the next item;
//   * warp 1 (one thread): S_t = K_t Q^T (M = 128 keys, N = the tile's rows,
//     K = head_dim) for both key tiles into one of two tensor-memory buffers
//     each; causal: tiles whose rows all lie before the keys are left out;
//   * warp 2 allocates tensor memory, warp 3 is idle (the lanes a warp may
//     read go by its number modulo 4);
//   * warps 4..7 and 8..11 (key tile 0 and 1): one key a thread.  Each stages
//     the rows' lse (base 2) in shared memory, loads S from tensor memory
//     32 columns at a time, and sums 2^(x scale log2 e - lse) over the columns
//     it may see -- a range [lo, hi) of the tile, from its key's position.
// Sums are fp32 in two levels: the 32-column steps of a tile, then tiles.
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
constexpr int kMaxCols = 128; // rows of a query tile
constexpr int kThreadsS = 384;
constexpr uint32_t kTmemColsS = 512;  // S of tile t, buffer b at 128 (2 t + b)
constexpr uint32_t kKSlice = kKeys * 128;  // bytes of a 64-element slice of a K tile

struct ScoreParams {
    CUtensorMap tmap_q;  // query as [head_dim/64][tokens][heads][64], box NQ x NH rows
    CUtensorMap tmap_k;  // pool rows as [head_dim/64][rows][64], box min(block, 64) rows
    const float *lse;
    const int32_t *block_tables, *query_start_loc, *context_lens;
    float *scores;
    long long score_stride;
    int max_blocks_per_seq, block_shift, num_blocks;
    int max_query_len, max_context_len, num_seqs, num_tokens, num_heads, num_kv_heads, G;
    int lg_nh, lg_nq;     // heads and tokens of a query tile
    int head_groups;      // G / NH
    unsigned num_items;   // 256-key ranges x num_seqs x num_kv_heads
    float scale_log2;
    unsigned int *err;
};

template <int D>
struct SLayout {
    static constexpr int KB = D / 64;
    static constexpr int RQ = D == 64 ? 6 : 3;                       // query stages
    static constexpr size_t ktile = (size_t)KB * kKSlice;            // [slice][128 keys][64]
    static constexpr size_t kbuf = kTiles * ktile;
    static constexpr size_t qstage = (size_t)KB * kMaxCols * 128;    // [slice][rows][64]
    static constexpr size_t k_off = 0;
    static constexpr size_t q_off = 2 * kbuf;
    static constexpr size_t tiles = q_off + RQ * qstage;
    // before the tiles: lse [tile][2][128], its dead-row flags [tile][2][4], barriers
    static constexpr size_t dead_off = kTiles * 2 * kMaxCols * 4;
    static constexpr size_t bar_off = dead_off + kTiles * 2 * 4 * 4;
    // k_full[2], k_free[2], q_full[RQ], q_free[RQ], s_full[2][2], s_free[2][2],
    // staged[2], done
    static constexpr int kBars = 4 + 2 * RQ + 8 + 2 + 1;
    static constexpr size_t tmem_off = bar_off + 8 * kBars;
    static constexpr size_t flag_off = tmem_off + 4;
    static constexpr size_t small = (flag_off + 4 + 1023) / 1024 * 1024;
    static constexpr size_t bytes = small + tiles;
    static_assert(bytes <= 232448, "dynamic shared memory of one CTA");
};

struct SBars {
    uint64_t *k_full, *k_free, *q_full, *q_free, *s_full, *s_free, *staged, *done;
};

// One work item, worked out by every role for itself.
struct SItem {
    int s, hk;
    int n, L, c, tok0;  // new tokens, context length, cached before, first query row
    int k0;             // first key
    int tt0, tt1;       // token tiles that see some key of the item
    bool ok, run;
};

__device__ __forceinline__ SItem score_item(const ScoreParams &P, unsigned id) {
    SItem it;
    const unsigned per = (unsigned)P.num_seqs * (unsigned)P.num_kv_heads;
    const unsigned range = id / per, rest = id - range * per;
    it.s = (int)(rest / (unsigned)P.num_kv_heads);
    it.hk = (int)(rest - (unsigned)it.s * (unsigned)P.num_kv_heads);
    const int a = __ldg(&P.query_start_loc[it.s]), b = __ldg(&P.query_start_loc[it.s + 1]);
    it.L = __ldg(&P.context_lens[it.s]);
    it.n = b - a;
    it.tok0 = a;
    it.ok = a >= 0 && b <= P.num_tokens && it.n >= 0 && it.n <= P.max_query_len &&
            it.L >= it.n && it.L <= P.max_context_len;
    it.c = it.L - it.n;
    it.k0 = (int)range * kItemKeys;
    it.run = it.ok && it.n > 0 && it.k0 < it.L;
    it.tt0 = max(0, it.k0 - it.c) >> P.lg_nq;
    it.tt1 = (it.n + (1 << P.lg_nq) - 1) >> P.lg_nq;
    return it;
}

// Item of the CTA's round r: forth and back over the CTAs.
__device__ __forceinline__ unsigned item_id(unsigned r) {
    return r * gridDim.x + ((r & 1u) ? gridDim.x - 1u - blockIdx.x : blockIdx.x);
}

// Whether key tile t has a product with token tile tt: it has keys, and the
// tile's last token sees the first of them.
__device__ __forceinline__ bool tile_on(const ScoreParams &P, const SItem &it, int t, int tt) {
    const int key = it.k0 + t * kKeys;
    return key < it.L && it.c + min(it.n, (tt + 1) << P.lg_nq) - 1 >= key;
}

// ---------------------------------------------------------------------------
// warp 0: K and query copies
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void run_score_producer(const ScoreParams &P, unsigned char *sk,
                                                   unsigned char *sq, const SBars &B,
                                                   volatile int *abort_flag, int lane) {
    using L = SLayout<D>;
    constexpr int KB = L::KB, RQ = L::RQ;
    const int lg_tbr = min(P.block_shift, 6);  // a copy: one block's share, 8 .. 64 keys
    const int units = kItemKeys >> lg_tbr;     // 4 .. 32: a lane each
    const int cols = 1 << (P.lg_nh + P.lg_nq);
    const uint32_t q_bytes = (uint32_t)cols * 128u * KB;
    const uint64_t policy = l2_evict_first_policy();
    // this lane's unit of an item: the block it lies in, -1 past the last key
    auto entry = [&](const SItem &it) {
        const int tok = it.k0 + (lane << lg_tbr);
        return it.run && lane < units && tok < it.L
                   ? __ldg(&P.block_tables[(size_t)it.s * P.max_blocks_per_seq + (tok >> P.block_shift)])
                   : -1;
    };
    int kc = 0, qc = 0;  // K buffers and query stages armed
    bool ok = true;
    SItem it, nx;
    int e = -1, en = -1;
    if (item_id(0) < P.num_items) {
        nx = score_item(P, item_id(0));
        en = entry(nx);
    }
    for (unsigned r = 0; ok && item_id(r) < P.num_items; ++r) {
        it = nx;
        e = en;
        if (item_id(r + 1) < P.num_items) {  // its table entries arrive meanwhile
            nx = score_item(P, item_id(r + 1));
            en = entry(nx);
        }
        if (!it.ok && it.k0 == 0 && it.hk == 0 && lane == 0 && P.err)
            atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
        if (!it.run) continue;
        const int tok = it.k0 + (lane << lg_tbr);
        const bool use = lane < units && tok < it.L;
        const bool bad = use && (e < 0 || e >= P.num_blocks);
        const unsigned good = __ballot_sync(0xffffffffu, use && !bad);
        if (__any_sync(0xffffffffu, bad) && lane == 0 && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
        const int kb = kc & 1;
        if (lane == 0) ok = mbar_wait(&B.k_free[kb], (uint32_t)((kc >> 1) & 1) ^ 1u, abort_flag);
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok) break;
        if (lane == 0)
            mbar_arrive_expect_tx(&B.k_full[kb], ((uint32_t)__popc(good) << lg_tbr) * 128u * KB);
        __syncwarp();
        if (use && !bad) {
            const int row = lane << lg_tbr;  // of the item's 256
            unsigned char *dst = sk + (size_t)kb * L::kbuf + (size_t)(row >> 7) * L::ktile +
                                 (size_t)(row & 127) * 128;
            const int y = ((e * P.num_kv_heads + it.hk) << P.block_shift) +
                          (tok & ((1 << P.block_shift) - 1));
#pragma unroll
            for (int z = 0; z < KB; ++z)
                tma_load_3d(dst + (size_t)z * kKSlice, &P.tmap_k, 0, y, z, &B.k_full[kb], policy);
        }
        __syncwarp();
        ++kc;
        if (lane == 0) {
            for (int tt = it.tt0; ok && tt < it.tt1; ++tt)
                for (int hg = 0; hg < P.head_groups; ++hg) {
                    const int st = qc % RQ;
                    ok = mbar_wait(&B.q_free[st], (uint32_t)((qc / RQ) & 1) ^ 1u, abort_flag);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&B.q_full[st], q_bytes);
                    asm volatile(
                        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                            smem_u32(sq + (size_t)st * L::qstage)),
                        "l"(&P.tmap_q), "r"(0), "r"(it.hk * P.G + (hg << P.lg_nh)),
                        "r"(it.tok0 + (tt << P.lg_nq)), "r"(0), "r"(smem_u32(&B.q_full[st]))
                        : "memory");
                    ++qc;
                }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0) {
        if (!ok) {
            *abort_flag = 1;
            if (P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
        }
        // every copy issued lands before the CTA can exit
        volatile int never = 0;
        for (int i = max(0, kc - 2); i < kc; ++i)
            mbar_drain_wait(&B.k_full[i & 1], (uint32_t)(i >> 1) & 1u, &never);
        for (int i = max(0, qc - RQ); i < qc; ++i)
            mbar_drain_wait(&B.q_full[i % RQ], (uint32_t)(i / RQ) & 1u, &never);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// warp 1, one thread: S = K Q^T
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void run_score_mma(const ScoreParams &P, uint32_t fmt,
                                              unsigned char *sk, unsigned char *sq, uint32_t tmem,
                                              const SBars &B, volatile int *abort_flag) {
    using L = SLayout<D>;
    constexpr int RQ = L::RQ;
    const uint32_t cols = 1u << (P.lg_nh + P.lg_nq);
    const uint32_t idesc = umma_idesc_f16(fmt, 0, 0, kKeys, cols);
    const uint32_t ak = smem_u32(sk), aq = smem_u32(sq);
    int kc = 0, qc = 0, sc[kTiles] = {0, 0};
    bool ok = true;
    for (unsigned r = 0; ok && item_id(r) < P.num_items; ++r) {
        const SItem it = score_item(P, item_id(r));
        if (!it.run) continue;
        const int kb = kc & 1;
        ok = mbar_wait(&B.k_full[kb], (uint32_t)(kc >> 1) & 1u, abort_flag);
        for (int tt = it.tt0; ok && tt < it.tt1; ++tt)
            for (int hg = 0; ok && hg < P.head_groups; ++hg, ++qc) {
                const int st = qc % RQ;
                ok = mbar_wait(&B.q_full[st], (uint32_t)(qc / RQ) & 1u, abort_flag);
                if (!ok) break;
                const uint32_t qt = aq + (uint32_t)(st * L::qstage);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    if (!ok || !tile_on(P, it, t, tt)) continue;
                    const int b = sc[t] & 1;
                    ok = mbar_wait(&B.s_free[2 * t + b], (uint32_t)((sc[t] >> 1) & 1) ^ 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t kt = ak + (uint32_t)(kb * L::kbuf + t * L::ktile);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t in_slice = (uint32_t)((kk & 3) * 32);
                        umma_f16(tmem + (uint32_t)(128 * (2 * t + b)),
                                 umma_desc_sw128(kt + (uint32_t)(kk >> 2) * kKSlice + in_slice, 16, 1024),
                                 umma_desc_sw128(qt + (uint32_t)(kk >> 2) * cols * 128u + in_slice, 16, 1024),
                                 idesc, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&B.s_full[2 * t + b]);
                    ++sc[t];
                }
                umma_commit(&B.q_free[st]);
            }
        umma_commit(&B.k_free[kb]);
        ++kc;
    }
    if (!ok) {
        *abort_flag = 1;
        if (P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
    }
    umma_commit(B.done);  // after every product issued: the teardown
}

// ---------------------------------------------------------------------------
// warps 4..11: weights and sums, key tile t, one key a thread
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
    tmem_ld16(taddr + 16u, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
}

// 32 columns from column c on: the sum of the weights.  ALL: every column is
// visible; else those in [lo, hi) whose row has a weight at all (a row
// without has lse = +inf here).
template <bool ALL>
__device__ __forceinline__ float sum32(const uint32_t (&u)[32], const float *lse, int c, int lo,
                                       int hi, float sc) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 l4 = *reinterpret_cast<const float4 *>(lse + c + i);
        const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float p = ex2(fmaf(__uint_as_float(u[i + k]), sc, -l[k]));
            const int col = c + i + k;
            a[(i + k) % 8] += ALL || (col >= lo && col < hi && l[k] != INFINITY) ? p : 0.f;
        }
    }
    return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
}

__device__ __forceinline__ void run_score_sums(const ScoreParams &P, int t, float *s_lse,
                                               volatile int *s_dead, uint32_t tmem,
                                               const SBars &B, volatile int *abort_flag, int wq,
                                               int lane) {
    const int rk = 32 * wq + lane;  // this thread's key of the tile, and the row it stages
    const int cols = 1 << (P.lg_nh + P.lg_nq);
    const uint32_t tm = tmem + (uint32_t)(256 * t) + ((uint32_t)(32 * wq) << 16);
    // the stream of this tile's products: item round r, token tile tt, head group hg
    struct Pos {
        unsigned r;
        SItem it;
        int tt, hg;
        bool live;
    };
    auto settle = [&](Pos &p) {  // to the first product at or after (r, tt, hg)
        for (;;) {
            if (p.it.run) {
                while (p.tt < p.it.tt1 && !tile_on(P, p.it, t, p.tt)) ++p.tt;
                if (p.tt < p.it.tt1) return;
            }
            const unsigned id = item_id(++p.r);
            if (id >= P.num_items) {
                p.live = false;
                return;
            }
            p.it = score_item(P, id);
            p.tt = p.it.tt0;
            p.hg = 0;
        }
    };
    auto row_lse = [&](const Pos &p) {  // staged row's lse, base 2; +inf: no such row, or no weight
        const int i = (p.tt << P.lg_nq) + (rk >> P.lg_nh);
        if (!p.live || rk >= cols || i >= p.it.n) return INFINITY;
        const int h = p.it.hk * P.G + (p.hg << P.lg_nh) + (rk & ((1 << P.lg_nh) - 1));
        const float l = __ldg(&P.lse[(size_t)(p.it.tok0 + i) * P.num_heads + h]);
        return l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
    };
    Pos cur;
    cur.r = 0;
    cur.live = item_id(0) < P.num_items;
    if (!cur.live) return;
    cur.it = score_item(P, item_id(0));
    cur.tt = cur.it.tt0;
    cur.hg = 0;
    settle(cur);
    float next_lse = row_lse(cur);
    int count = 0;  // products taken
    bool ok = true;
    while (cur.live) {
        // a new item: its score, if this key takes part
        const SItem it = cur.it;
        const int key = it.k0 + t * kKeys + rk;
        float *dst = nullptr;
        float old = 0.f, acc = 0.f;
        if (key < it.L) {
            const int blk = __ldg(&P.block_tables[(size_t)it.s * P.max_blocks_per_seq + (key >> P.block_shift)]);
            if (blk >= 0 && blk < P.num_blocks) {
                dst = P.scores + ((long long)it.s * P.num_kv_heads + it.hk) * P.score_stride + key;
                old = *dst;
            }
        }
        for (;;) {
            const int b = count & 1;
            float *lse = s_lse + (t * 2 + b) * kMaxCols;
            volatile int *dead = s_dead + (t * 2 + b) * 4;
            // stage this product's lse; buffer b was last read two products ago
            if (rk < cols) lse[rk] = next_lse;
            const bool any_dead = __any_sync(0xffffffffu, rk < cols && next_lse == INFINITY);
            if (lane == 0) dead[wq] = any_dead;
            mbar_arrive(&B.staged[t]);
            const int tt = cur.tt;
            if (++cur.hg == P.head_groups) {
                cur.hg = 0;
                ++cur.tt;
            }
            const unsigned r = cur.r;
            settle(cur);
            next_lse = row_lse(cur);  // arrives during this product
            ok = mbar_wait(&B.staged[t], (uint32_t)count & 1u, abort_flag) &&
                 mbar_wait(&B.s_full[2 * t + b], (uint32_t)(count >> 1) & 1u, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const int first = key - it.c - (tt << P.lg_nq);  // first token of the tile that sees the key
            const int lo = max(0, first) << P.lg_nh;
            const int hi = (it.n - (tt << P.lg_nq)) << P.lg_nh;
            const bool all = __all_sync(0xffffffffu, lo == 0) && hi >= cols &&
                             !(dead[0] | dead[1] | dead[2] | dead[3]);
            const uint32_t tb = tm + (uint32_t)(128 * b);
            uint32_t ua[32], ub[32];
            float sum = 0.f;
            tmem_ld32(tb, ua);
            for (int c = 0; c < cols; c += 64) {
                tmem_wait_ld();
                const bool more = c + 32 < cols;
                if (more) tmem_ld32(tb + (uint32_t)(c + 32), ub);
                if (!more) {
                    tc_fence_before();
                    mbar_arrive(&B.s_free[2 * t + b]);
                }
                sum += all ? sum32<true>(ua, lse, c, lo, hi, P.scale_log2)
                           : sum32<false>(ua, lse, c, lo, hi, P.scale_log2);
                if (!more) break;
                tmem_wait_ld();
                const bool again = c + 64 < cols;
                if (again) {
                    tmem_ld32(tb + (uint32_t)(c + 64), ua);
                } else {
                    tc_fence_before();
                    mbar_arrive(&B.s_free[2 * t + b]);
                }
                sum += all ? sum32<true>(ub, lse, c + 32, lo, hi, P.scale_log2)
                           : sum32<false>(ub, lse, c + 32, lo, hi, P.scale_log2);
            }
            acc += sum;
            ++count;
            if (!cur.live || cur.r != r) break;
        }
        if (!ok) break;
        if (dst) *dst = old + acc;
    }
    if (!ok) {
        *abort_flag = 1;
        if (lane == 0 && P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreadsS, 1)
    prefill_scores_kernel(const __grid_constant__ ScoreParams P, uint32_t fmt) {
    using L = SLayout<D>;
    constexpr int RQ = L::RQ;
    extern __shared__ __align__(1024) unsigned char smem[];
    pdl_trigger();
    // the swizzled tiles need 1024-byte alignment, which the start of dynamic
    // shared memory has
    if (smem_u32(smem) & 1023u) {
        pdl_wait();
        if (threadIdx.x == 0 && P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
        return;
    }
    float *s_lse = reinterpret_cast<float *>(smem);
    volatile int *s_dead = reinterpret_cast<volatile int *>(smem + L::dead_off);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::bar_off);
    unsigned char *sk = smem + L::small + L::k_off, *sq = smem + L::small + L::q_off;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::tmem_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::flag_off);
    SBars B;
    B.k_full = bars;
    B.k_free = B.k_full + 2;
    B.q_full = B.k_free + 2;
    B.q_free = B.q_full + RQ;
    B.s_full = B.q_free + RQ;
    B.s_free = B.s_full + 4;
    B.staged = B.s_free + 4;
    B.done = B.staged + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&P.tmap_q);
        prefetch_tmap(&P.tmap_k);
        for (int b = 0; b < L::kBars; ++b) mbar_init(&bars[b], 1);
        for (int b = 0; b < 4; ++b) mbar_init(&B.s_free[b], kKeys);
        for (int b = 0; b < 2; ++b) mbar_init(&B.staged[b], kKeys);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) tmem_alloc(tmem_slot, kTmemColsS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();  // the kernels before may still write what this reads
    if (warp == 0) {
        run_score_producer<D>(P, sk, sq, B, abort_flag, lane);
    } else if (warp == 1) {
        if (lane == 0) {
            run_score_mma<D>(P, fmt, sk, sq, tmem, B, abort_flag);
            // every product has completed before tensor memory is released
            volatile int never = 0;
            mbar_drain_wait(B.done, 0, &never);
        }
        __syncwarp();
    } else if (warp >= 4) {
        run_score_sums(P, (warp - 4) >> 2, s_lse, s_dead, tmem, B, abort_flag, warp & 3, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, kTmemColsS);
}

template <int D>
pa_status_t launch_scores(const ScoreParams &P, uint32_t fmt, unsigned grid, cudaStream_t stream) {
    using L = SLayout<D>;
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PA_ERR_CUDA;
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(prefill_scores_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)L::bytes) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_set[dev].store(true, std::memory_order_relaxed);
    }
    return launch_pdl(prefill_scores_kernel<D>, dim3(grid), dim3(kThreadsS), L::bytes, stream, P,
                      fmt) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
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
    if (!query || !lse || !k_cache || !block_tables || !query_start_loc || !context_lens || !scores ||
        !workspace)
        return PA_ERR_INVALID_ARG;
    if (!is_aligned(query, 16) || !is_aligned(k_cache, 16) || !is_aligned(lse, 4) ||
        !is_aligned(scores, 4))
        return PA_ERR_INVALID_ARG;
    if (!is_aligned(workspace, 256) ||
        workspace_bytes < pa_prefill_scores_workspace_size(num_seqs, num_heads, num_kv_heads,
                                                           head_dim, max_query_len, max_context_len))
        return PA_ERR_WORKSPACE;
    const int sms = device_sms();
    if (sms <= 0) return PA_ERR_CUDA;
    ScoreParams P;
    std::memset(&P, 0, sizeof(P));
    const int G = num_heads / num_kv_heads;
    // A query tile: NH heads, the largest power of two that divides the group
    // (at most 128), and NQ tokens, as many as make 128 rows but no more than
    // the longest sequence of queries needs (at least 32 rows, one step of a
    // thread's loads).
    while (P.lg_nh < 7 && G % (2 << P.lg_nh) == 0) ++P.lg_nh;
    while (P.lg_nh + P.lg_nq < 7 &&
           ((1 << P.lg_nq) < max_query_len || P.lg_nh + P.lg_nq < 5))
        ++P.lg_nq;
    P.head_groups = G >> P.lg_nh;
    const cuuint64_t KB = (cuuint64_t)head_dim / 64;
    {
        const cuuint64_t dims[4] = {64u, (cuuint64_t)num_heads, (cuuint64_t)num_tokens, KB};
        const cuuint64_t strides[3] = {(cuuint64_t)head_dim * 2,
                                       (cuuint64_t)num_heads * head_dim * 2, 128u};
        const cuuint32_t box[4] = {64u, 1u << P.lg_nh, 1u << P.lg_nq, (cuuint32_t)KB};
        if (!encode_tiled(&P.tmap_q, query, dtype, 4, dims, strides, box)) return PA_ERR_CUDA;
    }
    {
        const cuuint64_t dims[3] = {64u, (cuuint64_t)pool_rows, KB};
        const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, 128u};
        const cuuint32_t box[3] = {64u, (cuuint32_t)(block_size < 64 ? block_size : 64), 1u};
        if (!encode_tiled(&P.tmap_k, k_cache, dtype, 3, dims, strides, box)) return PA_ERR_CUDA;
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
    const unsigned grid = items < (unsigned long long)sms ? (unsigned)items : (unsigned)sms;
    const uint32_t fmt = dtype == PA_BF16 ? 1u : 0u;
    cudaStream_t st = (cudaStream_t)stream;
    return head_dim == 64 ? launch_scores<64>(P, fmt, grid, st) : launch_scores<128>(P, fmt, grid, st);
}
