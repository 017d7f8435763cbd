// pa_evict.cu -- pa_evict_tokens: keep the first, the last and the
// highest-scored tokens of every sequence, layer and KV head, in their order,
// and compact K, V and the scores onto them.
//
// A unit is one (layer, sequence, KV head).  Two kernels for all units:
//   * select: one CTA a unit, or a cluster of up to eight where units are few
//     and long, each CTA with a contiguous segment of the scores in shared
//     memory, read once.  Scores are mapped to whole numbers of the same
//     order, and the m-th largest of the middle is found digit by digit (a
//     radix selection: a histogram of 11, 11 and 10 bits, narrowed each time
//     to the digit that holds the m-th largest; a cluster adds its CTAs'
//     histograms through distributed shared memory).  Two more passes count
//     and place the kept tokens in index order -- those above the threshold
//     and the first of those at it -- so equal scores go to the lowest index
//     whatever the timing.
//   * move: the K and V rows of the kept tokens, 32 KB a CTA through
//     registers.
//
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_nvtx.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

// Threads of a select CTA: one of several on an SM, or one that has the SM (a
// long sequence's cluster).  131072 tokens over 8 CTAs: 25.5 us with 512, 22.6
// with 1024.
constexpr int kSelThreads = 512, kSelThreadsLong = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;  // 16-byte pieces a thread has in flight

struct EvictLayer {
    uint4 *k, *v;
    const float *scores;
    float *scores_out;
    int32_t *kept;  // or null
};

struct EvictParams {
    EvictLayer layer[PA_MAX_LAYERS];
    long long score_stride, score_out_stride, kept_stride;
    const int32_t *block_tables, *dst_block_tables;
    int max_blocks_per_seq, dst_max_blocks_per_seq;
    const int32_t *context_lens, *keep_lens;
    int32_t *new_lens;
    int32_t *index;   // [units][max_keep_len]: the kept tokens of each unit, ascending
    unsigned *ticket; // [units]: chunks taken (in place)
    unsigned *flags;  // [units][max_chunks]: chunks read (in place)
    int max_chunks;
    int max_context_len, max_keep_len, num_sink, num_recent;
    int num_seqs, num_kv_heads, num_blocks, block_shift;
    int lg_cpr;    // log2 of a row's 16-byte chunks
    int in_place;  // no other destination blocks
    unsigned int *err;
};

// What becomes of a sequence.
struct SeqPlan {
    int L, n;              // tokens before and after
    int sink, recent, mid; // of the n: first, last, and by score
    bool ok;
};

__device__ __forceinline__ SeqPlan seq_plan(const EvictParams &P, int s) {
    SeqPlan q;
    q.L = P.context_lens[s];
    const int keep = P.keep_lens[s];
    q.n = min(q.L, keep);
    q.ok = q.L >= 0 && q.L <= P.max_context_len && keep >= 0 && q.n <= P.max_keep_len;
    q.recent = min(P.num_recent, q.n);
    q.sink = min(P.num_sink, q.n - q.recent);
    q.mid = q.n - q.recent - q.sink;
    return q;
}

// A score as a whole number of the same order, and back: NaN is 0, below
// everything, and -0 is 0 (the only two whose bits do not come back).
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t key) {
    return __uint_as_float((key >> 31) ? key ^ 0x80000000u : ~key);
}

// Histogram digits of the radix selection: 11, 11 and 10 bits.
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// Another CTA of the cluster's copy of a word of this one's shared memory: read,
// write, add.
__device__ __forceinline__ uint32_t cluster_addr(const unsigned *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ unsigned ld_cluster(const unsigned *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(unsigned *p, uint32_t rank, unsigned v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void add_cluster(unsigned *p, uint32_t rank, unsigned v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)),
                 "r"(v)
                 : "memory");
}

// grid (cluster rank, unit): CS CTAs a unit, each with a contiguous segment of
// its tokens in shared memory.
template <int CS, int THREADS>
__global__ void __launch_bounds__(THREADS)
    evict_select_kernel(const __grid_constant__ EvictParams P) {
    extern __shared__ uint4 s_key4[];  // the order keys of this CTA's segment, four a word
    // hist: this CTA's counts; a cluster adds them up in all_hist of its CTA 0
    // (hist also holds a step's kept tokens of every warp, 128 each)
    __shared__ unsigned hist[THREADS * 4 > kBins ? THREADS * 4 : kBins], all_hist[CS > 1 ? kBins : 1];
    __shared__ unsigned s_warp[THREADS / 32], s_digit, s_need;
    __shared__ unsigned s_total;  // the segment's tokens above the threshold, and at it << 16
    uint32_t *const s_key = reinterpret_cast<uint32_t *>(s_key4);
    constexpr int kWarps = THREADS / 32;
    pdl_wait();  // earlier kernels may still write what this reads, or read what it writes
    // The move kernel may be set up now.  Without one the next call's kernels
    // come next, and those read new_lens (as their context lengths) as soon as
    // they start: then nothing is let through before this grid has ended.
    if (P.max_chunks) pdl_trigger();
    const unsigned unit = blockIdx.x / CS;
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    const int hk = (int)(unit % (unsigned)P.num_kv_heads);
    const unsigned ls = unit / (unsigned)P.num_kv_heads;
    const int s = (int)(ls % (unsigned)P.num_seqs), l = (int)(ls / (unsigned)P.num_seqs);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const SeqPlan q = seq_plan(P, s);
    if (tid == 0 && rank == 0 && hk == 0 && l == 0) {
        P.new_lens[s] = q.ok ? q.n : q.L;
        if (!q.ok && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
    }
    if (!q.ok || q.L == 0) return;  // the same in the whole cluster
    const size_t head = (size_t)s * P.num_kv_heads + hk;
    const float *sc = P.layer[l].scores + head * P.score_stride;
    float *out = P.layer[l].scores_out + head * P.score_out_stride;
    int32_t *idx = P.index + (size_t)unit * P.max_keep_len;
    int32_t *kept = P.layer[l].kept ? P.layer[l].kept + head * P.kept_stride : nullptr;
    if (P.in_place) {  // the move kernel's order of chunks
        if (tid == 0 && rank == 0) P.ticket[unit] = 0u;
        unsigned *flags = P.flags + (size_t)unit * P.max_chunks;
        for (int i = rank * THREADS + tid; i < P.max_chunks; i += CS * THREADS) flags[i] = 0u;
    }
    if (q.n == q.L) {  // everything stays where it is (the move needs no list)
        for (int t = rank * THREADS + tid; t < q.L; t += CS * THREADS) {
            if (kept) kept[t] = t;
            if (out != sc) out[t] = sc[t];
        }
        return;
    }
    const int seg = ((q.L + CS - 1) / CS + 3) & ~3, t0 = rank * seg;
    const int cnt = max(0, min(seg, q.L - t0));  // this CTA's tokens t0 .. t0 + cnt - 1
    for (int i = tid; i < kBins; i += THREADS) {
        hist[i] = 0u;
        if (CS > 1) all_hist[i] = 0u;
    }
    {
        int i = tid;
        for (; i + 7 * THREADS < cnt; i += 8 * THREADS) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = sc[t0 + i + u * THREADS];
#pragma unroll
            for (int u = 0; u < 8; ++u) s_key[i + u * THREADS] = order_key(x[u]);
        }
        for (; i < cnt; i += THREADS) s_key[i] = order_key(sc[t0 + i]);
    }
    __syncthreads();
    const int m0 = q.sink, m1 = q.L - q.recent;  // the middle

    // the mid-th largest key of the middle: threshold, and how many at it stay
    uint32_t thr = 0u;
    unsigned need = 0u;
    if (q.mid > 0) {
        unsigned left = (unsigned)q.mid;
        uint32_t mask = 0u;
        const int i0 = max(0, m0 - t0), i1 = min(cnt, m1 - t0);
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const int bins = pass == 2 ? 1024 : 2048;
#pragma unroll 2
            for (int j = tid; 4 * j < i1; j += THREADS) {
                const uint4 k4 = s_key4[j];
                const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = 4 * j + u;
                    if (i >= i0 && i < i1 && ((key[u] ^ thr) & mask) == 0u)
                        atomicAdd(&hist[(key[u] >> shift) & (unsigned)(bins - 1)], 1u);
                }
            }
            if constexpr (CS > 1) {
                // (the first pass: every CTA's all_hist is zero by now; later
                // ones: cleared before the barrier that ended the last pass)
                if (pass == 0) cluster_sync();
                else __syncthreads();
                for (int i = tid; i < bins; i += THREADS)
                    if (hist[i]) add_cluster(&all_hist[i], 0u, hist[i]);
                cluster_sync();
            } else {
                __syncthreads();
            }
            if (CS == 1 || rank == 0) {
                unsigned *h = CS > 1 ? all_hist : hist;
                // largest digits first: thread i has BPT bins from bins - 1 - BPT i down
                constexpr int BPT = kBins / THREADS;
                unsigned c[BPT], sum = 0u;
#pragma unroll
                for (int k = 0; k < BPT; ++k) {
                    const int b = bins - 1 - (BPT * tid + k);
                    c[k] = b >= 0 ? h[b] : 0u;
                    sum += c[k];
                }
                unsigned incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += u;
                }
                if (lane == 31) s_warp[wid] = incl;
                __syncthreads();
                const unsigned before =
                    incl - sum + __reduce_add_sync(0xffffffffu, lane < wid ? s_warp[lane] : 0u);
                const unsigned hit =
                    __ballot_sync(0xffffffffu, before < left && before + sum >= left);
                if (hit) {  // one warp, and in it one lane
                    int k = 0;
                    unsigned b4 = before;
#pragma unroll
                    for (int e = 0; e < BPT - 1; ++e)
                        if (k == e && b4 + c[e] < left) {
                            b4 += c[e];
                            k = e + 1;
                        }
                    const int src = __ffs((int)hit) - 1;
                    const unsigned digit =
                        __shfl_sync(0xffffffffu, (unsigned)(bins - 1 - (BPT * tid + k)), src);
                    const unsigned rest = __shfl_sync(0xffffffffu, left - b4, src);
                    if (lane < CS) {  // a lane for each CTA
                        if constexpr (CS > 1) {
                            st_cluster(&s_digit, (uint32_t)lane, digit);
                            st_cluster(&s_need, (uint32_t)lane, rest);
                        } else {
                            s_digit = digit;
                            s_need = rest;
                        }
                    }
                }
            }
            if (pass < 2)  // for the next pass (this one's scan has read them)
                for (int i = tid; i < kBins; i += THREADS) {
                    hist[i] = 0u;
                    if (CS > 1) all_hist[i] = 0u;
                }
            if (CS > 1) cluster_sync();
            else __syncthreads();
            thr |= s_digit << shift;
            mask |= (unsigned)(bins - 1) << shift;
            left = s_need;
        }
        need = left;
    }

    // Number the kept tokens in index order.  A warp has a contiguous part of
    // the segment, four tokens a lane and step: count, then place.
    const int part = ((cnt + kWarps - 1) / kWarps + 127) & ~127;
    const int w0 = wid * part, w1 = min(cnt, w0 + part);
    const int f0 = m0 - t0, f1 = m1 - t0;  // the middle, as places of the segment
    const bool some = q.mid > 0;
    // tokens i .. i + 3: bit u of the low half: above the threshold (or always
    // kept); of the high half: at it
    auto classify = [&](int i) -> unsigned {
        if (i >= w1) return 0u;
        const uint4 k4 = s_key4[i >> 2];
        const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
        unsigned c = 0u;
        if (i >= f0 && i + 4 <= f1 && i + 4 <= w1) {  // all in the middle
            if (!some) return 0u;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                c |= (key[u] > thr ? 1u << u : 0u) | (key[u] == thr ? 0x10000u << u : 0u);
            return c;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool in = i + u < w1, fixed = i + u < f0 || i + u >= f1;
            if (in && (fixed || (some && key[u] > thr))) c |= 1u << u;
            if (in && !fixed && some && key[u] == thr) c |= 0x10000u << u;
        }
        return c;
    };
    auto counts = [](unsigned c) -> unsigned {  // above, at << 16
        return (unsigned)__popc(c & 0xffffu) | ((unsigned)__popc(c >> 16) << 16);
    };
    unsigned mine = 0u;
#pragma unroll 2
    for (int i = w0 + 4 * lane; i < w1; i += 128) mine += counts(classify(i));
    mine = __reduce_add_sync(0xffffffffu, mine);  // (both halves stay below 2^16)
    if (lane == 0) s_warp[wid] = mine;
    __syncthreads();
    // the parts before this one: in the CTA, then in the cluster
    unsigned prior = lane < kWarps ? s_warp[lane] : 0u;
    const unsigned total = __reduce_add_sync(0xffffffffu, prior);
    prior = __reduce_add_sync(0xffffffffu, lane < wid ? prior : 0u);
    unsigned b_gt = prior & 0xffffu, b_eq = prior >> 16;
    if constexpr (CS > 1) {
        if (tid == 0) s_total = total;
        cluster_sync();
        unsigned other = lane < rank ? ld_cluster(&s_total, (uint32_t)lane) : 0u;
        b_gt += __reduce_add_sync(0xffffffffu, other & 0xffffu);
        b_eq += __reduce_add_sync(0xffffffffu, other >> 16);
    }
    // A step's kept tokens have consecutive places: gathered in shared memory,
    // then written out with neighbouring lanes on neighbouring places.
    unsigned *const gathered = hist + wid * 128;
    for (int i = w0 + 4 * lane; i - 4 * lane < w1; i += 128) {
        const unsigned c = classify(i), own = counts(c);
        unsigned incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned first = b_gt + min(b_eq, need);
        unsigned g = b_gt + ((incl - own) & 0xffffu), e = b_eq + ((incl - own) >> 16);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool above = (c >> u) & 1u, at = (c >> (16 + u)) & 1u;
            if (above || (at && e < need)) gathered[g + min(e, need) - first] = (unsigned)(i + u);
            g += above;
            e += at;
        }
        const unsigned all = __shfl_sync(0xffffffffu, incl, 31);
        b_gt += all & 0xffffu;
        b_eq += all >> 16;
        const unsigned last = b_gt + min(b_eq, need);
        __syncwarp();
        for (unsigned p = first + lane; p < last; p += 32) {
            const unsigned j = gathered[p - first];
            idx[p] = t0 + (int)j;
            if (kept) kept[p] = t0 + (int)j;
            out[p] = score_of(s_key[j]);
        }
        __syncwarp();
    }
    for (int p = q.n + rank * THREADS + tid; p < q.L; p += CS * THREADS) out[p] = 0.f;
    if (CS > 1) cluster_sync();  // no CTA leaves while another may read its counts
}

// The chunks before chunk c whose old rows its new rows [i0, i0 + rows) may lie
// on: at most `rows` kept tokens, so at most two chunks one after the other,
// the last that starts at or before old row i0 and the next.  Returns the first
// of the two: a warp searches idx, 32 places at a time.
__device__ __forceinline__ int first_below(const int32_t *idx, int c, int lg_rows) {
    const int i0 = c << lg_rows, lane = threadIdx.x & 31;
    int lo = 0, n = c;  // idx of chunk lo is at or before i0 (or lo = 0), that of lo + n is not
    while (n > 1) {
        const int step = (n + 31) >> 5, at = lo + lane * step;
        const bool in = lane * step < n && idx[(size_t)at << lg_rows] <= i0;
        const int hits = __popc(__ballot_sync(0xffffffffu, in));
        const int skip = hits ? (hits - 1) * step : 0;
        n = min(step, n - skip);
        lo += skip;
    }
    return lo;
}

// Wait until a chunk's flag is set; false if the wait gave up.
__device__ __forceinline__ bool wait_chunk(const unsigned *flag) {
    const uint64_t start = globaltimer_ns();
    for (uint32_t polls = 0;; ++polls) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        if (polls >= kWaitLimitPolls || globaltimer_ns() - start > kWaitLimitNs) return false;
    }
}

// grid (max_chunks x units): a CTA moves one chunk of a unit's K and V rows,
// kMoveBatch 16-byte pieces a thread; the chunks of a unit are apart in the
// grid, so that one rarely waits for another.  In place a chunk's new rows may
// lie on old rows of chunks before it, never of chunks after it (a kept token
// moves towards the front), so a CTA reads its chunk into registers, sets the
// chunk's flag, and writes once the chunks on whose old rows it writes have
// been read.  Chunks are taken in order by a counter, so those it waits for
// have been started, and a chunk's reads wait for nothing.  16 layers of 4
// prompts of up to 8000 tokens cut to 1200, in place: 128 us for both kernels,
// 125 into other blocks (a unit's chunks side by side and four CTAs an SM: 184).
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, IN_PLACE ? 5 : 4)
    evict_move_kernel(const __grid_constant__ EvictParams P) {
    __shared__ int s_chunk;
    // (no dependent is let through early)
    pdl_wait();
    const unsigned units = gridDim.x / (unsigned)P.max_chunks;
    int chunk = (int)(blockIdx.x / units);
    const unsigned unit = blockIdx.x - (unsigned)chunk * units;
    if (IN_PLACE && threadIdx.x == 0) s_chunk = (int)atomicAdd(&P.ticket[unit], 1u);
    const int hk = (int)(unit % (unsigned)P.num_kv_heads);
    const unsigned ls = unit / (unsigned)P.num_kv_heads;
    const int s = (int)(ls % (unsigned)P.num_seqs), l = (int)(ls / (unsigned)P.num_seqs);
    const SeqPlan q = seq_plan(P, s);
    if (!q.ok || (IN_PLACE && q.n == q.L)) return;
    const int lg_rows = 10 - P.lg_cpr;  // rows of a chunk: kMoveThreads * kMoveBatch / 2 pieces of K
    static_assert(kMoveThreads * kMoveBatch / 2 == 1 << 10, "pieces of a chunk");
    const int chunks = (q.n + (1 << lg_rows) - 1) >> lg_rows;
    if (IN_PLACE) {
        __syncthreads();
        chunk = s_chunk;
    }
    if ((unsigned)chunk >= (unsigned)chunks) return;
    unsigned *flags = P.flags + (size_t)unit * P.max_chunks;
    const int32_t *idx = P.index + (size_t)unit * P.max_keep_len;
    const int32_t *src = P.block_tables + (size_t)s * P.max_blocks_per_seq;
    const int32_t *dst = IN_PLACE ? src : P.dst_block_tables + (size_t)s * P.dst_max_blocks_per_seq;
    const int c = threadIdx.x & ((1 << P.lg_cpr) - 1), r = threadIdx.x >> P.lg_cpr;
    const int step = kMoveThreads >> P.lg_cpr, in_block = (1 << P.block_shift) - 1;
    const int i0 = chunk << lg_rows;
    constexpr int kRows = kMoveBatch / 2;  // a thread's rows; a K and a V piece each
    size_t from[kRows];
    int to[kRows];  // a row's new block; < 0: it is not moved
    bool oob = false;
    const size_t row_stride = (size_t)P.num_kv_heads << P.block_shift;
    auto piece = [&](int b, int t) -> size_t {  // of token t in block b
        return ((b * row_stride + ((size_t)hk << P.block_shift) + (t & in_block)) << P.lg_cpr) + c;
    };
    const bool all = q.n == q.L;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int i = i0 + u * step + r;
        to[u] = -1;
        if (i >= q.n) continue;
        const int t = all ? i : idx[i];
        // (list and counter come through the caller's workspace: checked before
        // they become an address)
        const bool in = t >= 0 && t < q.L;
        const int b0 = in ? src[t >> P.block_shift] : -1, b1 = dst[i >> P.block_shift];
        const bool ok = b0 >= 0 && b0 < P.num_blocks && b1 >= 0 && b1 < P.num_blocks;
        oob |= !ok;
        if (!ok || (IN_PLACE && t == i)) continue;  // a row that stays needs no move
        from[u] = piece(b0, t);
        to[u] = b1;
    }
    if (oob && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
    uint4 k[kRows], v[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        if (to[u] >= 0) {
            k[u] = P.layer[l].k[from[u]];
            v[u] = P.layer[l].v[from[u]];
        }
    if (IN_PLACE) {
        __syncthreads();  // the chunk has been read
        bool late = false;
        if (threadIdx.x == 0) {
            asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(flags + chunk), "r"(1u) : "memory");
        } else if (threadIdx.x >= 32 && threadIdx.x < 64) {
            const int j = first_below(idx, chunk, lg_rows) + (int)(threadIdx.x & 31);
            if ((threadIdx.x & 31) < 2 && j < chunk) late = !wait_chunk(flags + j);
        }
        if (__syncthreads_or(late)) {
            if (threadIdx.x == 0 && P.err) atomicOr(P.err, PA_ERRBIT_TIMEOUT);
            return;
        }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        if (to[u] >= 0) {
            const size_t at = piece(to[u], i0 + u * step + r);
            P.layer[l].k[at] = k[u];
            P.layer[l].v[at] = v[u];
        }
}

// Workspace: the kept tokens of every unit, then (in place) a chunk counter
// and the chunks' flags of every unit.  A chunk has 32, 64 or 128 rows.
struct EvictWork {
    size_t ticket, flags, bytes;
    long long max_chunks;
};
EvictWork evict_work(size_t units, int max_keep_len, int rows) {
    EvictWork w;
    w.max_chunks = ((long long)max_keep_len + rows - 1) / rows;
    w.ticket = round_up_256(units * max_keep_len * sizeof(int32_t));
    w.flags = round_up_256(w.ticket + units * sizeof(unsigned));
    w.bytes = round_up_256(w.flags + units * (size_t)w.max_chunks * sizeof(unsigned)) + 256;
    return w;
}

// Tokens of one CTA's segment at most: 48 Ki scores (192 KB) beside the
// histograms.
constexpr long long kMaxSegment = 48 * 1024;

template <int CS>
cudaError_t launch_select(const EvictParams &P, unsigned units, size_t smem, cudaStream_t stream) {
    constexpr int kThreads = CS > 1 ? kSelThreadsLong : kSelThreads;
    auto kern = evict_select_kernel<CS, kThreads>;
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kMaxSegment * 4));
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * CS);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_evict_workspace_size(int num_layers, int num_seqs, int num_kv_heads,
                                          int max_context_len, int max_keep_len) {
    if (num_layers <= 0 || num_layers > PA_MAX_LAYERS || num_seqs < 0 || num_kv_heads <= 0 ||
        max_context_len < 0 || max_keep_len < 0)
        return 0;
    return evict_work((size_t)num_layers * num_seqs * num_kv_heads, max_keep_len, 32).bytes;
}

extern "C" pa_status_t pa_evict_tokens(
    void *const *k_caches, void *const *v_caches, int num_layers, const float *const *scores,
    int64_t score_stride, float *const *scores_out, int64_t score_out_stride,
    int32_t *const *kept, int64_t kept_stride, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *dst_block_tables, int dst_max_blocks_per_seq,
    const int32_t *context_lens, const int32_t *keep_lens, int32_t *new_lens,
    int max_context_len, int max_keep_len, int num_sink, int num_recent, int num_seqs,
    int num_blocks, int block_size, int num_kv_heads, int head_dim, pa_dtype_t dtype,
    void *workspace, size_t workspace_bytes, unsigned int *dev_error_word, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_evict_tokens");
    if (num_layers <= 0 || num_seqs < 0 || num_blocks <= 0 || num_kv_heads <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0 || max_keep_len < 0 || num_sink < 0 ||
        num_recent < 0)
        return PA_ERR_INVALID_ARG;
    const int shift = pool_block_shift(block_size);
    if (shift < 0 || num_layers > PA_MAX_LAYERS) return PA_ERR_UNSUPPORTED;
    if (!is_16bit(dtype)) return PA_ERR_INVALID_ARG;
    if (!head_dim_supported(head_dim)) return PA_ERR_UNSUPPORTED;
    if (num_kv_heads > 65535 || num_seqs > 65535) return PA_ERR_UNSUPPORTED;
    const long long units = (long long)num_layers * num_seqs * num_kv_heads;
    if (max_context_len > kMaxSegment * kMaxCluster || units * kMaxCluster >= (1ll << 31) ||
        units * ((max_keep_len + 31ll) / 32) >= (1ll << 31))
        return PA_ERR_UNSUPPORTED;
    if (max_keep_len > max_context_len ||
        (long long)max_context_len > (long long)block_size * max_blocks_per_seq ||
        score_stride < max_context_len || (scores_out && score_out_stride < max_context_len) ||
        (kept && kept_stride < max_keep_len))
        return PA_ERR_INVALID_ARG;
    if (dst_block_tables &&
        (dst_max_blocks_per_seq <= 0 ||
         (long long)max_keep_len > (long long)block_size * dst_max_blocks_per_seq))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!k_caches || !v_caches || !scores || !block_tables || !context_lens || !keep_lens ||
        !new_lens || !workspace)
        return PA_ERR_INVALID_ARG;
    // every unit reads the lengths while one writes the new ones
    if (new_lens == context_lens || new_lens == keep_lens) return PA_ERR_INVALID_ARG;
    EvictParams P;
    std::memset(&P, 0, sizeof(P));
    for (int l = 0; l < num_layers; ++l) {
        if (!k_caches[l] || !v_caches[l] || !is_aligned(k_caches[l], 16) ||
            !is_aligned(v_caches[l], 16) || !scores[l] || !is_aligned(scores[l], 4))
            return PA_ERR_INVALID_ARG;
        if (scores_out && (!scores_out[l] || !is_aligned(scores_out[l], 4)))
            return PA_ERR_INVALID_ARG;
        if (kept && (!kept[l] || !is_aligned(kept[l], 4))) return PA_ERR_INVALID_ARG;
        P.layer[l].k = (uint4 *)k_caches[l];
        P.layer[l].v = (uint4 *)v_caches[l];
        P.layer[l].scores = scores[l];
        P.layer[l].scores_out = scores_out ? scores_out[l] : const_cast<float *>(scores[l]);
        P.layer[l].kept = kept ? kept[l] : nullptr;
    }
    if (!is_aligned(workspace, 256) ||
        workspace_bytes < pa_evict_workspace_size(num_layers, num_seqs, num_kv_heads,
                                                  max_context_len, max_keep_len))
        return PA_ERR_WORKSPACE;
    P.score_stride = score_stride;
    P.score_out_stride = scores_out ? score_out_stride : score_stride;
    P.kept_stride = kept_stride;
    P.block_tables = block_tables;
    P.dst_block_tables = dst_block_tables;
    P.max_blocks_per_seq = max_blocks_per_seq;
    P.dst_max_blocks_per_seq = dst_max_blocks_per_seq;
    P.context_lens = context_lens;
    P.keep_lens = keep_lens;
    P.new_lens = new_lens;
    const int rows = 2048 / (head_dim / 4);  // of a chunk
    const EvictWork w = evict_work((size_t)units, max_keep_len, rows);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    P.index = reinterpret_cast<int32_t *>(ws);
    P.ticket = reinterpret_cast<unsigned *>(ws + w.ticket);
    P.flags = reinterpret_cast<unsigned *>(ws + w.flags);
    P.max_chunks = (int)w.max_chunks;
    P.max_context_len = max_context_len;
    P.max_keep_len = max_keep_len;
    P.num_sink = num_sink;
    P.num_recent = num_recent;
    P.num_seqs = num_seqs;
    P.num_kv_heads = num_kv_heads;
    P.num_blocks = num_blocks;
    P.block_shift = shift;
    P.lg_cpr = head_dim == 64 ? 3 : head_dim == 128 ? 4 : 5;
    P.in_place = dst_block_tables ? 0 : 1;
    P.err = dev_error_word;
    const cudaStream_t st = (cudaStream_t)stream;
    // CTAs a unit: as many as its scores need to fit shared memory, and more
    // (8 at most) while that fills the GPU and leaves each 4096 tokens
    const int sms = device_sms();
    if (sms <= 0) return PA_ERR_CUDA;
    int cs = 1;
    while (cs < kMaxCluster && (max_context_len > kMaxSegment * cs ||
                                (units * cs * 2 <= sms && max_context_len >= 4096 * 2 * cs)))
        cs *= 2;
    const size_t smem = ((((size_t)max_context_len + cs - 1) / cs + 3) & ~(size_t)3) * sizeof(float);
    cudaError_t e = cs == 1   ? launch_select<1>(P, (unsigned)units, smem, st)
                    : cs == 2 ? launch_select<2>(P, (unsigned)units, smem, st)
                    : cs == 4 ? launch_select<4>(P, (unsigned)units, smem, st)
                              : launch_select<8>(P, (unsigned)units, smem, st);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    if (P.max_chunks == 0) return PA_OK;  // nothing is kept anywhere
    const dim3 grid((unsigned)(units * P.max_chunks));
    e = P.in_place ? launch_pdl(evict_move_kernel<true>, grid, dim3(kMoveThreads), 0, st, P)
                   : launch_pdl(evict_move_kernel<false>, grid, dim3(kMoveThreads), 0, st, P);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
