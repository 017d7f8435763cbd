// pa_evict.cu -- pa_evict_tokens: keep the first, the last and the
// highest-scored tokens of every sequence, layer and KV head, in their order,
// and compact K, V and the scores onto them.
//
// A unit is one (layer, sequence, KV head).  Two kernels for all units:
//   * select: one CTA a unit.  The scores are mapped to whole numbers of the
//     same order, the m-th largest of the middle is found digit by digit (a
//     radix selection: a histogram of 8 bits a pass, narrowed to the digit
//     that holds the m-th largest), and one more pass in index order numbers
//     the kept tokens -- those above the threshold and the first of those at
//     it -- with a scan, so equal scores go to the lowest index whatever the
//     timing.  The scores move to their new places in the same pass: a kept
//     token's place is never past its index, and a tile is read whole before
//     any of it is written.
//   * move: the K and V rows of the kept tokens, 16 bytes a thread, in
//     ascending tiles; again a tile is read before it is written, which makes
//     the move safe within the sequence's own blocks.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_nvtx.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelPer = 8;  // tokens a thread numbers at once
constexpr int kSelTile = kSelThreads * kSelPer;
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;  // 16-byte chunks a thread has in flight

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
    int32_t *index;  // [units][max_keep_len]: the kept tokens of each unit, ascending
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

// A score as a whole number of the same order; NaN below everything, -0 = 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// grid (KV head, sequence, layer)
__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictParams P) {
    __shared__ unsigned hist[256];
    __shared__ unsigned s_digit, s_need;
    __shared__ unsigned s_warp[kSelThreads / 32];
    pdl_trigger();
    pdl_wait();  // earlier kernels may still write what this reads, or read what it writes
    const int hk = blockIdx.x, s = blockIdx.y, l = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const SeqPlan q = seq_plan(P, s);
    if (tid == 0 && hk == 0 && l == 0) {
        P.new_lens[s] = q.ok ? q.n : q.L;
        if (!q.ok && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
    }
    if (!q.ok || q.L == 0) return;
    const size_t unit = ((size_t)l * P.num_seqs + s) * P.num_kv_heads + hk;
    const size_t head = (size_t)s * P.num_kv_heads + hk;
    const float *sc = P.layer[l].scores + head * P.score_stride;
    float *out = P.layer[l].scores_out + head * P.score_out_stride;
    int32_t *idx = P.index + unit * P.max_keep_len;
    int32_t *kept = P.layer[l].kept ? P.layer[l].kept + head * P.kept_stride : nullptr;
    const int m0 = q.sink, m1 = q.L - q.recent;  // the middle

    // the mid-th largest key of the middle: threshold, and how many at it stay
    uint32_t thr = 0u;
    unsigned need = 0u;
    if (q.n < q.L && q.mid > 0) {
        unsigned left = (unsigned)q.mid;
        uint32_t mask = 0u;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0u;
            __syncthreads();
            for (int t = m0 + tid; t < m1; t += kSelThreads) {
                const uint32_t key = order_key(sc[t]);
                if ((key & mask) == thr) atomicAdd(&hist[(key >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (wid == 0) {  // the digit whose keys, largest first, reach `left`
                unsigned c[8], sum = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - (lane * 8 + i)];
                unsigned incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += u;
                }
                unsigned before = incl - sum;
                if (before < left && incl >= left) {
                    int i = 0;
                    while (before + c[i] < left) before += c[i++];
                    s_digit = 255u - (unsigned)(lane * 8 + i);
                    s_need = left - before;
                }
            }
            __syncthreads();
            thr |= s_digit << shift;
            mask |= 255u << shift;
            left = s_need;
            __syncthreads();
        }
        need = left;
    }

    // number the kept tokens in index order
    int base_gt = 0, base_eq = 0;
    for (int t0 = 0; t0 < q.L; t0 += kSelTile) {
        const int t = t0 + tid * kSelPer;
        float x[kSelPer];
        unsigned cls = 0u;  // 2 bits a token: 1 above the threshold or fixed, 2 at it
        unsigned cnt = 0u;  // above in the low half, at it in the high half
#pragma unroll
        for (int i = 0; i < kSelPer; ++i) {
            x[i] = t + i < q.L ? sc[t + i] : 0.f;
            if (t + i >= q.L) continue;
            const uint32_t key = order_key(x[i]);
            const bool fixed = q.n == q.L || t + i < m0 || t + i >= m1;
            if (fixed || (q.mid > 0 && key > thr)) {
                cls |= 1u << (2 * i);
                cnt += 1u;
            } else if (q.mid > 0 && key == thr) {
                cls |= 2u << (2 * i);
                cnt += 1u << 16;
            }
        }
        unsigned incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) s_warp[wid] = incl;
        __syncthreads();  // and: the whole tile has been read
        unsigned before = incl - cnt, total = 0u;
        for (int w = 0; w < kSelThreads / 32; ++w) {
            if (w < wid) before += s_warp[w];
            total += s_warp[w];
        }
        int gt = base_gt + (int)(before & 0xffffu), eq = base_eq + (int)(before >> 16);
#pragma unroll
        for (int i = 0; i < kSelPer; ++i) {
            const unsigned c = (cls >> (2 * i)) & 3u;
            if (c == 1u || (c == 2u && eq < (int)need)) {
                const int p = gt + min(eq, (int)need);
                idx[p] = t + i;
                if (kept) kept[p] = t + i;
                out[p] = x[i];
            }
            gt += c == 1u;
            eq += c == 2u;
        }
        base_gt += (int)(total & 0xffffu);
        base_eq += (int)(total >> 16);
        __syncthreads();
    }
    for (int p = q.n + tid; p < q.L; p += kSelThreads) out[p] = 0.f;  // vacated positions
}

// grid (KV head, sequence, layer x {K, V})
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictParams P) {
    pdl_trigger();
    pdl_wait();
    const int hk = blockIdx.x, s = blockIdx.y, l = blockIdx.z >> 1;
    const SeqPlan q = seq_plan(P, s);
    if (!q.ok || (P.in_place && q.n == q.L)) return;
    uint4 *pool = blockIdx.z & 1 ? P.layer[l].v : P.layer[l].k;
    const int32_t *idx =
        P.index + (((size_t)l * P.num_seqs + s) * P.num_kv_heads + hk) * P.max_keep_len;
    const int32_t *src = P.block_tables + (size_t)s * P.max_blocks_per_seq;
    const int32_t *dst = P.in_place ? src : P.dst_block_tables + (size_t)s * P.dst_max_blocks_per_seq;
    const int c = threadIdx.x & ((1 << P.lg_cpr) - 1), r = threadIdx.x >> P.lg_cpr;
    const int rows = kMoveThreads >> P.lg_cpr, in_block = (1 << P.block_shift) - 1;
    auto at = [&](const int32_t *table, int t) -> uint4 * {
        const int b = table[t >> P.block_shift];
        if (b < 0 || b >= P.num_blocks) {
            if (c == 0 && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
            return nullptr;
        }
        return pool + (((((size_t)b * P.num_kv_heads + hk) << P.block_shift) + (t & in_block))
                       << P.lg_cpr) + c;
    };
    for (int i0 = 0; i0 < q.n; i0 += rows * kMoveBatch) {
        uint4 x[kMoveBatch];
        bool have[kMoveBatch];
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u) {
            const int i = i0 + u * rows + r;
            const uint4 *p = i < q.n ? at(src, idx[i]) : nullptr;
            have[u] = p != nullptr;
            if (have[u]) x[u] = *p;
        }
        __syncthreads();  // the tile has been read
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u) {
            const int i = i0 + u * rows + r;
            if (!have[u]) continue;
            uint4 *p = at(dst, i);
            if (p) *p = x[u];
        }
    }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_evict_workspace_size(int num_layers, int num_seqs, int num_kv_heads,
                                          int max_context_len, int max_keep_len) {
    if (num_layers <= 0 || num_layers > PA_MAX_LAYERS || num_seqs < 0 || num_kv_heads <= 0 ||
        max_context_len < 0 || max_keep_len < 0)
        return 0;
    const size_t units = (size_t)num_layers * num_seqs * num_kv_heads;
    return round_up_256(units * max_keep_len * sizeof(int32_t)) + 256;
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
    P.index = (int32_t *)workspace;
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
    if (launch_pdl(evict_select_kernel,
                   dim3((unsigned)num_kv_heads, (unsigned)num_seqs, (unsigned)num_layers),
                   dim3(kSelThreads), 0, st, P) != cudaSuccess)
        return PA_ERR_CUDA;
    return launch_pdl(evict_move_kernel,
                      dim3((unsigned)num_kv_heads, (unsigned)num_seqs, (unsigned)(2 * num_layers)),
                      dim3(kMoveThreads), 0, st, P) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}
