// pa_prefill_scores.cu -- the attention weight that the new tokens of a batch
// give to every cached token, added to the tokens' scores.
//
// What it computes: with p_ij = exp(scale <q_i, k_j> - lse_i) for new token i
// at position c + i and key j <= c + i (lse_i from pa_prefill_attention_lse),
//     scores[s][hk][j] += sum over the group's heads and the rows i of p_ij.
//
// One thread owns a key: its row sits in registers, the query rows pass
// through shared memory, and the sum over rows needs no other thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_nvtx.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kKeys = 128;  // keys (threads) of a CTA
constexpr int kRows = 16;   // query rows staged at once

struct ScoreParams {
    const void *q, *k;
    const float *lse;
    const int32_t *block_tables, *query_start_loc, *context_lens;
    float *scores;
    long long score_stride;
    int max_blocks_per_seq, block_shift, num_blocks;
    int max_query_len, max_context_len, num_tokens, num_heads, num_kv_heads, G;
    float scale_log2;
    unsigned int *err;
};

__device__ __forceinline__ float2 up2(uint32_t u, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
__device__ __forceinline__ float2 up2(uint32_t u, __nv_bfloat16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
}

// grid (128-key tile, KV head, sequence)
template <int D, typename T>
__global__ void __launch_bounds__(kKeys)
    prefill_scores_kernel(const __grid_constant__ ScoreParams P) {
    __shared__ float2 s_q[kRows][D / 2];
    __shared__ float s_lse[kRows];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.z, hk = blockIdx.y, tid = threadIdx.x;
    const int a = P.query_start_loc[s], b = P.query_start_loc[s + 1], L = P.context_lens[s];
    const int n = b - a, c = L - n;
    if (a < 0 || b > P.num_tokens || n < 0 || n > P.max_query_len || c < 0 || L > P.max_context_len) {
        if (tid == 0 && blockIdx.x == 0 && hk == 0 && P.err) atomicOr(P.err, PA_ERRBIT_CONTEXT_LEN);
        return;
    }
    const int j0 = (int)blockIdx.x * kKeys, j = j0 + tid;
    if (j0 >= L || n == 0) return;
    uint32_t k[D / 2];
    bool ok = j < L;
    if (ok) {
        const int blk = P.block_tables[(size_t)s * P.max_blocks_per_seq + (j >> P.block_shift)];
        ok = blk >= 0 && blk < P.num_blocks;
        if (!ok && P.err) atomicOr(P.err, PA_ERRBIT_BLOCK_OOB);
        if (ok) {
            const uint4 *row = reinterpret_cast<const uint4 *>(P.k) +
                               ((((size_t)blk * P.num_kv_heads + hk) << P.block_shift) +
                                (j & ((1 << P.block_shift) - 1))) * (D / 8);
#pragma unroll
            for (int e = 0; e < D / 8; ++e) *reinterpret_cast<uint4 *>(&k[4 * e]) = row[e];
        }
    }
    if (!ok) {
#pragma unroll
        for (int e = 0; e < D / 2; ++e) k[e] = 0u;
    }
    float sum = 0.f;
    // rows in (token, head) order from the first that sees the tile's first key
    const int r_end = n * P.G;
    for (int r0 = max(0, j0 - c) * P.G; r0 < r_end; r0 += kRows) {
        __syncthreads();
        for (int e = tid; e < kRows * (D / 2); e += kKeys) {
            const int r = r0 + e / (D / 2), d = e % (D / 2);
            float2 v = make_float2(0.f, 0.f);
            if (r < r_end) {
                const size_t at = ((size_t)(a + r / P.G) * P.num_heads + hk * P.G + r % P.G) * (D / 2) + d;
                v = up2(reinterpret_cast<const uint32_t *>(P.q)[at], T());
            }
            s_q[e / (D / 2)][d] = v;
        }
        if (tid < kRows) {
            const int r = r0 + tid;
            s_lse[tid] = r < r_end ? P.lse[(size_t)(a + r / P.G) * P.num_heads + hk * P.G + r % P.G] : 0.f;
        }
        __syncthreads();
        for (int r = 0; r < kRows; ++r) {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < D / 2; ++e) {
                const float2 q = s_q[r][e], kk = up2(k[e], T());
                x = fmaf(q.y, kk.y, fmaf(q.x, kk.x, x));
            }
            const float lse = s_lse[r];
            if (r0 + r < r_end && j <= c + (r0 + r) / P.G && lse != -INFINITY)
                sum += ex2(fmaf(x, P.scale_log2, -lse * 1.4426950408889634f));
        }
    }
    if (ok) P.scores[((long long)s * P.num_kv_heads + hk) * P.score_stride + j] += sum;
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
    ScoreParams P;
    P.q = query;
    P.k = k_cache;
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
    P.num_tokens = num_tokens;
    P.num_heads = num_heads;
    P.num_kv_heads = num_kv_heads;
    P.G = num_heads / num_kv_heads;
    P.scale_log2 = scale * 1.4426950408889634f;
    P.err = dev_error_word;
    const dim3 grid((unsigned)((max_context_len + kKeys - 1) / kKeys), (unsigned)num_kv_heads,
                    (unsigned)num_seqs);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (head_dim == 64)
        e = dtype == PA_F16
                ? launch_pdl(prefill_scores_kernel<64, __half>, grid, dim3(kKeys), 0, st, P)
                : launch_pdl(prefill_scores_kernel<64, __nv_bfloat16>, grid, dim3(kKeys), 0, st, P);
    else
        e = dtype == PA_F16
                ? launch_pdl(prefill_scores_kernel<128, __half>, grid, dim3(kKeys), 0, st, P)
                : launch_pdl(prefill_scores_kernel<128, __nv_bfloat16>, grid, dim3(kKeys), 0, st, P);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
