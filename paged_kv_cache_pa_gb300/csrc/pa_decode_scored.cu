// pa_decode_scored.cu -- the weight pass of pa_decode_attention_scored.
//
// The scored attention kernels leave every token's logit x_t (base-2 units)
// and every piece's maximum m_p and sum l_p in the workspace.  For each query
// head of the KV head's group
//     M = max_p m_p,  L = sum_p l_p 2^(m_p - M),
// and the pass adds the group's weights to the token's score:
//     scores[s][hk][t] += sum_g 2^(x_gt - M_g) / L_g.
// A row without weight (no readable block, every logit -inf: L = 0) adds
// nothing.  One thread owns a token's score, so the sum's order is fixed.
//
// Scores add up over calls, so weights made from what an attention kernel that
// gave up has left in the workspace would stay: once PA_ERRBIT_TIMEOUT is in
// the error word, nothing is added.
//
// A warp takes 256 tokens of one (sequence, KV head): it works out M and 1 / L
// of each head itself (a lane a piece), so the CTA has no barrier, and its
// loads of the logits, 16 bytes a lane, are all in flight together.  The
// first CTAs of the grid merge the sequences' partitions meanwhile (the same
// code as the merge kernel): one launch less than two kernels in turn.
//
// Bound: HBM, 4 bytes a logit (usually still in L2) and 8 a score, against 4
// head_dim bytes of K and V a token and KV head that the attention kernel
// reads.
#include <cuda_runtime.h>

#include <type_traits>

#include "pa_decode.cuh"
#include "pa_decode_merge.cuh"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kSteps = 2;  // 128 tokens each, four a lane
constexpr int kWarpTokens = 128 * kSteps;
constexpr int kWeightWarps = kMergeThreads / 32;

// Whether the attention kernels skipped the 16-token chunk that holds `token`
// (one block, or two of 8 tokens, outside the pool).
__device__ __noinline__ bool chunk_skipped(const DecodeParams &P, int s, int token, int L) {
    const int32_t *row = P.block_tables + (size_t)s * P.max_blocks_per_seq;
    const int c = token & ~(kBlock - 1);
    const int b0 = row[c >> P.block_shift];
    const int b1 = P.block_size < kBlock && c + P.block_size < L ? row[(c >> P.block_shift) + 1] : b0;
    return b0 < 0 || b0 >= P.num_blocks || b1 < 0 || b1 >= P.num_blocks;
}

// Tokens t0 .. t0 + 255 of (sequence s, KV head hk), by one warp.  GM: the
// group's heads, rounded up to 1, 2, 4 or 8.
template <int GM>
__device__ __forceinline__ void add_weights(const DecodeParams &P, float *__restrict__ scores,
                                            long long score_stride, int s, int hk, int t0,
                                            bool vec, int lane) {
    const int L = P.context_lens[s], G = P.G;
    if (L <= 0 || L > P.max_context_len || t0 >= L) return;  // empty or invalid: nothing to add
    const size_t row0 = (size_t)s * P.num_heads + (size_t)hk * G;
    // (used only before the stores: on its way beside everything else)
    const unsigned status = P.err ? __ldcg(P.err) : 0u;
    const int np = (L + P.part_tokens - 1) / P.part_tokens;
    const int n = min(kWarpTokens, L - t0);
    // every load of the first 32 pieces and of the old scores in flight at once
    float M[GM], inv[GM];
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        const bool in = g < G && lane < np;
        M[g] = in ? P.part_m[(row0 + g) * P.max_parts + lane] : -INFINITY;
        inv[g] = in ? P.part_l[(row0 + g) * P.max_parts + lane] : 0.f;
    }
    float *sc = scores + ((long long)s * P.num_kv_heads + hk) * score_stride + t0;
    float4 old[kSteps], w[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int t = i * 128 + 4 * lane;
        w[i] = old[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec && t + 4 <= n) {
            old[i] = *reinterpret_cast<const float4 *>(sc + t);
        } else {
            if (t < n) old[i].x = sc[t];
            if (t + 1 < n) old[i].y = sc[t + 1];
            if (t + 2 < n) old[i].z = sc[t + 2];
            if (t + 3 < n) old[i].w = sc[t + 3];
        }
    }
    for (int p = lane + 32; p < np; p += 32) {  // contexts of many pieces
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            if (g >= G) continue;
            const float mp = P.part_m[(row0 + g) * P.max_parts + p];
            const float lp = P.part_l[(row0 + g) * P.max_parts + p];
            const float mn = fmaxf(M[g], mp);
            const float ms = mn == -INFINITY ? 0.f : mn;
            inv[g] = inv[g] * ex2(M[g] - ms) + lp * ex2(mp - ms);
            M[g] = mn;
        }
    }
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        float m = M[g];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = m == -INFINITY ? 0.f : m;
        float l = inv[g] * ex2(M[g] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        M[g] = m;
        // an empty row weighs nothing; a NaN sum goes on to the weights
        inv[g] = l == 0.f ? 0.f : 1.f / l;
    }
    // (the logits' rows reach a multiple of 16 tokens)
    const float *lg = P.logits + row0 * P.logit_stride + t0;
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        if (g >= G) continue;
        float4 x[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int t = i * 128 + 4 * lane;
            if (t < n) x[i] = *reinterpret_cast<const float4 *>(lg + (size_t)g * P.logit_stride + t);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            w[i].x = fmaf(ex2(x[i].x - M[g]), inv[g], w[i].x);
            w[i].y = fmaf(ex2(x[i].y - M[g]), inv[g], w[i].y);
            w[i].z = fmaf(ex2(x[i].z - M[g]), inv[g], w[i].z);
            w[i].w = fmaf(ex2(x[i].w - M[g]), inv[g], w[i].w);
        }
    }
    if (status & PA_ERRBIT_TIMEOUT) return;
    // A row whose sum is NaN weighs NaN on every token but those of a skipped
    // block, whose weight of zero times 1 / L is NaN too: looked up only then, out
    // of line (inlined, 64 sequences of 12 heads on 2 take 41.7 us instead of 40.4).
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int t = i * 128 + 4 * lane;
        if (w[i].x != w[i].x && t < n && chunk_skipped(P, s, t0 + t, L)) continue;
        const float4 o = make_float4(old[i].x + w[i].x, old[i].y + w[i].y, old[i].z + w[i].z,
                                     old[i].w + w[i].w);
        if (vec && t + 4 <= n) {
            *reinterpret_cast<float4 *>(sc + t) = o;
        } else {
            if (t < n) sc[t] = o.x;
            if (t + 1 < n) sc[t + 1] = o.y;
            if (t + 2 < n) sc[t + 2] = o.z;
            if (t + 3 < n) sc[t + 3] = o.w;
        }
    }
}

// CTAs 0 .. merges - 1: the merge of (sequence, HPC heads); the others: warp
// tasks (sequence, KV head, 256-token range), ranges fastest.
template <int D, int HPC, int GM>
__global__ void __launch_bounds__(kMergeThreads)
    decode_weights_kernel(const __grid_constant__ DecodeParams P, float *__restrict__ scores,
                          long long score_stride, int merges, int head_groups, int ranges,
                          unsigned tasks, bool vec) {
    // (no dependent is let through early: the next call's plan writes its lists
    // as soon as it starts, which for other sizes lie where this call's logits
    // and states do)
    pdl_wait();  // the logits and the pieces' states
    if ((int)blockIdx.x < merges) {
        merge_heads<D, HPC>(P, (int)blockIdx.x / head_groups, (int)blockIdx.x % head_groups);
        return;
    }
    const unsigned task = (blockIdx.x - (unsigned)merges) * kWeightWarps + threadIdx.x / 32;
    if (task >= tasks) return;
    const unsigned unit = task / (unsigned)ranges;
    add_weights<GM>(P, scores, score_stride, (int)(unit / (unsigned)P.num_kv_heads),
                     (int)(unit % (unsigned)P.num_kv_heads),
                     (int)(task - unit * (unsigned)ranges) * kWarpTokens, vec, threadIdx.x & 31);
}

}  // namespace

pa_status_t launch_decode_weights(const DecodeParams &P, float *scores, long long score_stride,
                                  bool merge, cudaStream_t stream) {
    const long long ranges = (P.max_context_len + kWarpTokens - 1) / kWarpTokens;
    const long long tasks = (long long)P.num_seqs * P.num_kv_heads * ranges;
    // heads a merging CTA: several when there are many (see merge_heads)
    const int hpc = (long long)P.num_seqs * P.num_heads > kMergeMaxCtas ? 4 : 1;
    const int groups = (P.num_heads + hpc - 1) / hpc;
    const long long merges = merge ? (long long)P.num_seqs * groups : 0;
    const long long ctas = merges + (tasks + kWeightWarps - 1) / kWeightWarps;
    if (ctas == 0) return PA_OK;
    if (ctas >= (1ll << 31) || tasks >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    const bool vec = (reinterpret_cast<uintptr_t>(scores) & 15u) == 0 && score_stride % 4 == 0;
    cudaError_t e = cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kMergeThreads), 0, stream, P, scores,
                       score_stride, (int)merges, groups, (int)ranges, (unsigned)tasks, vec);
    };
    const int gm = P.G == 1 ? 1 : P.G == 2 ? 2 : P.G <= 4 ? 4 : 8;
    auto group = [&](auto d, auto h) {
        constexpr int D = decltype(d)::value, H = decltype(h)::value;
        if (gm == 1) go(decode_weights_kernel<D, H, 1>);
        else if (gm == 2) go(decode_weights_kernel<D, H, 2>);
        else if (gm == 4) go(decode_weights_kernel<D, H, 4>);
        else go(decode_weights_kernel<D, H, 8>);
    };
    auto dim = [&](auto d) {
        if (hpc == 1) group(d, std::integral_constant<int, 1>());
        else group(d, std::integral_constant<int, 4>());
    };
    if (P.head_dim == 64) dim(std::integral_constant<int, 64>());
    else if (P.head_dim == 128) dim(std::integral_constant<int, 128>());
    else dim(std::integral_constant<int, 256>());
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
