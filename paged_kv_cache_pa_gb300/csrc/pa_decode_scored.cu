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
// A warp takes 512 tokens of one (sequence, KV head): it works out M and 1 / L
// of each head itself (a lane a piece), so the CTA has no barrier, and its
// loads of the logits, 16 bytes a lane, are all in flight together.  The
// first CTAs of the grid merge the sequences' partitions meanwhile (the same
// code as the merge kernel): one launch less than two kernels in turn.
//
// Bound: HBM, 4 bytes a logit (usually still in L2) and 8 a score, against 4
// head_dim bytes of K and V a token and KV head that the attention kernel
// reads.
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_decode_merge.cuh"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kWarpTokens = 512;
constexpr int kWeightWarps = kMergeThreads / 32;
constexpr int kMaxGroup = 8;

// Tokens t0 .. t0 + 511 of (sequence s, KV head hk), by one warp.
template <bool VEC>
__device__ __forceinline__ void add_weights(const DecodeParams &P, float *__restrict__ scores,
                                            long long score_stride, int s, int hk, int t0,
                                            int lane) {
    const int L = P.context_lens[s], G = P.G;
    if (L <= 0 || L > P.max_context_len || t0 >= L) return;  // empty or invalid: nothing to add
    const size_t row0 = (size_t)s * P.num_heads + (size_t)hk * G;
    const int np = (L + P.part_tokens - 1) / P.part_tokens;
    float M[kMaxGroup], inv[kMaxGroup];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
        M[g] = inv[g] = 0.f;
        if (g >= G) continue;
        const float *pm = P.part_m + (row0 + g) * P.max_parts;
        const float *pl = P.part_l + (row0 + g) * P.max_parts;
        float m = -INFINITY, l = 0.f;
        for (int p = lane; p < np; p += 32) {
            const float mp = pm[p], lp = pl[p];
            const float mn = fmaxf(m, mp);
            if (mn != -INFINITY) l = l * ex2(m - mn) + lp * ex2(mp - mn);
            m = mn;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m, o);
            const float lo = __shfl_xor_sync(0xffffffffu, l, o);
            const float mn = fmaxf(m, mo);
            if (mn != -INFINITY) l = l * ex2(m - mn) + lo * ex2(mo - mn);
            m = mn;
        }
        M[g] = m == -INFINITY ? 0.f : m;
        // an empty row weighs nothing; a NaN sum goes on to the weights
        inv[g] = l == 0.f ? 0.f : 1.f / l;
    }
    const float *lg = P.logits + row0 * P.logit_stride + t0;
    float *sc = scores + ((long long)s * P.num_kv_heads + hk) * score_stride + t0;
    const int n = min(kWarpTokens, L - t0);
#pragma unroll
    for (int i = 0; i < kWarpTokens / 128; ++i) {
        const int t = i * 128 + 4 * lane;
        if (t >= n) break;
        // (the logits' rows reach a multiple of 16 tokens)
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (g >= G) break;
            const float4 x = *reinterpret_cast<const float4 *>(lg + (size_t)g * P.logit_stride + t);
            w.x = fmaf(ex2(x.x - M[g]), inv[g], w.x);
            w.y = fmaf(ex2(x.y - M[g]), inv[g], w.y);
            w.z = fmaf(ex2(x.z - M[g]), inv[g], w.z);
            w.w = fmaf(ex2(x.w - M[g]), inv[g], w.w);
        }
        if (VEC && t + 4 <= n) {
            float4 o = *reinterpret_cast<float4 *>(sc + t);
            o.x += w.x;
            o.y += w.y;
            o.z += w.z;
            o.w += w.w;
            *reinterpret_cast<float4 *>(sc + t) = o;
        } else {
            sc[t] += w.x;
            if (t + 1 < n) sc[t + 1] += w.y;
            if (t + 2 < n) sc[t + 2] += w.z;
            if (t + 3 < n) sc[t + 3] += w.w;
        }
    }
}

// CTAs 0 .. merges - 1: the merge of (sequence, HPC heads); the others: warp
// tasks (sequence, KV head, 512-token range), ranges fastest.
template <int D, int HPC, bool VEC>
__global__ void __launch_bounds__(kMergeThreads)
    decode_weights_kernel(const __grid_constant__ DecodeParams P, float *__restrict__ scores,
                          long long score_stride, int merges, int head_groups, int ranges,
                          unsigned tasks) {
    pdl_trigger();
    pdl_wait();  // the logits and the pieces' states
    if ((int)blockIdx.x < merges) {
        merge_heads<D, HPC>(P, (int)blockIdx.x / head_groups, (int)blockIdx.x % head_groups);
        return;
    }
    const unsigned task = (blockIdx.x - (unsigned)merges) * kWeightWarps + threadIdx.x / 32;
    if (task >= tasks) return;
    const unsigned unit = task / (unsigned)ranges;
    add_weights<VEC>(P, scores, score_stride, (int)(unit / (unsigned)P.num_kv_heads),
                     (int)(unit % (unsigned)P.num_kv_heads),
                     (int)(task - unit * (unsigned)ranges) * kWarpTokens, threadIdx.x & 31);
}

}  // namespace

pa_status_t launch_decode_weights(const DecodeParams &P, float *scores, long long score_stride,
                                  bool merge, cudaStream_t stream) {
    const long long ranges = (P.max_context_len + kWarpTokens - 1) / kWarpTokens;
    const long long tasks = (long long)P.num_seqs * P.num_kv_heads * ranges;
    // heads a merging CTA, as in the merge kernel's launch
    int hpc = 1;
    while (hpc < 8 && (long long)P.num_seqs * ((P.num_heads + hpc - 1) / hpc) > kMergeMaxCtas)
        hpc *= 2;
    const int groups = (P.num_heads + hpc - 1) / hpc;
    const long long merges = merge ? (long long)P.num_seqs * groups : 0;
    const long long ctas = merges + (tasks + kWeightWarps - 1) / kWeightWarps;
    if (ctas == 0) return PA_OK;
    if (ctas >= (1ll << 31) || tasks >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    const bool vec = (reinterpret_cast<uintptr_t>(scores) & 15u) == 0 && score_stride % 4 == 0;
    cudaError_t e = cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kMergeThreads), 0, stream, P, scores,
                       score_stride, (int)merges, groups, (int)ranges, (unsigned)tasks);
    };
#define PA_WEIGHTS(D, H)                             \
    if (P.head_dim == D && hpc == H) {               \
        if (vec) go(decode_weights_kernel<D, H, true>); \
        else go(decode_weights_kernel<D, H, false>); \
    }
    PA_WEIGHTS(64, 1) PA_WEIGHTS(64, 2) PA_WEIGHTS(64, 4) PA_WEIGHTS(64, 8)
    PA_WEIGHTS(128, 1) PA_WEIGHTS(128, 2) PA_WEIGHTS(128, 4) PA_WEIGHTS(128, 8)
    PA_WEIGHTS(256, 1) PA_WEIGHTS(256, 2) PA_WEIGHTS(256, 4) PA_WEIGHTS(256, 8)
#undef PA_WEIGHTS
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
