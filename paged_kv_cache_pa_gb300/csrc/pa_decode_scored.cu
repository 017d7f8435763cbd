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
// Bound: HBM, 4 bytes a logit (usually still in L2) and 8 a score, against 4
// head_dim bytes of K and V a token and KV head that the attention kernel
// reads.
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kWeightThreads = 256;
constexpr int kTokensPerThread = 4;
constexpr int kWeightTokens = kWeightThreads * kTokensPerThread;
constexpr int kMaxGroup = 8;

// grid (sequence, KV head, 1024-token range)
__global__ void __launch_bounds__(kWeightThreads)
    decode_weights_kernel(const __grid_constant__ DecodeParams P, float *__restrict__ scores,
                          long long score_stride) {
    __shared__ float s_m[kMaxGroup], s_inv[kMaxGroup];
    pdl_trigger();
    pdl_wait();  // the logits and the pieces' states
    const int s = blockIdx.x, hk = blockIdx.y, G = P.G;
    const int L = P.context_lens[s];
    const int t0 = (int)blockIdx.z * kWeightTokens;
    if (L <= 0 || L > P.max_context_len || t0 >= L) return;  // empty or invalid: nothing to add
    const size_t row0 = (size_t)s * P.num_heads + (size_t)hk * G;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp < G) {  // warp g: head g's maximum and sum over the pieces
        const int np = (L + P.part_tokens - 1) / P.part_tokens;
        const float *pm = P.part_m + (row0 + warp) * P.max_parts;
        const float *pl = P.part_l + (row0 + warp) * P.max_parts;
        float M = -INFINITY;
        for (int p = lane; p < np; p += 32) M = fmaxf(M, pm[p]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float sum = 0.f;
        for (int p = lane; p < np; p += 32)
            if (pm[p] != -INFINITY) sum += pl[p] * ex2(pm[p] - M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            s_m[warp] = M == -INFINITY ? 0.f : M;
            // an empty row weighs nothing; a NaN sum goes on to the weights
            s_inv[warp] = sum == 0.f ? 0.f : 1.f / sum;
        }
    }
    __syncthreads();
    const float *lg = P.logits + row0 * P.logit_stride;
    float *sc = scores + ((long long)s * P.num_kv_heads + hk) * score_stride;
#pragma unroll
    for (int i = 0; i < kTokensPerThread; ++i) {
        const int t = t0 + i * kWeightThreads + (int)threadIdx.x;
        if (t >= L) break;
        float w = 0.f;
        for (int g = 0; g < G; ++g)
            w = fmaf(ex2(lg[(size_t)g * P.logit_stride + t] - s_m[g]), s_inv[g], w);
        sc[t] += w;
    }
}

}  // namespace

pa_status_t launch_decode_weights(const DecodeParams &P, float *scores, long long score_stride,
                                  cudaStream_t stream) {
    const int ranges = (P.max_context_len + kWeightTokens - 1) / kWeightTokens;
    if (ranges == 0) return PA_OK;
    if (ranges > 65535) return PA_ERR_UNSUPPORTED;
    return launch_pdl(decode_weights_kernel,
                      dim3((unsigned)P.num_seqs, (unsigned)P.num_kv_heads, (unsigned)ranges),
                      dim3(kWeightThreads), 0, stream, P, scores, score_stride) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace pa
