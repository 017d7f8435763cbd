// pa_decode_merge.cuh -- the merge of a sequence's partitions, by the merge
// kernel and by the weight pass of the scored form.
#pragma once

#include "pa_decode.cuh"

namespace pa {

// Fewest tokens of a shared prefix.
constexpr int kMinSharedTokens = 64;

// One CTA per (sequence, HPC query heads) of a multi-partition sequence:
//   M = max_p m_p,  c_p = 2^(m_p - M),  L = sum_p l_p c_p,
//   o = sum_p acc_p c_p / L.
// One pass over the partials: the TPH = 128 / HPC threads of a head cover its
// head_dim / 4 float4 columns (CPT columns a thread) and, when there are more
// threads than columns, form NG partition groups; group g folds partitions
// g, g + NG, ... into a running (M, L, o), rescaling it whenever the maximum
// grows, so a partition's m, l and acc are loaded together instead of in
// three dependent rounds.  The groups' states are then folded the same way
// through shared memory.  Several heads a CTA (HPC > 1) keep the grid small
// when most sequences need no merge: those CTAs only read a length and leave,
// and it is their launches, not the merges, that would cost the time.
constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 4;  // partitions a thread loads before folding them
constexpr int kMergeMaxCtas = 3072;  // heads per CTA grow until the grid is no larger

// (M, L, o) <- the merge of (M, L, o) and (mp, lp, a); an empty state has
// M = -inf (ex2(-inf) = 0 drops it).
__device__ __forceinline__ void fold_state(float &M, float &L, float4 &o, float mp, float lp,
                                           float4 a) {
    const float Mn = fmaxf(M, mp);
    if (Mn == -INFINITY) return;  // both empty
    const float c0 = ex2(M - Mn), c1 = ex2(mp - Mn);
    L = fmaf(L, c0, lp * c1);
    o.x = fmaf(o.x, c0, a.x * c1);
    o.y = fmaf(o.y, c0, a.y * c1);
    o.z = fmaf(o.z, c0, a.z * c1);
    o.w = fmaf(o.w, c0, a.w * c1);
    M = Mn;
}

// Sequence s, heads hgroup * HPC and on; kMergeThreads threads.  The lengths
// and tables are inputs, complete before the grid launched; the partials are
// read after the programmatic-dependent-launch wait.
template <int D, int HPC>
__device__ __forceinline__ void merge_heads(const DecodeParams &P, int s, int hgroup) {
    constexpr int C = D / 4;                       // float4 columns of a head
    constexpr int TPH = kMergeThreads / HPC;       // threads of a head
    constexpr int CPT = C > TPH ? C / TPH : 1;     // columns a thread
    constexpr int NG = TPH > C ? TPH / C : 1;      // partition groups of a head
    static_assert(CPT * TPH == C * NG && (NG == 1 || CPT == 1), "merge shape");
    __shared__ float s_m[HPC][NG], s_l[HPC][NG];
    __shared__ float4 s_acc[HPC][NG][C];
    const int tid = threadIdx.x;
    const int hl = tid / TPH, th = tid % TPH;        // head within the CTA, thread within the head
    const int h = hgroup * HPC + hl;
    const int grp = th / (C / CPT), c0 = (th % (C / CPT)) * CPT;  // partition group, first column
    const int L = P.context_lens[s];  // an input: complete before this grid launched
    if (L <= 0 || L > P.max_context_len) return;  // empty or invalid: a zero row
    // One partition for sure: no split, and no shared prefix.  A sequence can
    // share a prefix only with a neighbour whose first block id equals its
    // own (tables are inputs too, complete before this grid launched).
    if (L <= P.part_tokens) {
        if (!P.grouping || L <= kMinSharedTokens) return;
        const int32_t *row = P.block_tables + (size_t)s * P.max_blocks_per_seq;
        const int b0 = __ldg(row);
        const bool prev = s > 0 && __ldg(row - P.max_blocks_per_seq) == b0;
        const bool next = s + 1 < P.num_seqs && __ldg(row + P.max_blocks_per_seq) == b0;
        if (!prev && !next) return;
    }
    pdl_wait();  // partials from the attention kernels; the plan's counts
    const int np = P.grouping ? P.nparts[s] : (L + P.part_tokens - 1) / P.part_tokens;
    if constexpr (kDebugChecks) {
        if (np > P.max_parts) {
            if (tid == 0 && hgroup == 0 && P.err) atomicOr(P.err, PA_ERRBIT_INTERNAL);
            return;
        }
    }
    if (np <= 1) return;
    const bool live = h < P.num_heads;  // the last CTA of a row may hold fewer heads
    const size_t base = ((size_t)s * P.num_heads + (live ? h : 0)) * P.max_parts;
    const float4 *acc = reinterpret_cast<const float4 *>(P.part_acc + base * D) + c0;

    float M = -INFINITY, Lsum = 0.f;
    float4 o[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    float Mc[CPT], Lc[CPT];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        Mc[c] = -INFINITY;
        Lc[c] = 0.f;
    }
    for (int p0 = grp; live && p0 < np; p0 += kMergeBatch * NG) {
        float mp[kMergeBatch], lp[kMergeBatch];
        float4 a[kMergeBatch][CPT];
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            const int p = p0 + u * NG;
            const bool in = p < np;
            mp[u] = in ? P.part_m[base + p] : -INFINITY;
            lp[u] = in ? P.part_l[base + p] : 0.f;
#pragma unroll
            for (int c = 0; c < CPT; ++c)
                a[u][c] = in ? acc[(size_t)p * C + c] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u)
#pragma unroll
            for (int c = 0; c < CPT; ++c) fold_state(Mc[c], Lc[c], o[c], mp[u], lp[u], a[u][c]);
    }
    M = Mc[0];
    Lsum = Lc[0];  // every column folds the same (m, l): the same M and L
    if constexpr (NG > 1) {  // (then CPT == 1)
        if (c0 == 0) {
            s_m[hl][grp] = M;
            s_l[hl][grp] = Lsum;
        }
        s_acc[hl][grp][c0] = o[0];
        __syncthreads();
        if (grp != 0) return;
#pragma unroll
        for (int g = 1; g < NG; ++g) fold_state(M, Lsum, o[0], s_m[hl][g], s_l[hl][g], s_acc[hl][g][c0]);
    }
    if (!live) return;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const size_t ob = ((size_t)s * P.num_heads + h) * D + (size_t)(c0 + c) * 4;
        store_out(P.out, P.out_dtype, ob + 0, Lsum > 0.f ? o[c].x / Lsum : 0.f);
        store_out(P.out, P.out_dtype, ob + 1, Lsum > 0.f ? o[c].y / Lsum : 0.f);
        store_out(P.out, P.out_dtype, ob + 2, Lsum > 0.f ? o[c].z / Lsum : 0.f);
        store_out(P.out, P.out_dtype, ob + 3, Lsum > 0.f ? o[c].w / Lsum : 0.f);
    }
}

}  // namespace pa
