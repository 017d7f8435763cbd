// pa_q4_decode.cu -- pa_decode_attention_q4 and pa_decode_q4_workspace_size: checks,
// sizes and launches (the kernels: pa_q4_decode.cuh).
#include <cuda_runtime.h>

#include <climits>
#include <cstring>

#include "pa_host.cuh"
#include "pa_nvtx.cuh"
#include "pa_q4_decode.cuh"

namespace pa {

cudaError_t launch_q4_decode_d64(const Q4DecodeParams &, int, pa_dtype_t, int, bool, cudaStream_t);
cudaError_t launch_q4_decode_d128(const Q4DecodeParams &, int, pa_dtype_t, int, bool, cudaStream_t);
cudaError_t launch_q4_decode_d256(const Q4DecodeParams &, int, pa_dtype_t, int, bool, cudaStream_t);

namespace {

// Contexts of at most this many chunks are not cut: a warp takes a (sequence, head,
// rows) alone, and no merge kernel runs.
constexpr int kWholeChunks = 16;
// A warp's least share of a batch whose contexts may be cut.
constexpr int kMinShare = 8;

constexpr int kMostUnitCost = 7;
static_assert(Q4Shape<128, 1>::kUnitCost <= kMostUnitCost, "what a unit costs");

struct Plan {
    int rows;     // query rows of a tile
    int ctas;
    bool whole;
    size_t tails, ml, part, bytes;  // offsets in the workspace
};

template <int D>
int max_workers(int rows) {
    return rows <= 4   ? Q4Shape<D, 4>::kWorkers
           : rows <= 8 ? Q4Shape<D, 8>::kWorkers
                       : Q4Shape<D, 16>::kWorkers;
}

// False: sizes past what the kernels count in 32 bits.
bool make_plan(Plan *p, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
               int max_query_len, int max_context_len) {
    const long long G = num_heads / num_kv_heads, most = G * max_query_len;
    p->rows = most <= (head_dim == 256 ? 2 : 1) ? (head_dim == 256 ? 2 : 1)
              : most <= 2                       ? 2
              : most <= 4                       ? 4
              : most <= 8 || head_dim == 256    ? 8
                                                : 16;
    const long long chunks = ((long long)max_context_len + kQ4Tokens - 1) / kQ4Tokens;
    const long long units = num_kv_heads * ((most + p->rows - 1) / p->rows);
    // (rows of a sequence: q4_token_of)
    if (most >= 65536 || units > INT_MAX || units * (chunks + kMostUnitCost) > INT_MAX) return false;
    // (bytes of a block; below, a warp's share of the chunks)
    if ((long long)num_kv_heads * PA_MAX_BLOCK_SIZE * PA_Q4_ROW_BYTES(head_dim) > INT_MAX ||
        num_seqs * (units * (chunks + kMostUnitCost) / 1024) > INT_MAX)
        return false;
    p->whole = chunks <= kWholeChunks;
    const int top = head_dim == 64    ? max_workers<64>(p->rows)
                    : head_dim == 128 ? max_workers<128>(p->rows)
                                      : max_workers<256>(p->rows);
    // no more warps than units, or than shares of the longest batch
    const long long want =
        p->whole ? num_seqs * units : (num_seqs * units * chunks + kMinShare - 1) / kMinShare;
    const long long workers = want < top ? (want > 0 ? want : 1) : top;
    p->ctas = (int)((workers + kQ4Warps - 1) / kQ4Warps);
    const size_t n = p->whole ? 0 : (size_t)p->ctas * kQ4Warps;
    p->tails = 0;
    p->ml = round_up_256(n * sizeof(int4));
    p->part = p->ml + round_up_256(n * 2 * p->rows * sizeof(float2));
    p->bytes = p->part + round_up_256(n * 2 * p->rows * head_dim * sizeof(float));
    if (p->bytes == 0) p->bytes = 256;
    return true;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_q4_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                              int head_dim, int max_query_len,
                                              int max_context_len) {
    pa::Plan p;
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
        !pa::head_dim_supported(head_dim) || max_query_len < 1 ||
        max_query_len > PA_MAX_Q4_QUERY || max_context_len < 0 ||
        !pa::make_plan(&p, num_seqs, num_heads, num_kv_heads, head_dim, max_query_len,
                       max_context_len))
        return 0;
    return p.bytes;
}

extern "C" pa_status_t pa_decode_attention_q4(
    void *out, pa_dtype_t out_dtype, const void *query, const void *k_cache, const void *v_cache,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *query_start_loc,
    const int32_t *context_lens, int max_query_len, int max_context_len, int num_seqs,
    int num_tokens, int num_heads, int num_kv_heads, int head_dim, int num_blocks, int block_size,
    float scale, pa_dtype_t dtype, void *workspace, size_t workspace_bytes,
    unsigned int *dev_error_word, pa_stream_t stream) {
    PA_NVTX_RANGE("pa_decode_attention_q4");
    using namespace pa;
    const int shift = q4_block_shift(block_size);
    if (shift < 0) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        max_context_len < 0 || max_query_len < 1 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (!is_16bit(dtype) || (out_dtype != PA_F32 && out_dtype != dtype)) return PA_ERR_INVALID_ARG;
    if (!head_dim_supported(head_dim) || max_query_len > PA_MAX_Q4_QUERY) return PA_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)block_size * max_blocks_per_seq)
        return PA_ERR_INVALID_ARG;
    if (!query_start_loc && (num_tokens != num_seqs || max_query_len != 1))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens || !workspace)
        return PA_ERR_INVALID_ARG;
    for (const void *p : {(const void *)out, query, k_cache, v_cache})
        if (!is_aligned(p, 16)) return PA_ERR_INVALID_ARG;
    if (!is_aligned(workspace, 256)) return PA_ERR_WORKSPACE;
    Plan plan;
    if (!make_plan(&plan, num_seqs, num_heads, num_kv_heads, head_dim, max_query_len,
                   max_context_len))
        return PA_ERR_UNSUPPORTED;
    if (workspace_bytes < plan.bytes) return PA_ERR_WORKSPACE;

    unsigned char *ws = static_cast<unsigned char *>(workspace);
    Q4DecodeParams P;
    std::memset(&P, 0, sizeof(P));
    P.out = out;
    P.query = query;
    P.k_cache = static_cast<const uint8_t *>(k_cache);
    P.v_cache = static_cast<const uint8_t *>(v_cache);
    P.block_tables = block_tables;
    P.context_lens = context_lens;
    P.query_start_loc = query_start_loc;
    P.tails = reinterpret_cast<int4 *>(ws + plan.tails);
    P.part_ml = reinterpret_cast<float2 *>(ws + plan.ml);
    P.part = reinterpret_cast<float *>(ws + plan.part);
    P.err = dev_error_word;
    P.out_f32 = out_dtype == PA_F32;
    P.max_blocks_per_seq = max_blocks_per_seq;
    P.max_context_len = max_context_len;
    P.max_query_len = max_query_len;
    P.num_seqs = num_seqs;
    P.num_tokens = num_tokens;
    P.num_heads = num_heads;
    P.num_kv_heads = num_kv_heads;
    P.G = num_heads / num_kv_heads;
    P.num_blocks = num_blocks;
    P.sub_shift = shift - 4;
    P.whole = plan.whole;
    P.workers = plan.ctas * kQ4Warps;
    P.scale_log2 = scale * 1.4426950408889634f;
    P.inv_G = 1.0f / (float)P.G;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e =
        head_dim == 64    ? launch_q4_decode_d64(P, plan.rows, dtype, plan.ctas, !plan.whole, st)
        : head_dim == 128 ? launch_q4_decode_d128(P, plan.rows, dtype, plan.ctas, !plan.whole, st)
                          : launch_q4_decode_d256(P, plan.rows, dtype, plan.ctas, !plan.whole, st);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
