// pa_q4_decode_d128.cu -- 4-bit decode kernels for head_dim 128 (pa_q4_decode.cuh).
#include "pa_q4_decode_launch.cuh"

namespace pa {
cudaError_t launch_q4_decode_d128(const Q4DecodeParams &P, int rows, pa_dtype_t dtype, int ctas,
                                  bool merge, cudaStream_t stream) {
    return launch_q4_decode<128>(P, rows, dtype, ctas, merge, stream);
}
}  // namespace pa
