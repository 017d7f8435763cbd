// pa_q4_decode_d256.cu -- 4-bit decode kernels for head_dim 256 (pa_q4_decode.cuh).
#include "pa_q4_decode_launch.cuh"

namespace pa {
cudaError_t launch_q4_decode_d256(const Q4DecodeParams &P, int rows, pa_dtype_t dtype, int ctas,
                                  bool merge, cudaStream_t stream) {
    return launch_q4_decode<256>(P, rows, dtype, ctas, merge, stream);
}
}  // namespace pa
