// pa_decode_scored_d256.cu -- instantiations of the scored form of paged decode
// attention for head_dim 256 (fp16 / bf16).
#include "pa_decode_launch.cuh"

namespace pa {
pa_status_t launch_decode_scored_d256(const DecodeParams &P, pa_dtype_t dtype, int grid_cap,
                                     cudaStream_t stream) {
    return dispatch_scored<256>(P, dtype, grid_cap, stream);
}
}  // namespace pa
