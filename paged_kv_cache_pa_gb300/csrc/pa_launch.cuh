// pa_launch.cuh -- host helper: launch a kernel on a stream with programmatic
// dependent launch allowed, so its launch overlaps the tail of the previous
// kernel on the stream.  Every kernel launched this way calls
// griddepcontrol.wait (pa::pdl_wait) before it writes to global memory, and
// before it reads what earlier work may write.  Lengths, tables and starts are
// read before it: they are complete before a call (pa.h).  No write comes
// before it, not even to a call's own workspace: the kernels ahead may let
// this one start while they still read their inputs and use their
// workspaces, and the caller may have given this call that memory.
#pragma once

#include <cuda_runtime.h>

namespace pa {

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace pa
