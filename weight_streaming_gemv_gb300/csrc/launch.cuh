// Launches that may start while the kernel before them on the stream finishes.
#pragma once
#include "common.cuh"

namespace qlin {

// A launch with programmatic stream serialisation: the kernel may start while
// the previous one on the stream finishes, and waits (griddepcontrol.wait)
// before it touches what that one reads or writes.
inline qlin_status launch_pdl(const void *kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st, void **args,
                              const char *name) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    QLIN_CUDA(cudaLaunchKernelExC(&cfg, kern, args));
    QLIN_LAUNCHED(name);
    return QLIN_OK;
}

}  // namespace qlin
