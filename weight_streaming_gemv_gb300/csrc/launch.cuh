// Launches that may start while the kernel before them on the stream finishes.
#pragma once
#include "common.cuh"

namespace qlin {

// Clusters of `cluster` CTAs along x, of `threads` threads each, that can be on
// the current device at once.  The kernel's limits are raised for them; kept
// per kernel, device and sizes.
int max_clusters(const void *kern, size_t smem, int threads, int cluster);

// A launch with programmatic stream serialisation: the kernel may start while
// the previous one on the stream finishes, and waits (griddepcontrol.wait)
// before it touches what that one reads or writes.  cluster: CTAs of one along
// x, 16 at most, or 0.
inline qlin_status launch_pdl(const void *kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st, void **args,
                              const char *name, int cluster = 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    QLIN_CUDA(cudaLaunchKernelExC(&cfg, kern, args));
    QLIN_LAUNCHED(name);
    return QLIN_OK;
}

}  // namespace qlin
