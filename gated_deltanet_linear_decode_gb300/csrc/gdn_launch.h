// gdn_launch.h -- launches as a programmatic dependent of the previous kernel in the stream: the CTAs of the next
// kernel may be set up while the previous one ends; every kernel launched this way waits (grid_dependency_wait) before its
// first global access.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdn {

// cluster > 1: thread-block clusters of that many CTAs.
template <typename... P, typename... A>
cudaError_t launch_dependent_cluster(void (*kernel)(P...), int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    return launch_dependent_cluster(kernel, 1, grid, block, smem, stream, args...);
}

}  // namespace gdn
