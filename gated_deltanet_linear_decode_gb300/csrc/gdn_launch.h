// gdn_launch.h -- launches as a programmatic dependent of the previous kernel in the stream: the CTAs of the next
// kernel may be set up while the previous one ends; every kernel launched this way waits (grid_dependency_wait) before its
// first global access.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdn {

// SMs of the current device; 0 where there is none.
inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

// The attributes of a launch; cluster > 1: thread-block clusters of that many CTAs.
struct LaunchConfig {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    LaunchConfig(int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
        cfg.gridDim = grid;
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
    }
    LaunchConfig(const LaunchConfig&) = delete;
};

template <typename... P, typename... A>
cudaError_t launch_dependent_cluster(void (*kernel)(P...), int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    const LaunchConfig c(cluster, grid, block, smem, stream);
    return cudaLaunchKernelEx(&c.cfg, kernel, static_cast<P>(args)...);
}

// How many such clusters run at a time; 0 where none does, or the runtime does not say.
template <typename... P>
int clusters_at_once(void (*kernel)(P...), int cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    const LaunchConfig c(cluster, grid, block, smem, stream);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &c.cfg) == cudaSuccess) return n;
    cudaGetLastError();   // (not an error of the call)
    return 0;
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    return launch_dependent_cluster(kernel, 1, grid, block, smem, stream, args...);
}

}  // namespace gdn
