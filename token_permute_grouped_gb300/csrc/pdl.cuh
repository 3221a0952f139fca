// Programmatic dependent launch of the expert-layer kernels: each may be put
// on the SMs while the kernel before it in the stream finishes, and waits for
// that kernel's end (its writes visible) before it touches memory that another
// kernel reads or writes.  For calls of a few microseconds this hides most of
// the launch and of each kernel's set-up.
//
// Every CTA of a kernel that is launched this way passes pdl_wait() before it
// ends, so that a kernel's completion implies that of all kernels before it.
#pragma once

#include <cuda_runtime.h>

namespace a2av {

// The kernel before this one in the stream has completed.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel after this one may be launched (when every CTA has said so or ended).
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// CTAs of a cluster (0: no cluster dimension), and how an SM's L1 and shared
// memory are to be split while this launch runs (percent; -1: as the kernel needs).
struct PdlShape {
    int cluster, carveout;
    PdlShape(int cluster, int carveout = -1) : cluster(cluster), carveout(carveout) {}
};
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, PdlShape shape,
                       cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[3];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (shape.cluster > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = shape.cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (shape.carveout >= 0) {
        attr[n].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
        attr[n++].val.sharedMemCarveout = shape.carveout;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Clusters of this size resident at once (0: the query failed).
template <typename... Params>
int max_clusters(void (*kernel)(Params...), int threads, size_t smem, int cluster) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1024 * cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}

}  // namespace a2av
