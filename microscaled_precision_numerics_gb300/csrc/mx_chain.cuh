// mx_chain.cuh -- launches of a generation step's kernels one behind the other: each may be set up on the device while the one
// before it in the stream still runs (programmatic stream serialization), since every CTA of these kernels waits for the
// earlier grid's completion before it touches memory.  A kernel without chain_begin() must not be launched this way.
#pragma once

#include <cuda_runtime.h>

namespace mxk {

// First statement of the kernel that comes before any access to global memory, in every thread of every CTA: lets the next
// kernel of the stream be set up, then waits until the ones before have completed and their writes are visible.
__device__ __forceinline__ void chain_begin() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A load that stays behind chain_begin(): through the read-only path (__ldg, restrict pointers) it need not, as that
// path takes what it reads as unchanged for as long as the kernel is on the device.
template <typename T>
__device__ __forceinline__ T load_global(const T* p) {
    return *p;
}

// cluster 0: a launch without clusters.
template <typename... Params, typename... Args>
inline cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                                  cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {cluster, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace mxk
