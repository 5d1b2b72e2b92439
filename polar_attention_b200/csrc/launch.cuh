// launch.cuh -- thread-block clusters and programmatic dependent launch: the
// device side's barriers and address mapping, and the host's launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace polar {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; shared-memory writes before it are seen after it.
// The instructions are for whole warps: a warp comes together first.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}
// The same shared-memory address in the cluster's CTA `rank` (generic).
template <typename T>
__device__ __forceinline__ const T *cluster_map(const T *p, uint32_t rank) {
    uint64_t r;
    asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
    return reinterpret_cast<const T *>(r);
}
// Programmatic dependent launch: waits until the kernels before this one on the
// stream are done and their writes visible (nothing to wait for otherwise).
__device__ __forceinline__ void wait_for_previous_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_kernel_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch with a cluster along x and, for a kernel that starts with
// wait_for_previous_kernel(), its launch overlapped with the kernel before.
template <typename... Args>
cudaError_t launch_ex(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, int cluster,
                      bool overlapped, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        ++n;
    }
    if (overlapped) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    c.attrs = at;
    c.numAttrs = n;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace polar
