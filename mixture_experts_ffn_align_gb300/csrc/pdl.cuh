// Programmatic dependent launch for the training and 4-bit operators: each of
// their kernels may be scheduled while the kernel before it on the stream still
// runs, sets itself up (barriers, tensor memory), and waits for that kernel's
// completion before its first access to global memory.  Small calls follow one
// another a few microseconds apart, and the set-up is much of that.
//
// Every thread block of every such kernel executes griddep_wait, so the
// completion of one implies that of all kernels before it.
//
// Kernels of clusters keep the ordinary order, before and after: on SM pairs, and
// while their tail waits (ragged_pair.cuh) were missing too, about one in
// 10,000 launches did not end, and no overlap is worth that.  The long ones would gain
// 2 of some hundred microseconds, sliced products and the update's launch of small
// matrices (55 us and more) as much of less.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace moe {

// Lets the next kernel's blocks be scheduled as soon as all of this kernel's run.
__device__ __forceinline__ void griddep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Waits until the kernel before has completed and its writes are visible.
__device__ __forceinline__ void griddep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches kernel<<<grid, block, smem, stream>>>(args...) with that permission,
// or, cluster > 1, in the ordinary order and with clusters of so many CTAs along x.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream, unsigned cluster, A&&... args) {
  cudaLaunchAttribute attr[1];
  if (cluster > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(std::forward<A>(args))...);
}

}  // namespace moe
