// zp_launch.h — launches of the kernels that a step makes once per layer.
//
// On a stream of short kernels the time between the end of one and the start of the next is as long as
// the kernels (256 tokens' rotary positions: 3.4 us of GPU time, 5.6 us a call on a stream).  So these
// kernels are launched with programmatic stream serialization: the next one's CTAs come in as soon as
// all of the one before have begun, and wait on the device (after_previous) until it is complete
// and its writes are visible.  Every thread waits before its first access to global memory and before
// it returns, so a kernel that is complete stands for all before it, and the order on the stream is what
// it was; after a kernel without next_may_start the wait is for its end, as ever.
#pragma once

#include <cuda_runtime.h>

namespace zp {

// First in a kernel (before any access to global memory, and on every path).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's CTAs may come in when every CTA has passed this.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_in_order(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attrs[2]{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
}

}  // namespace zp
