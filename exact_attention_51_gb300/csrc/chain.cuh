// Launches that overlap the end of the launch before them.
//
// A serving step runs kernels of a few microseconds one after another, and a
// plain launch begins only when the one before it has ended: 4.1 us from one to
// the next on GB300, whatever they do.  With programmatic stream
// serialization a kernel's blocks are placed while the one before still runs, and
// wait (chain_begin) until it has completed and its writes can be seen.
//
// Every thread of every block of a kernel launched this way calls chain_begin
// before it reads or writes global memory or leaves: so a kernel completes only
// after all that were launched before it, and what follows it, launched either
// way, sees their results.
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace ea51 {

// Waits for the launches before this one; then lets the next one's blocks be placed, as
// far as this one's leave room for them.
__device__ __forceinline__ void chain_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// kern<<<grid, block, smem, stream>>>(args...) with blocks placed early, in clusters of
// `cluster` along x.
template <typename... Params, typename... Args>
cudaError_t chain_launch(void (*kern)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                         unsigned cluster, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace ea51
