// Launches of the sequence-block kernels.  Each is launched while the one before
// it on its stream still runs, sets itself up (indexes, barriers, tensor memory),
// and waits for that kernel's end, and so for all before it, where it first
// touches memory.  Loads of what another kernel may have written are coherent ones.
#pragma once

#include <cuda_runtime.h>

#include "host_common.h"

namespace lr {

// the stream's next kernel may be launched: of use once every block has passed here
__device__ __forceinline__ void next_may_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// every thread that touches memory passes here first
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: blocks of one, or 0 (or 1) for a kernel that has none or brings its own
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                          cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;  // a launch with a cluster's attribute takes 2 us longer
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  g_kernel_launches.fetch_add(1, std::memory_order_relaxed);
  return e;
}

}  // namespace lr
