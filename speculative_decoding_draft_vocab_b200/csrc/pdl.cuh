// Programmatic dependent launches: a kernel is scheduled while the one before it on the
// stream runs and waits for it (pdl_wait) before it reads or writes anything.  Every kernel
// of such a chain waits, so a chain's last kernel has them all behind it.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace dspark {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;"); }

struct PdlLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  PdlLaunch(int64_t grid, int threads, size_t smem, cudaStream_t s, int cluster = 1) {
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cluster > 1) {
      at[1].id = cudaLaunchAttributeClusterDimension;
      at[1].val.clusterDim.x = unsigned(cluster);
      at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
    }
  }
};

}  // namespace dspark
