// Host helpers of the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

namespace sv {

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A plain launch that may start while the preceding kernel on the stream
// drains (programmatic dependent launch).  Only for kernels that call
// wait_for_preceding_grid() before their first memory access; without the
// attribute (refused) it falls back to plain stream order.
inline cudaError_t launch_early(const void* fn, dim3 grid, dim3 block, void** args, cudaStream_t st,
                                size_t shared = 0, unsigned cluster = 1) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cfg.dynamicSmemBytes = shared;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    cfg.attrs = attr + 1;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    e = cudaLaunchKernelExC(&cfg, fn, args);
  }
  return e;
}

}  // namespace sv
