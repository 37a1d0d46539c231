// Launch of a kernel beside the one before it in the stream (programmatic dependent
// launch; the kernel waits with griddep_wait before it touches memory).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "tg_internal.h"

namespace tg {

// cluster > 1: thread-block clusters of that many.
template <class... P, class... A>
int launch_chained(void (*kern)(P...), int64_t blocks, int threads, size_t smem, int cluster,
                   cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

}  // namespace tg
