// Host helpers of the one-dimensional launches (scoring, head, embedding).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "vsamp.h"

namespace vsamp {

// CTAs of a launch over n blocks of work; the kernels stride over what is beyond it.
inline unsigned grid_of(int64_t n) { return (unsigned)(n < 0x3FFFFFFFLL ? n : 0x3FFFFFFFLL); }

// A launch that may be set up while the stream's previous kernel drains; the kernel begins with begin_overlapped(), which
// waits for that kernel's writes before any memory is touched. Back-to-back calls save about a microsecond each.
template <typename... KArgs, typename... Args>
vsamp_status launch_1d(void (*kern)(KArgs...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  return VSAMP_OK;
}

// The same for clusters of `cluster` CTAs (at most 8).
template <typename... KArgs, typename... Args>
vsamp_status launch_clusters(void (*kern)(KArgs...), unsigned grid, unsigned cluster, unsigned threads, size_t smem,
                             cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return VSAMP_ERR_CUDA;
  }
  return VSAMP_OK;
}

}  // namespace vsamp
