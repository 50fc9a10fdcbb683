// Shared by the label head's kernels (layer norm, log-probabilities, cross
// entropy): limits and includes.
#pragma once

#include "ctcpb_kernels.h"
#include "ctcpb_mma.cuh"

namespace ctcpb {

typedef unsigned short u16;

constexpr long long kHeadMaxRows = 1 << 24;  // rows (frames) of a call
constexpr int kHeadMaxWidth = 8192;         // features of a row

// A launch that may begin while the one before it on the stream ends: each
// kernel waits for that (pdl_wait) before it touches memory, so only its set-up
// overlaps.
template <class... P, class... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace ctcpb
