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
// overlaps.  `coop`: every block resident at once, or an error.
template <class... P, class... A>
cudaError_t launch_as(bool coop, void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                      A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[3];
  int n = 0;
  at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[n++].val.programmaticStreamSerializationAllowed = 1;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  if (coop) {
    at[n].id = cudaLaunchAttributeCooperative;
    at[n++].val.cooperative = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <class... P, class... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, A&&... args) {
  return launch_as(false, kern, grid, threads, smem, s, cluster, args...);
}

}  // namespace ctcpb
