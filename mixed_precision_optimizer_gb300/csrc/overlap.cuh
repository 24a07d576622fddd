// Launches whose start overlaps the end of the kernel before them
// (programmatic dependent launch).  A kernel launched by launch_overlapped may
// begin while its predecessor on the stream still runs, as soon as every CTA of
// the predecessor has called let_next_start() or left; it calls
// wait_for_predecessors() before it touches global memory (its parameters and
// tensor maps are not global memory), which returns once the predecessors have
// completed and their writes are visible.  So a kernel's launch, its barriers
// and its TMEM allocation overlap what is left of the kernel before, and
// nothing else changes: behind a kernel that never calls let_next_start() the
// order is the ordinary one.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mpopt {
namespace {

__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void wait_for_predecessors() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs to a cluster, or 0 for the kernel's own (none, or __cluster_dims__).
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              int cluster, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace mpopt
