// Process-wide launch counter, optional per-launch CUDA-event timing, and the
// launch helper every kernel launch of the library goes through.
#pragma once
#include <cuda_runtime.h>

#include <utility>

#include "moe_internal.h"

namespace moe {

// Bracket one kernel launch: counts it and, when profiling is enabled,
// records a CUDA event before and after it on the launch stream.
class Prof {
 public:
  Prof(const char* name, cudaStream_t s);
  ~Prof();
  Prof(const Prof&) = delete;
  Prof& operator=(const Prof&) = delete;

 private:
  const char* name_;
  cudaStream_t s_;
  cudaEvent_t a_ = nullptr, b_ = nullptr;
};

// Launch `kern` with the given shape on `s` through cudaLaunchKernelEx and
// note its return code in the calling entry point's error slot.
template <typename... Kp, typename... Ar>
inline void launch_kernel(const char* name, void (*kern)(Kp...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                          Ar&&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  Prof prof(name, s);
  note(cudaLaunchKernelEx(&lc, kern, std::forward<Ar>(args)...));
}

// The same, for a kernel that orders itself after the stream's previous kernel
// with griddepcontrol.wait: it may be placed while that one still runs. `cluster`
// blocks of the grid form a cluster.
template <typename... Kp, typename... Ar>
inline void launch_cluster_after(const char* name, void (*kern)(Kp...), dim3 grid, int cluster, dim3 block, size_t smem,
                                 cudaStream_t s, Ar&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = cluster > 1 ? 2 : 1;
  Prof prof(name, s);
  note(cudaLaunchKernelEx(&lc, kern, std::forward<Ar>(args)...));
}
template <typename... Kp, typename... Ar>
inline void launch_kernel_after(const char* name, void (*kern)(Kp...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t s, Ar&&... args) {
  launch_cluster_after(name, kern, grid, 1, block, smem, s, std::forward<Ar>(args)...);
}

}  // namespace moe
