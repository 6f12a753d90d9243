// pdl.cuh -- programmatic dependent launch: a kernel may be set up while the one before it
// on the stream still runs, and waits for that one's end (and its writes) in pdl_wait().
// Every kernel launched this way calls pdl_wait() before it touches global memory, but for two of the shared prefix:
// own_slots_kernel, where a prefix launch stands in front of it, and what shared_join_kernel reads of the lengths.  They
// may, because that launch's CTAs call pdl_wait() before pdl_launch(): once own_slots_kernel runs, all that came before
// the call is complete (it waits itself before it ends, so that its end still stands for the prefix's).
#pragma once

#include <cuda_runtime.h>

namespace kvc {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may be set up once every CTA has got here.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_pdl_cluster(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st,
                               int cluster, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st, A &&...args) {
  return launch_pdl_cluster(kernel, grid, threads, smem, st, 0, args...);
}

}  // namespace kvc
