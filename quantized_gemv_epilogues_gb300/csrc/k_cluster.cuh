// k_cluster.cuh - blocks of a thread-block cluster that share out one row: its
// barrier, stores to one another's shared memory, and the launch.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "mt_device.cuh"
#include "mt_internal.h"

namespace mt {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every block: what was written before an arrival (to any
// block's shared memory) is seen after the wait.  Blocks that have ended do not
// hold up the others.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores to the same place in the shared memory of the cluster's block `rank`.
__device__ __forceinline__ void cluster_put(uint64_t* p, uint32_t rank, uint64_t v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// launch() with clusters of `size` blocks along x (grid.x is a multiple of it).
template <typename... KArgs, typename... Args>
mt_status launch_cluster(void (*kernel)(KArgs...), int size, dim3 grid, dim3 block, size_t smem, const Launch& l, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = l.pdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  return e == cudaSuccess ? MT_OK : cuda_fail(e);
}

}  // namespace mt
