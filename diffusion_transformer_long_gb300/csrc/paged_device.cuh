// What the paged-cache kernels share: programmatic launch order, and loads under it.
#pragma once

#include <cuda_runtime.h>

namespace ditattn {

// The kernels are launched as programmatic dependents: the stream's next kernel is made ready while
// the last one runs and starts when its blocks have all ended, 0.5 to 1 us sooner than otherwise, or
// as soon as the last kernel, whoever's it is, lets its successors start.  They read and write memory
// only behind this wait for that kernel's end.  (None of them lets its own successor start any earlier:
// that gained nothing more.)
//
// What a kernel before may have written is read by ordinary loads, never through the read-only path
// (__ldg, ld.global.nc): that one is for data that stays as it is for as long as this kernel is on the
// GPU, which begins before the wait, and neither the compiler nor the cache has to order it behind.
// (Lengths, tables and queries read that way were once seen stale behind a kernel that started its
// successors early; by ordinary loads none is, cluster launches with the attribute included.)
__device__ __forceinline__ void wait_for_inputs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The same, for a kernel whose inputs are also copied by TMA.
__device__ __forceinline__ void wait_for_inputs_and_copies() {
  wait_for_inputs();
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

// 16 bytes that are read once (evicted first); volatile: not before the wait.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 x;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(__cvta_generic_to_global(p)));
  return x;
}

// kClusterSize > 1: blocks of a cluster.  Such a launch waits for the stream in the ordinary way.
template <int kClusterSize = 1, typename K, typename... Args>
cudaError_t launch_after(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (kClusterSize > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kClusterSize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ditattn
