// launch.cuh -- launches whose start-up overlaps the end of the kernel before them in the stream.
//
// A call here is a chain of short kernels, and each ordinary boundary costs a launch latency. A
// kernel of the chain says at its start that the next one may be set up (dep_launch), and every
// thread of every kernel waits for the whole grid before it, results included (dep_wait), before
// it reads or writes global memory or leaves. A kernel of the caller's on either side is
// ordered as usual: one that says nothing is waited for to its end.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace relay {
namespace {

__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Streaming load of 16 bytes. Not the read-only path: a kernel here may start before the one that
// writes what it reads has ended.
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
// One value, fp32 or bf16, for the same reason.
__device__ __forceinline__ float ld_value(const float* p) { return *p; }
__device__ __forceinline__ float ld_value(const uint32_t* p) { return __uint_as_float(*p); }
__device__ __forceinline__ float ld_value(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

template <class... Params, class... Args>
cudaError_t launch_chained_clusters(void (*kernel)(Params...), int cluster, dim3 grid, int threads, size_t smem,
                                    cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(std::forward<Args>(args))...);
}
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                           Args&&... args) {
  return launch_chained_clusters(kernel, 1, grid, threads, smem, stream, std::forward<Args>(args)...);
}

}  // namespace
}  // namespace relay
