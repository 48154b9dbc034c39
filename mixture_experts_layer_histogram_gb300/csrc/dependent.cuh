// Launching a kernel as a programmatic dependent of the one before it, and what such a kernel reads with.
#pragma once

#include "common.cuh"

namespace moe {

// Programmatic dependent launch. A kernel launched with launch_after() may start while the kernel before it in the
// stream still runs, once every block of that one has called start_next() (or ended); wait_previous()
// returns when it has completed and its writes are visible. A kernel that never calls start_next() lets its
// successor start at its end, as usual.
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
inline cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ld_stream for a kernel launched with launch_after(): the kernel before it may be writing *p while this one already lives
// (it reads after wait_previous()), and the non-coherent path is only for what nobody writes meanwhile.
__device__ __forceinline__ uint4 ld_stream_coherent(const uint4 *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

}  // namespace moe
