// Programmatic dependent launch: a kernel that may be brought up while the one before it on the
// stream still runs.
#pragma once
#include <cuda_runtime.h>

namespace rx {

// Waits for the kernels before this one to be complete and their writes visible.  Nothing that they
// may have written, and nothing that they may still read, is touched before it.
__device__ __forceinline__ void wait_for_predecessors() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next kernel be brought up (once every CTA of this one has said so or left).
__device__ __forceinline__ void let_successors_start() {
  asm volatile("griddepcontrol.launch_dependents;");
}

// Launches `kernel` that way.  Every kernel launched so calls wait_for_predecessors() in some
// thread: its own completion then says that everything before it is complete, too, which is what
// the next one's wait relies on.
template <class... P, class... A>
cudaError_t launch_beside(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) (void)cudaGetLastError();  // reported here, not by the caller's next check
  return e;
}

}  // namespace rx
