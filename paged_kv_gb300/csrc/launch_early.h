// Launches whose start overlaps the end of the stream's kernel before.
#pragma once

#include <cuda_runtime.h>

namespace pkv {

// Launches `kernel`, whose blocks may be placed as soon as all blocks of the kernel before
// it on the stream have ended or called launch_dependents().  Each of its blocks calls
// grid_dependency_wait() before it touches memory and before it ends: then that kernel has
// ended and what it wrote is seen, but by plain loads alone, not by the read-only path
// (__ldg), whose data may not change while a kernel runs.  After anything but a kernel it
// is a plain launch.
template <class Kernel, class... A>
cudaError_t launch_early(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(static_cast<unsigned>(threads));
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

}  // namespace pkv
