// Launches of the many-token operators: programmatic dependent launch, and an
// optional cluster size.
//
// Each of these kernels lets its successor start as soon as all its own blocks
// run (pdl_launch_dependents) and touches global memory only after pdl_wait, in
// every block, so that whatever stands before it on the stream is complete and
// visible first, and the same holds for any kernel behind it that waits for it.
// What a kernel does before that (barriers, tensor memory, its parameters)
// overlaps the end of its predecessor: about 2 us per launch in a chain.
#pragma once
#include <cuda_runtime.h>

namespace tern {

template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), int grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                     A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

}  // namespace tern
