// Dynamic shared memory above 48 KB has to be allowed for a kernel once on each
// device that runs it.
#pragma once

#include <cuda_runtime.h>

namespace tpmlp {

template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static bool done[64] = {};  // only ever set, by calls that agree
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

// A kernel whose warps exchange registers waits forever if it was not launched
// with as many as they take together: refused then.  Looked up once.
template <auto Kernel>
cudaError_t check_regs(int threads, int needed) {
  static int regs = 0;  // only ever set to one value
  if (!regs) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, Kernel);
    if (e != cudaSuccess) return e;
    regs = a.numRegs;
  }
  return regs * threads >= needed ? cudaSuccess : cudaErrorLaunchOutOfResources;
}

}  // namespace tpmlp
