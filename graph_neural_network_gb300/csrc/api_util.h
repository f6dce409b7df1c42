// Checks and conversions shared by the C-ABI entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gnnagg.h"

namespace gnn {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// The status of a call's launches.  A refused one (cudaLaunchKernelEx, an attribute) also
// stays as the thread's last error, which the next call's cudaGetLastError would take for
// its own: it is taken here.
inline gnn_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return GNN_OK;
  (void)cudaGetLastError();
  return GNN_ERR_CUDA;
}

inline bool current_sms(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

}  // namespace gnn
