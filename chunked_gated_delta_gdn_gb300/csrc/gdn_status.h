// gdn_status.h -- an entry point's status from the CUDA runtime's (not public).
#pragma once

#include <cuda_runtime.h>

#include "gdn.h"

namespace gdn {

// The runtime remembers an error of a call that it refused until someone asks for the last one.
// Every launch here asks, and would report an error of a call before it: so a refusal is returned
// once and forgotten.
inline gdn_status_t status_of(cudaError_t err) {
  if (err == cudaSuccess) return GDN_OK;
  cudaGetLastError();
  return GDN_ERR_CUDA;
}

}  // namespace gdn
