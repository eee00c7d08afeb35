// gdn_group_norm.h -- launchers of group norm with an activation, channels last (not public).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "gdn.h"

namespace gdn {

struct GroupNormArgs {
  const void* x;       // [N, L, C] io_dtype
  const void* weight;  // [C] wb_dtype or NULL (1)
  const void* bias;    // [C] wb_dtype or NULL (0)
  const void* gate;    // [N, L, C] io_dtype or NULL
  int N, L, C, G;
  int io_dtype, wb_dtype;
  float eps;
  int act;             // GDN_ACT_NONE or GDN_ACT_SILU
  void* y;             // forward: [N, L, C] io_dtype
  float* mean;         // [N, G]: forward output (or NULL), backward input
  float* rstd;
  // backward
  const void* dy;      // [N, L, C] io_dtype
  void* dx;            // [N, L, C] io_dtype
  void* dgate;         // [N, L, C] io_dtype (with gate)
  float* dweight;      // [C] or NULL
  float* dbias;        // [C] or NULL
  void* workspace;
  cudaStream_t stream;
};

size_t group_norm_fwd_workspace_bytes(int N, int L, int C, int G, int io_dtype);
size_t group_norm_bwd_workspace_bytes(int N, int L, int C, int G, int io_dtype);
cudaError_t launch_group_norm_fwd(const GroupNormArgs& a);
cudaError_t launch_group_norm_bwd(const GroupNormArgs& a);

}  // namespace gdn
