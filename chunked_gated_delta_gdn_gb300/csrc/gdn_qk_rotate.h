// gdn_qk_rotate.h -- launchers of the norm of queries and keys with rotation (not public).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// Queries or keys.
struct QkSide {
  const void* x;           // [B, T, H, K] io_dtype with these strides, in elements
  long long sb, st, sh;
  int H;
  const void* w;           // [K] w_dtype or NULL (1)
  void* out;               // [B, T, H, K]: forward y, backward dx
  const void* dy;          // [B, T, H, K]
  float* dw;               // [K] or NULL
};

struct QkRotateArgs {
  QkSide side[2];
  int B, T, K, R;
  int io_dtype, w_dtype;
  int norm;
  float eps;
  const float* inv_freq;     // [R / 2]
  const int32_t* positions;  // [num_axes, B, T] or NULL
  int num_axes;
  int axis_end[GDN_MAX_AXES];  // pairs below axis_end[0] turn by axis 0, below axis_end[1] by axis 1 ...
  int interleaved;
  void* workspace;
  cudaStream_t stream;
};

size_t qk_rotate_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int K, bool need_weights);
cudaError_t launch_qk_rotate_fwd(const QkRotateArgs& a);
cudaError_t launch_qk_rotate_bwd(const QkRotateArgs& a);

}  // namespace gdn
