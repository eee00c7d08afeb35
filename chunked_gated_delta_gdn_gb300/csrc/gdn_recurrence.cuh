// gdn_recurrence.cuh -- what the kernels of the gated linear recurrence share: the gates and their
// derivatives, the check of packed lengths.
#pragma once

#include "gdn_common.cuh"
#include "gdn_launch.cuh"
#include "gdn_recurrence.h"

namespace gdn {
namespace {

// One token of one channel with gates from r and i: log a = la, and what is added to the state,
// s sigmoid(i) x with s = sqrt(1 - a^2).
struct FusedGate {
  float la, sr, si, s;
};
__device__ __forceinline__ FusedGate fused_gate(float r, float i, float minus_c_softplus) {
  FusedGate f;
  f.sr = sigmoid_f(r);
  f.si = sigmoid_f(i);
  f.la = minus_c_softplus * f.sr;
  f.s = sqrtf(-expm1f(2.f * f.la));
  return f;
}

// a h + b, a = exp(la), without the error that rounding a makes in the same direction at every token
// of a long memory (1 - a to 24 bits instead of a); short memories take a itself, as h + (a - 1) h
// would lose what is left of h there.
__device__ __forceinline__ float decayed(float la, float h, float b) {
  if (la < -0.7f) return fmaf(expf(la), h, b);
  return h + fmaf(expm1f(la), h, b);
}

// Whether cu_seqlens [N + 1] starts at 0 and rises to at most T; called by every thread of the CTA.
__device__ __forceinline__ bool packed_lengths_fit(const int32_t* cu, int N, int T) {
  int bad = 0;
  for (int n = threadIdx.x; n <= N; n += blockDim.x) {
    const int at = cu[n];
    bad |= at > T || at < (n == 0 ? 0 : cu[n - 1]) || (n == 0 && at != 0);
  }
  return __syncthreads_or(bad) == 0;
}

}  // namespace
}  // namespace gdn
