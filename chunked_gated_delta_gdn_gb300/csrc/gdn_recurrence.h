// gdn_recurrence.h -- launchers of the gated linear recurrence (not public).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// Tokens from one saved state to the next (`carries`): the state that enters token 32 m of the flat
// token axis, for every m.  The backward starts there.
constexpr int kRecCarry = 32;

struct RecurrenceArgs {
  const void* x;        // [tokens, D] io_dtype, rows x_pitch apart
  const void* g;        // the log-decay, or with lam the recurrence gate r; g_dtype, rows g_pitch apart
  const void* i;        // the input gate, with lam; g_dtype, rows i_pitch apart
  const float* lam;     // [D] or NULL: gates given
  float c;
  long long x_pitch, g_pitch, i_pitch;
  int B, T, D;
  int io_dtype, g_dtype;
  const float* initial_state;   // [N, D], or the slots [num_slots, D]; NULL: zero
  float* final_state;           // likewise; NULL: not wanted
  const int32_t* cu_seqlens;    // NULL: rows of T tokens
  int num_seqs;                 // N
  const int32_t* state_indices;
  int num_slots;
  void* y;                      // [tokens, D] io_dtype; NULL: carries alone
  float* carries;               // [ceil(tokens / kRecCarry), D] or NULL
  // backward
  const void* dy;               // [tokens, D] io_dtype
  const float* d_final_state;   // [N, D] or NULL
  void* dx;                     // [tokens, D] io_dtype
  void* dg;                     // [tokens, D] g_dtype
  void* di;                     // [tokens, D] g_dtype, with lam
  float* dlam;                  // [D] or NULL
  float* d_initial_state;       // [N, D] or NULL
  void* workspace;              // (forward: segments' steps and states; backward: more)
  // decode
  float* state;                 // [num_slots, D]
  const int32_t* batch_indices; // [n] or NULL
  int n;
  int* dev_status;
  cudaStream_t stream;
};

// The forward's launch that makes a backward's carries again.  What goes wrong in it is the caller's to know: wrong
// carries are wrong gradients, and the backward's own kernel cannot tell.
inline RecurrenceArgs carries_again(const RecurrenceArgs& a, float* carries, void* workspace) {
  RecurrenceArgs f = a;
  f.carries = carries;
  f.workspace = workspace;
  f.y = nullptr;
  return f;
}

size_t recurrence_carries_bytes(long long tokens, int D);
size_t recurrence_fwd_workspace_bytes(int B, int T, int D, int num_seqs);
size_t recurrence_bwd_workspace_bytes(int B, int T, int D, int num_seqs, bool fused);
cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a);
cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a);
cudaError_t launch_recurrence_decode(const RecurrenceArgs& a);

}  // namespace gdn
