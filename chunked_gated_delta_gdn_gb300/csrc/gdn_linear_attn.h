// gdn_linear_attn.h -- launchers of linear attention with a decay for each head (not public).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// One pass of decayed linear attention over every (sequence n, value head h).  With
// gamma = exp(log_decay[h]) and X the K x V state, forwards in time
//   X_t = gamma X_{t-1} + s_in k_t v_t^T,      o_t = s_out X_t^T q_t,
// and, reverse != 0, backwards in time with the decay after the read-out (the adjoint order)
//   Y_t = X_{t+1} + s_in k_t v_t^T,  o_t = s_out Y_t^T q_t,  X_t = gamma Y_t.
// The backward is three such passes: dq reads (d_o, v, k), dv reads (k, q, d_o) and dk reads
// (v, d_o, q), the last two in reverse.  q, k, v, o here are the roles in the pass, each with
// its own head count (H / heads value heads share a row).
struct LinAttnPass {
  const void* q;             // [T, Hq, K]
  const void* k;             // [T, Hk, K]
  const void* v;             // [T, Hv, V]
  int Hq, Hk, Hv;
  int K, V;
  int H;                     // value heads of the operator (chains per sequence)
  const float* log_decay;    // [H]
  int B, T;                  // uniform rows; with cu_seqlens B = 1 and T the packed token count
  const int32_t* cu_seqlens;
  int num_seqs;
  const int32_t* state_indices;
  int num_slots;
  const float* initial;      // fp32 [N or slots, H, K, V] ([.., V, K] with initial_t), or NULL
  int initial_t;
  float* final_state;        // fp32 [N or slots, H, K, V], or NULL
  float s_in, s_out;
  int reverse;
  void* o;                   // [T, H, V]: io_dtype, or fp32 with o_f32
  int o_f32;
  int io_dtype;
  int* dev_status;
  cudaStream_t stream;
};

// Segments that each chain is cut into where there are too few to fill the GPU (1: none): by what
// the host knows, the chains of a launch, the most tokens that a sequence can have, the CTAs that
// run at a time, and the chunks that a segment needs to be worth its share of the two launches.
constexpr int kLaMaxPasses = 3, kLaMaxSegments = 16, kLaMinSegmentChunks = 4;
int linear_attn_segments(long long chains, long long most_tokens, int places, int min_chunks);
// How a run on the tensor cores is launched: the first `whole` chains uncut, in the first launch,
// the others in `segs` segments each (1: all whole, one launch).
struct LaPlan {
  long long whole;
  int segs;
};
// For `uniform` chains, all of most_tokens, the plan that would end first.
LaPlan linear_attn_plan(long long chains, long long most_tokens, bool uniform, int places);

// Up to three passes over the same sequences and heads, with the same product K V, in one launch.
// CUDA cores: fp32, any accepted head dims.  scratch: segs > 1: segs K V floats a chain and pass.
cudaError_t launch_linear_attn_generic(const LinAttnPass* passes, int num_passes, int segs, float* scratch);
// Its CTAs an SM (shared memory).
int linear_attn_generic_per_sm(int K, int V);
// Tensor cores: bf16 (o may be fp32), any accepted head dims.  scratch: segs > 1: segs 128 128
// floats a chain that is cut.
cudaError_t launch_linear_attn_tc(const LinAttnPass* passes, int num_passes, LaPlan plan, float* scratch);

// out[i][t, hq, :] = sum over the group's value heads of part[i][t, hq * group + j, :], i = 0, 1
// (fp32 in, io dtype out, heads added in order).
cudaError_t launch_linear_attn_fold(const float* const (&part)[2], void* const (&out)[2], long long T_total,
                                    int Hqk, int group, int D, int io_dtype, cudaStream_t stream);

struct LinAttnDecodeArgs {
  const void* q;             // [n, Hqk, K]
  const void* k;             // [n, Hqk, K]
  const void* v;             // [n, Hv, V]
  const float* log_decay;    // [Hv]
  float* state;              // [num_slots, Hv, K, V]
  int num_slots;
  const int32_t* batch_indices;
  int n, Hqk, Hv, K, V;
  int io_dtype;
  float scale;
  void* o;                   // [n, Hv, V]
  int* dev_status;
  cudaStream_t stream;
};
cudaError_t launch_linear_attn_decode(const LinAttnDecodeArgs& a);

}  // namespace gdn
