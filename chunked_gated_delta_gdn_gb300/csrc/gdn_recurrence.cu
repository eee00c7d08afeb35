// gdn_recurrence.cu -- the gated linear recurrence: forward and single-token decode.
//
//     h_t = a_t h_{t-1} + b_t   per channel, with a_t = exp(g_t), b_t = x_t, or
//     a_t = exp(-c softplus(lam) sigmoid(r_t)),  b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t.
//
// One thread walks one channel of one sequence.
#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

__global__ void recurrence_fwd_kernel(RecurrenceArgs a) {
  const int n = blockIdx.y, d = blockIdx.x * kThreads + threadIdx.x;
  const int total = a.cu_seqlens ? a.T : a.B * a.T;
  int bos = n * a.T, eos = bos + a.T, tail = total;
  bool n_ok = n < a.num_seqs;
  if (a.cu_seqlens) {
    const bool bad = !packed_lengths_fit(a.cu_seqlens, a.num_seqs, a.T);
    if (bad && threadIdx.x == 0) report(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    n_ok = n_ok && !bad;
    bos = n_ok ? a.cu_seqlens[n] : 0;
    eos = n_ok ? a.cu_seqlens[n + 1] : 0;
    tail = bad ? (n == 0 ? 0 : total) : n + 1 >= a.num_seqs ? eos : total;
  }
  if (d >= a.D) return;
  bool mute = false;
  int slot = n;
  if (a.state_indices && n_ok) {
    slot = a.state_indices[n];
    mute = slot < 0 || slot >= a.num_slots;
    if (mute && slot != -1 && d == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
  }
  if (tail < total && a.y)
    for (int t = tail; t < total; ++t) store_elem(a.y, (size_t)t * a.D + d, 0.f, a.io_dtype);
  if (!n_ok) return;
  const size_t at = (size_t)slot * a.D + d;
  float h = !mute && a.initial_state ? a.initial_state[at] : 0.f;
  const float rate = a.lam ? -a.c * softplus_f(a.lam[d]) : 0.f;
  for (int t = bos; t < eos; ++t) {
    if (a.carries && t % kRecCarry == 0) a.carries[(size_t)(t / kRecCarry) * a.D + d] = h;
    float la = load_elem(a.g, (size_t)t * a.g_pitch + d, a.g_dtype);
    float b = load_elem(a.x, (size_t)t * a.x_pitch + d, a.io_dtype);
    if (a.lam) {
      const FusedGate f = fused_gate(la, load_elem(a.i, (size_t)t * a.i_pitch + d, a.g_dtype), rate);
      la = f.la;
      b *= f.s * f.si;
    }
    h = decayed(la, h, b);
    if (a.y) store_elem(a.y, (size_t)t * a.D + d, mute ? 0.f : h, a.io_dtype);
  }
  if (a.final_state && !mute) a.final_state[at] = h;
}

__global__ void recurrence_decode_kernel(RecurrenceArgs a) {
  const int n = blockIdx.y, d = blockIdx.x * kThreads + threadIdx.x;
  if (d >= a.D) return;
  const int slot = a.batch_indices ? a.batch_indices[n] : n;
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1 && d == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
    store_elem(a.y, (size_t)n * a.D + d, 0.f, a.io_dtype);
    return;
  }
  float la = load_elem(a.g, (size_t)n * a.g_pitch + d, a.g_dtype);
  float b = load_elem(a.x, (size_t)n * a.x_pitch + d, a.io_dtype);
  if (a.lam) {
    const FusedGate f = fused_gate(la, load_elem(a.i, (size_t)n * a.i_pitch + d, a.g_dtype), -a.c * softplus_f(a.lam[d]));
    la = f.la;
    b *= f.s * f.si;
  }
  float* const state = a.state + (size_t)slot * a.D + d;
  const float h = decayed(la, *state, b);
  *state = h;
  store_elem(a.y, (size_t)n * a.D + d, h, a.io_dtype);
}

}  // namespace

size_t recurrence_carries_bytes(long long tokens, int D) {
  return (size_t)((tokens + kRecCarry - 1) / kRecCarry) * D * sizeof(float);
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
  const dim3 grid((a.D + kThreads - 1) / kThreads, a.num_seqs ? a.num_seqs : 1);
  recurrence_fwd_kernel<<<grid, kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_recurrence_decode(const RecurrenceArgs& a) {
  recurrence_decode_kernel<<<dim3((a.D + kThreads - 1) / kThreads, a.n), kThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
