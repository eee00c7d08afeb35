// gdn_recurrence_bwd.cu -- gradients of the gated linear recurrence.
//
//     delta_t = dy_t + a_{t+1} delta_{t+1}   (the final state's gradient in place of the last term),
//     dx_t = delta_t,   d(log a_t) = delta_t a_t h_{t-1},   d h_0 = a_1 delta_1,
//
// and through the fused gates, with s = sqrt(1 - a^2) and u = sigmoid(i) x:
//     d(log a) = delta a (h_{t-1} - u a / s),   dr = d(log a) log a (1 - sigmoid(r)),
//     dx = delta s sigmoid(i),   di = delta s u (1 - sigmoid(i)),
//     dlam = sum of d(log a) sigmoid(r), times -c sigmoid(lam).
//
// One thread walks one channel of one sequence: forwards with the states into the workspace, then
// backwards.  Sequences' parts of dlam are added in order by a second launch.
#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

__global__ void recurrence_bwd_kernel(RecurrenceArgs a, float* states, float* part) {
  const int n = blockIdx.y, d = blockIdx.x * kThreads + threadIdx.x;
  const int total = a.cu_seqlens ? a.T : a.B * a.T;
  int bos = n * a.T, eos = bos + a.T, tail = total;
  bool bad = false;
  if (a.cu_seqlens) {
    bad = !packed_lengths_fit(a.cu_seqlens, a.num_seqs, a.T);
    if (bad && threadIdx.x == 0) report(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    bos = eos = 0;
    if (!bad && n < a.num_seqs) {
      bos = a.cu_seqlens[n];
      eos = a.cu_seqlens[n + 1];
    }
    tail = bad || !a.num_seqs ? 0 : n + 1 == a.num_seqs ? eos : total;
  }
  if (d >= a.D) return;
  for (int t = tail; t < total; ++t) {
    store_elem(a.dx, (size_t)t * a.D + d, 0.f, a.io_dtype);
    store_elem(a.dg, (size_t)t * a.D + d, 0.f, a.g_dtype);
    if (a.lam) store_elem(a.di, (size_t)t * a.D + d, 0.f, a.g_dtype);
  }
  if (n >= a.num_seqs) {
    if (part) part[d] = 0.f;
    return;
  }
  const size_t at = (size_t)n * a.D + d;
  if (bad) {
    if (a.d_initial_state) a.d_initial_state[at] = 0.f;
    if (part) part[at] = 0.f;
    return;
  }
  const float rate = a.lam ? gate_rate(a.c, a.lam[d], false) : 0.f;
  float h = a.initial_state ? a.initial_state[at] : 0.f;
  for (int t = bos; t < eos; ++t) {
    states[(size_t)t * a.D + d] = h;
    float la = load_elem(a.g, (size_t)t * a.g_pitch + d, a.g_dtype);
    float b = load_elem(a.x, (size_t)t * a.x_pitch + d, a.io_dtype);
    if (a.lam) {
      const FusedGate<false> f(la, load_elem(a.i, (size_t)t * a.i_pitch + d, a.g_dtype), rate);
      la = f.l;
      b *= f.s * f.si;
    }
    h = decayed(la, h, b);
  }
  float e = a.d_final_state ? a.d_final_state[at] : 0.f, sum = 0.f;
  for (int t = eos - 1; t >= bos; --t) {
    const size_t o = (size_t)t * a.D + d;
    const float g = load_elem(a.g, (size_t)t * a.g_pitch + d, a.g_dtype);
    const float x = load_elem(a.x, (size_t)t * a.x_pitch + d, a.io_dtype);
    const float delta = load_elem(a.dy, o, a.io_dtype) + e;
    float la = g;
    if (!a.lam) {
      e = decayed(la, delta, 0.f);
      store_elem(a.dx, o, delta, a.io_dtype);
      store_elem(a.dg, o, e * states[o], a.g_dtype);
    } else {
      const FusedGate<false> f(g, load_elem(a.i, (size_t)t * a.i_pitch + d, a.g_dtype), rate);
      e = decayed(f.l, delta, 0.f);
      const float u = f.si * x;
      // where nothing decays, s = 0 and what multiplies 1 / s below goes to 0 faster
      const float dla = e * (states[o] - (f.s > 0.f ? u * expf(f.l) / f.s : 0.f));
      sum += dla * f.sr;
      store_elem(a.dx, o, delta * f.s * f.si, a.io_dtype);
      store_elem(a.dg, o, dla * f.l * (1.f - f.sr), a.g_dtype);
      store_elem(a.di, o, delta * f.s * u * (1.f - f.si), a.g_dtype);
    }
  }
  if (a.d_initial_state) a.d_initial_state[at] = e;
  if (part) part[at] = sum;
}

__global__ void recurrence_dlam_kernel(RecurrenceArgs a, const float* part, int parts) {
  const int d = blockIdx.x * kThreads + threadIdx.x;
  if (d >= a.D) return;
  float sum = 0.f;
  for (int n = 0; n < parts; ++n) sum += part[(size_t)n * a.D + d];
  a.dlam[d] = sum * (-a.c * sigmoid_f(a.lam[d]));
}

}  // namespace

size_t recurrence_bwd_workspace_bytes(int B, int T, int D, int num_seqs, bool fused) {
  return ((size_t)B * T + (fused ? (num_seqs ? num_seqs : 1) : 0)) * D * sizeof(float);
}

cudaError_t launch_recurrence_bwd(const RecurrenceArgs& a) {
  const int parts = a.num_seqs ? a.num_seqs : 1;
  float* const states = static_cast<float*>(a.workspace);
  float* const part = a.dlam ? states + (size_t)a.B * a.T * a.D : nullptr;
  const unsigned blocks = (a.D + kThreads - 1) / kThreads;
  recurrence_bwd_kernel<<<dim3(blocks, parts), kThreads, 0, a.stream>>>(a, states, part);
  if (part) recurrence_dlam_kernel<<<blocks, kThreads, 0, a.stream>>>(a, part, parts);
  return cudaGetLastError();
}

}  // namespace gdn
