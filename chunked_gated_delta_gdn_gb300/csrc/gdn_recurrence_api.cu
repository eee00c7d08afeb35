// gdn_recurrence_api.cu -- the extern "C" entry points of the gated linear recurrence: argument
// validation and dispatch.  Declarations and the contract are in gdn.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_recurrence.h"
#include "gdn_status.h"

namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem_size(int d) { return d == GDN_BF16 ? 2 : 4; }
constexpr int kMaxChannels = 1 << 28;   // (a row's bytes are counted in 32 bits)
constexpr int kMaxPacked = 1 << 30;     // packed sequences (the search for one halves sums of two counts in 32 bits)
bool is_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }

// Sizes, and the gates' form: lam and i come together.
gdn_status_t check(const void* x, const void* g, const void* i, const float* lam, float c, long long x_pitch,
                   long long g_pitch, long long i_pitch, long long tokens, int D, int io_dtype, int g_dtype) {
  if (!is_dtype(io_dtype) || !is_dtype(g_dtype) || (g_dtype != GDN_F32 && g_dtype != io_dtype))
    return GDN_ERR_DTYPE;
  if (D <= 0 || D > kMaxChannels || tokens < 0 || tokens > 0x7fff0000LL) return GDN_ERR_SHAPE;
  if (tokens > 0 && (x_pitch < D || g_pitch < D || (lam && i_pitch < D))) return GDN_ERR_SHAPE;
  if (lam && !(c >= 0.f && c <= 3.0e38f)) return GDN_ERR_SHAPE;
  if (tokens > 0 && (!x || !g || (lam && !i))) return GDN_ERR_NULL;
  if (!lam && i) return GDN_ERR_NULL;
  if (!aligned_to(x, elem_size(io_dtype)) || !aligned_to(g, elem_size(g_dtype)) ||
      !aligned_to(i, elem_size(g_dtype)) || !aligned_to(lam, 4))
    return GDN_ERR_LAYOUT;
  return GDN_OK;
}

gdn_status_t check_batch(int B, int T, const int32_t* cu_seqlens, int num_seqs, const int32_t* state_indices,
                         int* N) {
  if (B < 0 || T < 0 || num_seqs < 0) return GDN_ERR_SHAPE;
  if (cu_seqlens && (B != 1 || num_seqs > kMaxPacked)) return GDN_ERR_SHAPE;
  *N = cu_seqlens ? num_seqs : B;
  if (!aligned_to(cu_seqlens, 4) || !aligned_to(state_indices, 4)) return GDN_ERR_LAYOUT;
  return GDN_OK;
}

// The sizes of a question for scratch, whose num_seqs is B where sequences are rows.
bool sizes_fit(int B, int T, int D, int num_seqs) {
  return B >= 0 && T >= 0 && D > 0 && D <= kMaxChannels && num_seqs >= 0 && (num_seqs <= kMaxPacked || num_seqs == B) &&
         (long long)B * T <= 0x7fff0000LL;
}

}  // namespace

extern "C" {

size_t gdn_linear_recurrence_carries_size(int B, int T, int D) {
  if (!sizes_fit(B, T, D, 0)) return (size_t)-1;
  return gdn::recurrence_carries_bytes((long long)B * T, D);
}

size_t gdn_linear_recurrence_fwd_workspace_size(int B, int T, int D, int num_seqs) {
  if (!sizes_fit(B, T, D, num_seqs)) return (size_t)-1;
  return gdn::recurrence_fwd_workspace_bytes(B, T, D, num_seqs);
}

gdn_status_t gdn_linear_recurrence_fwd(const void* x, const void* g, const void* i, const float* lam, float c,
                                       long long x_pitch, long long g_pitch, long long i_pitch, int B, int T,
                                       int D, gdn_dtype_t io_dtype, gdn_dtype_t g_dtype,
                                       const float* initial_state, int output_final_state, float* final_state,
                                       const int32_t* cu_seqlens, int num_seqs, const int32_t* state_indices,
                                       int num_slots, void* y, float* carries, void* workspace,
                                       size_t workspace_bytes, int* dev_status, void* stream) {
  int N = 0;
  gdn_status_t st = check_batch(B, T, cu_seqlens, num_seqs, state_indices, &N);
  if (st != GDN_OK) return st;
  const long long tokens = (long long)B * T;
  st = check(x, g, i, lam, c, x_pitch, g_pitch, i_pitch, tokens, D, io_dtype, g_dtype);
  if (st != GDN_OK) return st;
  if (state_indices && (num_slots <= 0 || (!initial_state && !output_final_state))) return GDN_ERR_SHAPE;
  if (output_final_state && !final_state && N > 0) return GDN_ERR_NULL;
  if (tokens > 0 && !y && !carries) return GDN_ERR_NULL;
  if (!aligned_to(y, elem_size(io_dtype)) || !aligned_to(initial_state, 4) || !aligned_to(final_state, 4) ||
      !aligned_to(carries, 4))
    return GDN_ERR_LAYOUT;
  if (N == 0 && tokens == 0) return GDN_OK;
  const size_t need = gdn::recurrence_fwd_workspace_bytes(B, T, D, N);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return GDN_ERR_LAYOUT;
  }
  gdn::RecurrenceArgs a{};
  a.x = x; a.g = g; a.i = i; a.lam = lam; a.c = c;
  a.x_pitch = x_pitch; a.g_pitch = g_pitch; a.i_pitch = i_pitch;
  a.B = B; a.T = T; a.D = D;
  a.io_dtype = io_dtype; a.g_dtype = g_dtype;
  a.initial_state = initial_state;
  a.final_state = output_final_state ? final_state : nullptr;
  a.cu_seqlens = cu_seqlens;
  a.num_seqs = N;
  a.state_indices = state_indices;
  a.num_slots = num_slots;
  a.y = y;
  a.carries = carries;
  a.workspace = workspace;
  a.dev_status = dev_status;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return gdn::status_of(gdn::launch_recurrence_fwd(a));
}

size_t gdn_linear_recurrence_bwd_workspace_size(int B, int T, int D, int num_seqs, int fused_gates) {
  if (!sizes_fit(B, T, D, num_seqs)) return (size_t)-1;
  return gdn::recurrence_bwd_workspace_bytes(B, T, D, num_seqs, fused_gates != 0);
}

gdn_status_t gdn_linear_recurrence_bwd(const void* x, const void* g, const void* i, const float* lam, float c,
                                       long long x_pitch, long long g_pitch, long long i_pitch, int B, int T,
                                       int D, gdn_dtype_t io_dtype, gdn_dtype_t g_dtype,
                                       const float* initial_state, const int32_t* cu_seqlens, int num_seqs,
                                       const void* d_y, const float* d_final_state, const float* carries,
                                       void* dx, void* dg, void* di, float* dlam, float* d_initial_state,
                                       void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  int N = 0;
  gdn_status_t st = check_batch(B, T, cu_seqlens, num_seqs, nullptr, &N);
  if (st != GDN_OK) return st;
  const long long tokens = (long long)B * T;
  st = check(x, g, i, lam, c, x_pitch, g_pitch, i_pitch, tokens, D, io_dtype, g_dtype);
  if (st != GDN_OK) return st;
  if (tokens > 0 && (!d_y || !dx || !dg || (lam && !di))) return GDN_ERR_NULL;
  if (!lam && (di || dlam)) return GDN_ERR_NULL;
  if (!aligned_to(d_y, elem_size(io_dtype)) || !aligned_to(dx, elem_size(io_dtype)) ||
      !aligned_to(dg, elem_size(g_dtype)) || !aligned_to(di, elem_size(g_dtype)) || !aligned_to(dlam, 4) ||
      !aligned_to(initial_state, 4) || !aligned_to(d_final_state, 4) || !aligned_to(d_initial_state, 4) ||
      !aligned_to(carries, 4))
    return GDN_ERR_LAYOUT;
  if (N == 0 && tokens == 0 && !dlam) return GDN_OK;
  const size_t need = gdn::recurrence_bwd_workspace_bytes(B, T, D, N, lam != nullptr);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return GDN_ERR_LAYOUT;
  }
  gdn::RecurrenceArgs a{};
  a.x = x; a.g = g; a.i = i; a.lam = lam; a.c = c;
  a.x_pitch = x_pitch; a.g_pitch = g_pitch; a.i_pitch = i_pitch;
  a.B = B; a.T = T; a.D = D;
  a.io_dtype = io_dtype; a.g_dtype = g_dtype;
  a.initial_state = initial_state;
  a.cu_seqlens = cu_seqlens;
  a.num_seqs = N;
  a.carries = const_cast<float*>(carries);
  a.dy = d_y;
  a.d_final_state = d_final_state;
  a.dx = dx; a.dg = dg; a.di = di; a.dlam = dlam;
  a.d_initial_state = d_initial_state;
  a.workspace = workspace;
  a.dev_status = dev_status;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return gdn::status_of(gdn::launch_recurrence_bwd(a));
}

gdn_status_t gdn_linear_recurrence_decode(const void* x, const void* g, const void* i, const float* lam, float c,
                                          long long x_pitch, long long g_pitch, long long i_pitch, int n, int D,
                                          gdn_dtype_t io_dtype, gdn_dtype_t g_dtype, float* state, int num_slots,
                                          const int32_t* batch_indices, void* y, int* dev_status,
                                          void* stream) {
  if (n < 0 || num_slots < 0 || (!batch_indices && n > num_slots)) return GDN_ERR_SHAPE;
  gdn_status_t st = check(x, g, i, lam, c, x_pitch, g_pitch, i_pitch, n, D, io_dtype, g_dtype);
  if (st != GDN_OK) return st;
  if (n == 0) return GDN_OK;
  if (!y || !state) return GDN_ERR_NULL;
  if (!aligned_to(y, elem_size(io_dtype)) || !aligned_to(state, 4) || !aligned_to(batch_indices, 4))
    return GDN_ERR_LAYOUT;
  gdn::RecurrenceArgs a{};
  a.x = x; a.g = g; a.i = i; a.lam = lam; a.c = c;
  a.x_pitch = x_pitch; a.g_pitch = g_pitch; a.i_pitch = i_pitch;
  a.D = D;
  a.io_dtype = io_dtype; a.g_dtype = g_dtype;
  a.state = state;
  a.num_slots = num_slots;
  a.batch_indices = batch_indices;
  a.n = n;
  a.y = y;
  a.dev_status = dev_status;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return gdn::status_of(gdn::launch_recurrence_decode(a));
}

}  // extern "C"
