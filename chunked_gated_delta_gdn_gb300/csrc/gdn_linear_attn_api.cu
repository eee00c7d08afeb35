// gdn_linear_attn_api.cu -- the extern "C" entry points of linear attention with a decay for
// each head: argument validation and dispatch.  Declarations and the contract are in gdn.h.
#include <math.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_linear_attn.h"

namespace {

size_t elem_size(int d) { return d == GDN_BF16 ? 2 : 4; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
float resolve_scale(float scale, int K) { return isnan(scale) ? 1.0f / sqrtf((float)K) : scale; }

gdn_status_t check_shapes(int B, int T, int Hqk, int Hv, int K, int V, int io_dtype) {
  if (io_dtype != GDN_F32 && io_dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (B < 0 || T < 0 || Hqk <= 0 || Hv <= 0 || Hv % Hqk != 0) return GDN_ERR_SHAPE;
  if (K <= 0 || V <= 0 || K > GDN_MAX_HEAD_DIM || V > GDN_MAX_HEAD_DIM) return GDN_ERR_SHAPE;
  if ((K * elem_size(io_dtype)) % 16 != 0 || (V * elem_size(io_dtype)) % 16 != 0)
    return GDN_ERR_SHAPE;
  if ((long long)B * T > 0x7fffffffLL) return GDN_ERR_SHAPE;
  return GDN_OK;
}

// What the forward and the backward passes share.
gdn::LinAttnPass base_pass(const float* log_decay, int B, int T, int Hv, gdn_dtype_t io_dtype,
                           const int32_t* cu_seqlens, int num_seqs, int* dev_status, void* stream) {
  gdn::LinAttnPass p{};
  p.H = Hv;
  p.log_decay = log_decay;
  p.B = B; p.T = T;
  p.cu_seqlens = cu_seqlens;
  p.num_seqs = num_seqs;
  p.s_in = p.s_out = 1.f;
  p.io_dtype = io_dtype;
  p.dev_status = dev_status;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return p;
}

// bf16 runs on the tensor cores; fp32, whose 24-bit products they do not offer, on the CUDA cores.
cudaError_t run_pass(const gdn::LinAttnPass& p) {
  return p.io_dtype == GDN_BF16 ? gdn::launch_linear_attn_tc(p) : gdn::launch_linear_attn_generic(p);
}

// Scratch of the backward: per-value-head dq and dk (fp32) where value heads share a query/key
// head.  One buffer serves both, one after the other.
size_t bwd_part_bytes(long long T_total, int Hqk, int Hv, int K) {
  return Hqk == Hv ? 0 : align256((size_t)T_total * Hv * K * sizeof(float));
}

}  // namespace

extern "C" {

size_t gdn_linear_attn_chunk_fwd_workspace_size(int B, int T, int Hqk, int Hv, int K, int V,
                                                int num_seqs, gdn_dtype_t io_dtype) {
  if (check_shapes(B, T, Hqk, Hv, K, V, io_dtype) != GDN_OK || num_seqs < 0) return (size_t)-1;
  return 0;
}

gdn_status_t gdn_linear_attn_chunk_fwd(const void* q, const void* k, const void* v,
                                       const float* log_decay, int B, int T, int Hqk, int Hv, int K,
                                       int V, gdn_dtype_t io_dtype, float scale,
                                       const float* initial_state, int output_final_state,
                                       float* final_state, const int32_t* cu_seqlens, int num_seqs,
                                       const int32_t* state_indices, int num_slots, void* o,
                                       void* workspace, size_t workspace_bytes, int* dev_status,
                                       void* stream) {
  gdn_status_t st = check_shapes(B, T, Hqk, Hv, K, V, io_dtype);
  if (st != GDN_OK) return st;
  if (cu_seqlens) {
    if (B != 1 || num_seqs < 0) return GDN_ERR_SHAPE;
  } else {
    num_seqs = B;
  }
  const long long T_total = (long long)B * T;
  if (T_total > 0 && (!q || !k || !v || !o)) return GDN_ERR_NULL;
  if (!log_decay) return GDN_ERR_NULL;
  if (num_seqs > 0 && output_final_state && !final_state) return GDN_ERR_NULL;
  if (state_indices && num_slots <= 0) return GDN_ERR_SHAPE;
  if (T_total > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)))
    return GDN_ERR_LAYOUT;
  if (((uintptr_t)log_decay & 3u) || (initial_state && !aligned16(initial_state)) ||
      (output_final_state && !aligned16(final_state)))
    return GDN_ERR_LAYOUT;
  gdn::LinAttnPass p =
      base_pass(log_decay, B, T, Hv, io_dtype, cu_seqlens, num_seqs, dev_status, stream);
  if (num_seqs == 0)   // no sequence: no token belongs to one
    return T_total == 0 || cudaMemsetAsync(o, 0, (size_t)T_total * Hv * V * elem_size(io_dtype),
                                           p.stream) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
  p.q = q; p.k = k; p.v = v;
  p.Hq = p.Hk = Hqk;
  p.Hv = Hv;
  p.K = K; p.V = V;
  p.state_indices = state_indices;
  p.num_slots = num_slots;
  p.initial = initial_state;
  p.final_state = output_final_state ? final_state : nullptr;
  p.s_out = resolve_scale(scale, K);
  p.o = o;
  (void)workspace;
  (void)workspace_bytes;
  return run_pass(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_linear_attn_chunk_bwd_workspace_size(int B, int T, int Hqk, int Hv, int K, int V,
                                                int num_seqs, gdn_dtype_t io_dtype) {
  if (check_shapes(B, T, Hqk, Hv, K, V, io_dtype) != GDN_OK || num_seqs < 0) return (size_t)-1;
  return bwd_part_bytes((long long)B * T, Hqk, Hv, K);
}

gdn_status_t gdn_linear_attn_chunk_bwd(const void* q, const void* k, const void* v,
                                       const float* log_decay, int B, int T, int Hqk, int Hv, int K,
                                       int V, gdn_dtype_t io_dtype, float scale,
                                       const float* initial_state, const int32_t* cu_seqlens,
                                       int num_seqs, const void* d_o, const float* d_final_state,
                                       void* dq, void* dk, void* dv, float* d_initial_state,
                                       void* workspace, size_t workspace_bytes, int* dev_status,
                                       void* stream) {
  gdn_status_t st = check_shapes(B, T, Hqk, Hv, K, V, io_dtype);
  if (st != GDN_OK) return st;
  if (cu_seqlens) {
    if (B != 1 || num_seqs < 0) return GDN_ERR_SHAPE;
  } else {
    num_seqs = B;
  }
  const long long T_total = (long long)B * T;
  if (T_total > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)) return GDN_ERR_NULL;
  if (!log_decay) return GDN_ERR_NULL;
  if (T_total > 0 && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(d_o) ||
                      !aligned16(dq) || !aligned16(dk) || !aligned16(dv)))
    return GDN_ERR_LAYOUT;
  if (((uintptr_t)log_decay & 3u) || (initial_state && !aligned16(initial_state)) ||
      (d_final_state && !aligned16(d_final_state)) ||
      (d_initial_state && !aligned16(d_initial_state)))
    return GDN_ERR_LAYOUT;
  const size_t need = gdn_linear_attn_chunk_bwd_workspace_size(B, T, Hqk, Hv, K, V, num_seqs, io_dtype);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 255u) return GDN_ERR_LAYOUT;
  }
  const gdn::LinAttnPass base =
      base_pass(log_decay, B, T, Hv, io_dtype, cu_seqlens, num_seqs, dev_status, stream);
  if (num_seqs == 0) {
    const size_t es = elem_size(io_dtype) * (size_t)T_total;
    const bool ok = T_total == 0 ||
                    (cudaMemsetAsync(dq, 0, es * Hqk * K, base.stream) == cudaSuccess &&
                     cudaMemsetAsync(dk, 0, es * Hqk * K, base.stream) == cudaSuccess &&
                     cudaMemsetAsync(dv, 0, es * Hv * V, base.stream) == cudaSuccess);
    return ok ? GDN_OK : GDN_ERR_CUDA;
  }
  const float sc = resolve_scale(scale, K);
  const int group = Hv / Hqk;
  cudaError_t err;
  // dq_i = scale (sum_{j <= i} gamma^{i-j} (d_o_i . v_j) k_j + gamma^{i+1} S_0 d_o_i): the forward
  // pass over (d_o, v, k) with the state transposed
  gdn::LinAttnPass p = base;
  p.q = d_o; p.k = v; p.v = k;
  p.Hq = p.Hk = Hv;
  p.Hv = Hqk;
  p.K = V; p.V = K;
  p.initial = initial_state;
  p.initial_t = 1;
  p.s_out = sc;
  p.o = group > 1 ? workspace : dq;
  p.o_f32 = group > 1;
  if ((err = run_pass(p)) != cudaSuccess) return GDN_ERR_CUDA;
  if (group > 1 && gdn::launch_linear_attn_fold(reinterpret_cast<const float*>(workspace), dq, T_total,
                                                Hqk, group, K, io_dtype, p.stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  // dk_j = sum_{i >= j} gamma^{i-j} (v_j . d_o_i) scale q_i + ..: backwards over (v, d_o, q), the
  // state being dS^T
  p = base;
  p.q = v; p.k = d_o; p.v = q;
  p.Hq = p.Hk = Hv;
  p.Hv = Hqk;
  p.K = V; p.V = K;
  p.initial = d_final_state;
  p.initial_t = 1;
  p.s_in = sc;
  p.reverse = 1;
  p.o = group > 1 ? workspace : dk;
  p.o_f32 = group > 1;
  if ((err = run_pass(p)) != cudaSuccess) return GDN_ERR_CUDA;
  if (group > 1 && gdn::launch_linear_attn_fold(reinterpret_cast<const float*>(workspace), dk, T_total,
                                                Hqk, group, K, io_dtype, p.stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  // dv_j = sum_{i >= j} gamma^{i-j} (k_j . q_i) scale d_o_i + ..: backwards over (k, q, d_o); its
  // state is dS, which ends as the gradient of the initial state
  p = base;
  p.q = k; p.k = q; p.v = d_o;
  p.Hq = p.Hk = Hqk;
  p.Hv = Hv;
  p.K = K; p.V = V;
  p.initial = d_final_state;
  p.final_state = d_initial_state;
  p.s_in = sc;
  p.reverse = 1;
  p.o = dv;
  return run_pass(p) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_linear_attn_decode(const void* q, const void* k, const void* v,
                                    const float* log_decay, float* ssm_state, int num_slots,
                                    const int32_t* batch_indices, int n, int Hqk, int Hv, int K,
                                    int V, gdn_dtype_t io_dtype, float scale, void* o,
                                    int* dev_status, void* stream) {
  gdn_status_t st = check_shapes(1, 1, Hqk, Hv, K, V, io_dtype);
  if (st != GDN_OK) return st;
  if (n < 0 || num_slots < 0 || (!batch_indices && n > num_slots)) return GDN_ERR_SHAPE;
  if (n == 0) return GDN_OK;
  if (!q || !k || !v || !log_decay || !o || !ssm_state) return GDN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(ssm_state) ||
      ((uintptr_t)log_decay & 3u))
    return GDN_ERR_LAYOUT;
  gdn::LinAttnDecodeArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.log_decay = log_decay;
  a.state = ssm_state;
  a.num_slots = num_slots;
  a.batch_indices = batch_indices;
  a.n = n; a.Hqk = Hqk; a.Hv = Hv; a.K = K; a.V = V;
  a.io_dtype = io_dtype;
  a.scale = resolve_scale(scale, K);
  a.o = o;
  a.dev_status = dev_status;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return gdn::launch_linear_attn_decode(a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
