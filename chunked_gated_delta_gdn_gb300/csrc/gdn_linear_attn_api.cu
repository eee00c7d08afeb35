// gdn_linear_attn_api.cu -- the extern "C" entry points of linear attention with a decay for
// each head: argument validation and dispatch.  Declarations and the contract are in gdn.h.
#include <math.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_linear_attn.h"
#include "gdn_status.h"

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

// Scratch of a call: the segments' states, then (backward) per-value-head dq and dk in fp32 where
// value heads share a query/key head.
struct Scratch {
  gdn::LaPlan plan;
  size_t local, part, total;   // bytes; part: one of the two
};
Scratch scratch(int num_passes, int B, int T, int num_seqs, bool packed, int Hqk, int Hv, int K, int V,
                int io_dtype) {
  Scratch s{{0, 1}, 0, 0, 0};
  const long long most = packed ? (long long)B * T : T, chains = (long long)num_seqs * Hv * num_passes;
  // the tensor cores pad the state to 128 x 128; on the CUDA cores a chunk takes long enough to
  // stand alone
  const bool tc = io_dtype == GDN_BF16;
  const int sms = gdn::current_sm_count();
  if (tc) s.plan = gdn::linear_attn_plan(chains, most, !packed, sms);
  else
    s.plan.segs =
        gdn::linear_attn_segments(chains, most, sms * gdn::linear_attn_generic_per_sm(K, V), 1);
  if (s.plan.segs > 1)
    s.local = align256((size_t)s.plan.segs * (chains - s.plan.whole) * (tc ? 16384 : K * V) * sizeof(float));
  if (num_passes > 1 && Hqk != Hv) s.part = align256((size_t)B * T * Hv * K * sizeof(float));
  s.total = s.local + 2 * s.part;
  return s;
}

// bf16 runs on the tensor cores; fp32, whose 24-bit products they do not offer, on the CUDA cores.
cudaError_t run_passes(const gdn::LinAttnPass* p, int n, const gdn::LaPlan& plan, void* local) {
  if (p[0].io_dtype == GDN_BF16)
    return gdn::launch_linear_attn_tc(p, n, plan, reinterpret_cast<float*>(local));
  return gdn::launch_linear_attn_generic(p, n, plan.segs, reinterpret_cast<float*>(local));
}

gdn_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return GDN_OK;
  if (!ws || bytes < need) return GDN_ERR_WORKSPACE;
  return ((uintptr_t)ws & 255u) ? GDN_ERR_LAYOUT : GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_linear_attn_chunk_fwd_workspace_size(int B, int T, int Hqk, int Hv, int K, int V,
                                                int num_seqs, gdn_dtype_t io_dtype) {
  if (check_shapes(B, T, Hqk, Hv, K, V, io_dtype) != GDN_OK || num_seqs < 0) return (size_t)-1;
  // (a batch of one row needs as much whether it is packed or not)
  return scratch(1, B, T, num_seqs, B == 1, Hqk, Hv, K, V, io_dtype).total;
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
    return T_total == 0 ? GDN_OK
                        : gdn::status_of(cudaMemsetAsync(
                              o, 0, (size_t)T_total * Hv * V * elem_size(io_dtype), p.stream));
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
  const Scratch sc = scratch(1, B, T, num_seqs, B == 1, Hqk, Hv, K, V, io_dtype);
  if ((st = check_workspace(workspace, workspace_bytes, sc.total)) != GDN_OK) return st;
  return gdn::status_of(run_passes(&p, 1, sc.plan, workspace));
}

size_t gdn_linear_attn_chunk_bwd_workspace_size(int B, int T, int Hqk, int Hv, int K, int V,
                                                int num_seqs, gdn_dtype_t io_dtype) {
  if (check_shapes(B, T, Hqk, Hv, K, V, io_dtype) != GDN_OK || num_seqs < 0) return (size_t)-1;
  return scratch(3, B, T, num_seqs, B == 1, Hqk, Hv, K, V, io_dtype).total;
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
  const Scratch ws = scratch(3, B, T, num_seqs, B == 1, Hqk, Hv, K, V, io_dtype);
  if ((st = check_workspace(workspace, workspace_bytes, num_seqs > 0 ? ws.total : 0)) != GDN_OK) return st;
  const gdn::LinAttnPass base =
      base_pass(log_decay, B, T, Hv, io_dtype, cu_seqlens, num_seqs, dev_status, stream);
  if (num_seqs == 0) {
    const size_t es = elem_size(io_dtype) * (size_t)T_total;
    if (T_total == 0) return GDN_OK;
    st = gdn::status_of(cudaMemsetAsync(dq, 0, es * Hqk * K, base.stream));
    if (st == GDN_OK) st = gdn::status_of(cudaMemsetAsync(dk, 0, es * Hqk * K, base.stream));
    if (st == GDN_OK) st = gdn::status_of(cudaMemsetAsync(dv, 0, es * Hv * V, base.stream));
    return st;
  }
  const float sc = resolve_scale(scale, K);
  const int group = Hv / Hqk;
  float* part[2] = {nullptr, nullptr};   // per-value-head dq, dk
  if (group > 1) {
    part[0] = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + ws.local);
    part[1] = part[0] + ws.part / sizeof(float);
  }
  gdn::LinAttnPass p[3] = {base, base, base};
  // dq_i = scale (sum_{j <= i} gamma^{i-j} (d_o_i . v_j) k_j + gamma^{i+1} S_0 d_o_i): the forward
  // pass over (d_o, v, k) with the state transposed
  p[0].q = d_o; p[0].k = v; p[0].v = k;
  p[0].Hq = p[0].Hk = Hv;
  p[0].Hv = Hqk;
  p[0].K = V; p[0].V = K;
  p[0].initial = initial_state;
  p[0].initial_t = 1;
  p[0].s_out = sc;
  p[0].o = group > 1 ? part[0] : dq;
  p[0].o_f32 = group > 1;
  // dk_j = sum_{i >= j} gamma^{i-j} (v_j . d_o_i) scale q_i + ..: backwards over (v, d_o, q), the
  // state being dS^T
  p[1].q = v; p[1].k = d_o; p[1].v = q;
  p[1].Hq = p[1].Hk = Hv;
  p[1].Hv = Hqk;
  p[1].K = V; p[1].V = K;
  p[1].initial = d_final_state;
  p[1].initial_t = 1;
  p[1].s_in = sc;
  p[1].reverse = 1;
  p[1].o = group > 1 ? part[1] : dk;
  p[1].o_f32 = group > 1;
  // dv_j = sum_{i >= j} gamma^{i-j} (k_j . q_i) scale d_o_i + ..: backwards over (k, q, d_o); its
  // state is dS, which ends as the gradient of the initial state
  p[2].q = k; p[2].k = q; p[2].v = d_o;
  p[2].Hq = p[2].Hk = Hqk;
  p[2].Hv = Hv;
  p[2].K = K; p[2].V = V;
  p[2].initial = d_final_state;
  p[2].final_state = d_initial_state;
  p[2].s_in = sc;
  p[2].reverse = 1;
  p[2].o = dv;
  st = gdn::status_of(run_passes(p, 3, ws.plan, workspace));
  if (st != GDN_OK) return st;
  if (group > 1) {
    const float* const in[2] = {part[0], part[1]};
    void* const out[2] = {dq, dk};
    st = gdn::status_of(
        gdn::launch_linear_attn_fold(in, out, T_total, Hqk, group, K, io_dtype, base.stream));
  }
  return st;
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
  return gdn::status_of(gdn::launch_linear_attn_decode(a));
}

}  // extern "C"
