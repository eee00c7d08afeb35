// gdn_qk_rotate_api.cu -- the extern "C" entry points of the norm of queries and keys with rotation:
// argument validation and dispatch.  Declarations and the contract are in gdn.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_qk_rotate.h"
#include "gdn_status.h"

namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem_size(int d) { return d == GDN_BF16 ? 2 : 4; }
bool is_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }

gdn_status_t check_sizes(int B, int T, int Hq, int Hk, int K) {
  if (B < 0 || T < 0 || Hq < 1 || Hk < 1 || K < 1 || K > GDN_MAX_ROTATE_DIM || Hq > (1 << 20) || Hk > (1 << 20))
    return GDN_ERR_SHAPE;
  if ((long long)B * T > 0x7fffffffLL) return GDN_ERR_SHAPE;
  return GDN_OK;
}

// Everything that forward and backward share, into `a`.
gdn_status_t prepare(gdn::QkRotateArgs* a, const void* q, const void* k, const long long* q_strides,
                     const long long* k_strides, int B, int T, int Hq, int Hk, int K, int R,
                     gdn_dtype_t io_dtype, gdn_norm_t norm, float eps, const void* q_weight,
                     const void* k_weight, gdn_dtype_t w_dtype, const float* inv_freq,
                     const int32_t* positions, int num_axes, const int* sections, int interleaved,
                     void* stream) {
  gdn_status_t st = check_sizes(B, T, Hq, Hk, K);
  if (st != GDN_OK) return st;
  if (!is_dtype(io_dtype) || !is_dtype(w_dtype) || (w_dtype != GDN_F32 && w_dtype != io_dtype))
    return GDN_ERR_DTYPE;
  if (R < 0 || R > K || (R & 1)) return GDN_ERR_SHAPE;
  if (norm != GDN_NORM_NONE && norm != GDN_NORM_RMS && norm != GDN_NORM_L2) return GDN_ERR_UNSUPPORTED;
  if (!(eps >= 0.f)) return GDN_ERR_SHAPE;
  if (num_axes < 1 || num_axes > GDN_MAX_AXES) return GDN_ERR_SHAPE;
  if (num_axes > 1 && !sections) return GDN_ERR_NULL;
  int pairs = 0;
  for (int i = 0; i < GDN_MAX_AXES; ++i) {
    if (i < num_axes) {
      const int n = sections ? sections[i] : R / 2;
      if (n < 0 || n > R / 2 - pairs) return GDN_ERR_SHAPE;
      pairs += n;
    }
    a->axis_end[i] = i < num_axes ? pairs : R / 2;
  }
  if (pairs != R / 2) return GDN_ERR_SHAPE;
  if ((long long)B * T > 0) {
    if (!q || !k || !q_strides || !k_strides || (R > 0 && !inv_freq)) return GDN_ERR_NULL;
    for (int i = 0; i < 3; ++i)
      if (q_strides[i] < 0 || k_strides[i] < 0) return GDN_ERR_SHAPE;
  }
  if (!aligned_to(q, elem_size(io_dtype)) || !aligned_to(k, elem_size(io_dtype)) ||
      !aligned_to(q_weight, elem_size(w_dtype)) || !aligned_to(k_weight, elem_size(w_dtype)) ||
      !aligned_to(inv_freq, 4) || !aligned_to(positions, 4))
    return GDN_ERR_LAYOUT;
  gdn::QkSide* s = a->side;
  s[0].x = q; s[0].H = Hq; s[0].w = q_weight;
  s[1].x = k; s[1].H = Hk; s[1].w = k_weight;
  if ((long long)B * T > 0) {
    s[0].sb = q_strides[0]; s[0].st = q_strides[1]; s[0].sh = q_strides[2];
    s[1].sb = k_strides[0]; s[1].st = k_strides[1]; s[1].sh = k_strides[2];
  }
  a->B = B; a->T = T; a->K = K; a->R = R;
  a->io_dtype = io_dtype; a->w_dtype = w_dtype;
  a->norm = norm;
  a->eps = eps;
  a->inv_freq = inv_freq;
  a->positions = positions;
  a->num_axes = num_axes;
  a->interleaved = interleaved != 0;
  a->stream = reinterpret_cast<cudaStream_t>(stream);
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_qk_norm_rotate_fwd(const void* q, const void* k, const long long* q_strides,
                                    const long long* k_strides, int B, int T, int Hq, int Hk, int K, int R,
                                    gdn_dtype_t io_dtype, gdn_norm_t norm, float eps, const void* q_weight,
                                    const void* k_weight, gdn_dtype_t w_dtype, const float* inv_freq,
                                    const int32_t* positions, int num_axes, const int* sections,
                                    int interleaved, void* q_out, void* k_out, void* stream) {
  gdn::QkRotateArgs a{};
  gdn_status_t st = prepare(&a, q, k, q_strides, k_strides, B, T, Hq, Hk, K, R, io_dtype, norm, eps, q_weight,
                            k_weight, w_dtype, inv_freq, positions, num_axes, sections, interleaved, stream);
  if (st != GDN_OK) return st;
  if ((long long)B * T == 0) return GDN_OK;
  if (!q_out || !k_out) return GDN_ERR_NULL;
  if (!aligned_to(q_out, elem_size(io_dtype)) || !aligned_to(k_out, elem_size(io_dtype))) return GDN_ERR_LAYOUT;
  a.side[0].out = q_out;
  a.side[1].out = k_out;
  return gdn::status_of(gdn::launch_qk_rotate_fwd(a));
}

size_t gdn_qk_norm_rotate_bwd_workspace_size(int B, int T, int Hq, int Hk, int K, int need_weights) {
  if (check_sizes(B, T, Hq, Hk, K) != GDN_OK) return (size_t)-1;
  return gdn::qk_rotate_bwd_workspace_bytes(B, T, Hq, Hk, K, need_weights != 0);
}

gdn_status_t gdn_qk_norm_rotate_bwd(const void* d_q, const void* d_k, const void* q, const void* k,
                                    const long long* q_strides, const long long* k_strides, int B, int T,
                                    int Hq, int Hk, int K, int R, gdn_dtype_t io_dtype, gdn_norm_t norm,
                                    float eps, const void* q_weight, const void* k_weight, gdn_dtype_t w_dtype,
                                    const float* inv_freq, const int32_t* positions, int num_axes,
                                    const int* sections, int interleaved, void* dq, void* dk,
                                    float* dq_weight, float* dk_weight, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  gdn::QkRotateArgs a{};
  gdn_status_t st = prepare(&a, q, k, q_strides, k_strides, B, T, Hq, Hk, K, R, io_dtype, norm, eps, q_weight,
                            k_weight, w_dtype, inv_freq, positions, num_axes, sections, interleaved, stream);
  if (st != GDN_OK) return st;
  if (!aligned_to(dq_weight, 4) || !aligned_to(dk_weight, 4)) return GDN_ERR_LAYOUT;
  if ((long long)B * T == 0) {   // no token: the weights' gradients are zero
    if (dq_weight) st = gdn::status_of(cudaMemsetAsync(dq_weight, 0, sizeof(float) * K, a.stream));
    if (st == GDN_OK && dk_weight) st = gdn::status_of(cudaMemsetAsync(dk_weight, 0, sizeof(float) * K, a.stream));
    return st;
  }
  if (!d_q || !d_k || !dq || !dk) return GDN_ERR_NULL;
  const size_t eb = elem_size(io_dtype);
  if (!aligned_to(d_q, eb) || !aligned_to(d_k, eb) || !aligned_to(dq, eb) || !aligned_to(dk, eb))
    return GDN_ERR_LAYOUT;
  const size_t need = gdn::qk_rotate_bwd_workspace_bytes(B, T, Hq, Hk, K, dq_weight || dk_weight);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return GDN_ERR_LAYOUT;
  }
  a.side[0].dy = d_q; a.side[0].out = dq; a.side[0].dw = dq_weight;
  a.side[1].dy = d_k; a.side[1].out = dk; a.side[1].dw = dk_weight;
  a.workspace = workspace;
  return gdn::status_of(gdn::launch_qk_rotate_bwd(a));
}

}  // extern "C"
