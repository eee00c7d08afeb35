// gdn_group_norm_api.cu -- the extern "C" entry points of group norm with an activation: argument
// validation and dispatch.  Declarations and the contract are in gdn.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_group_norm.h"
#include "gdn_status.h"

namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem_size(int d) { return d == GDN_BF16 ? 2 : 4; }
bool is_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }

gdn_status_t check_sizes(int N, int L, int C, int G, int io_dtype) {
  if (!is_dtype(io_dtype)) return GDN_ERR_DTYPE;
  if (N < 0 || L < 0 || C <= 0 || G <= 0 || C % G != 0) return GDN_ERR_SHAPE;
  if ((long long)N * G > 0x7fffffffLL || (long long)N * L > 0x7fffffffLL) return GDN_ERR_SHAPE;
  return GDN_OK;
}

gdn_status_t check_params(const void* weight, const void* bias, int io_dtype, int wb_dtype, int act) {
  if (!is_dtype(wb_dtype) || (wb_dtype != GDN_F32 && wb_dtype != io_dtype)) return GDN_ERR_DTYPE;
  if (act != GDN_ACT_NONE && act != GDN_ACT_SILU) return GDN_ERR_UNSUPPORTED;
  if (!aligned_to(weight, elem_size(wb_dtype)) || !aligned_to(bias, elem_size(wb_dtype)))
    return GDN_ERR_LAYOUT;
  return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_group_norm_act_fwd_workspace_size(int N, int L, int C, int G, gdn_dtype_t io_dtype) {
  if (check_sizes(N, L, C, G, io_dtype) != GDN_OK) return (size_t)-1;
  return gdn::group_norm_fwd_workspace_bytes(N, L, C, G, io_dtype);
}

gdn_status_t gdn_group_norm_act_fwd(const void* x, const void* weight, const void* bias,
                                    const void* gate, int N, int L, int C, int G,
                                    gdn_dtype_t io_dtype, gdn_dtype_t wb_dtype, float eps,
                                    gdn_act_t act, void* y, float* mean, float* rstd,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status_t st = check_sizes(N, L, C, G, io_dtype);
  if (st == GDN_OK) st = check_params(weight, bias, io_dtype, wb_dtype, act);
  if (st != GDN_OK) return st;
  if (!(eps >= 0.f)) return GDN_ERR_SHAPE;
  if ((long long)N * L == 0) return GDN_OK;
  if (!x || !y) return GDN_ERR_NULL;
  if (!aligned_to(x, 16) || !aligned_to(y, 16) || !aligned_to(gate, 16) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return GDN_ERR_LAYOUT;
  const size_t need = gdn::group_norm_fwd_workspace_bytes(N, L, C, G, io_dtype);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return GDN_ERR_LAYOUT;
  }
  gdn::GroupNormArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.gate = gate;
  a.N = N; a.L = L; a.C = C; a.G = G;
  a.io_dtype = io_dtype; a.wb_dtype = wb_dtype;
  a.eps = eps;
  a.act = act;
  a.y = y; a.mean = mean; a.rstd = rstd;
  a.workspace = workspace;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return gdn::status_of(gdn::launch_group_norm_fwd(a));
}

size_t gdn_group_norm_act_bwd_workspace_size(int N, int L, int C, int G, gdn_dtype_t io_dtype) {
  if (check_sizes(N, L, C, G, io_dtype) != GDN_OK) return (size_t)-1;
  return gdn::group_norm_bwd_workspace_bytes(N, L, C, G, io_dtype);
}

gdn_status_t gdn_group_norm_act_bwd(const void* dy, const void* x, const void* weight,
                                    const void* bias, const void* gate, const float* mean,
                                    const float* rstd, int N, int L, int C, int G,
                                    gdn_dtype_t io_dtype, gdn_dtype_t wb_dtype, gdn_act_t act,
                                    void* dx, void* dgate, float* dweight, float* dbias,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status_t st = check_sizes(N, L, C, G, io_dtype);
  if (st == GDN_OK) st = check_params(weight, bias, io_dtype, wb_dtype, act);
  if (st != GDN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4)) return GDN_ERR_LAYOUT;
  if ((long long)N * L == 0) {   // no element: the parameters' gradients are zero
    if (dweight) st = gdn::status_of(cudaMemsetAsync(dweight, 0, sizeof(float) * C, s));
    if (st == GDN_OK && dbias) st = gdn::status_of(cudaMemsetAsync(dbias, 0, sizeof(float) * C, s));
    return st;
  }
  if (!dy || !x || !mean || !rstd || !dx || (gate && !dgate)) return GDN_ERR_NULL;
  if (!aligned_to(dy, 16) || !aligned_to(x, 16) || !aligned_to(gate, 16) || !aligned_to(dx, 16) ||
      !aligned_to(dgate, 16) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return GDN_ERR_LAYOUT;
  const size_t need = gdn::group_norm_bwd_workspace_bytes(N, L, C, G, io_dtype);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return GDN_ERR_LAYOUT;
  }
  gdn::GroupNormArgs a{};
  a.x = x; a.weight = weight; a.bias = bias; a.gate = gate;
  a.N = N; a.L = L; a.C = C; a.G = G;
  a.io_dtype = io_dtype; a.wb_dtype = wb_dtype;
  a.act = act;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dx = dx; a.dgate = dgate; a.dweight = dweight; a.dbias = dbias;
  a.workspace = workspace;
  a.stream = s;
  return gdn::status_of(gdn::launch_group_norm_bwd(a));
}

}  // extern "C"
