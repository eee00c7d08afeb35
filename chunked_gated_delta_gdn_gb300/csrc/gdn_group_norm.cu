// gdn_group_norm.cu -- group norm with an activation, channels last: forward and backward.
//
// For each row n and group g of C / G channels, over the L positions and the group's channels:
//   xhat = (x - mean) rstd,  u = xhat w + b,  y = act(u), or u act(z) with a gate z.
// Backward, with s = act:  du = dy s'(u)   (gate: du = dy s(z), dz = dy u s'(z)),
//   dw = sum du xhat,  db = sum du,  dx = rstd (du w - mean(du w) - xhat mean(du w xhat)).
#include <stdint.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_group_norm.h"

namespace gdn {
namespace {

constexpr int kGnThreads = 256;

__device__ __forceinline__ float act_value(float x, int act) {
  return act == GDN_ACT_SILU ? x / (1.f + expf(-x)) : x;
}
__device__ __forceinline__ float act_slope(float x, int act) {
  if (act != GDN_ACT_SILU) return 1.f;
  const float s = 1.f / (1.f + expf(-x));
  return s * (1.f + x * (1.f - s));
}

// Sum over the CTA; every thread gets the result.
__device__ float block_sum(float x, float* red) {
  x = warp_sum(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kGnThreads / 32; ++w) s += red[w];
  return s;
}

// One CTA per (n, g).
__global__ void __launch_bounds__(kGnThreads) group_norm_fwd_kernel(const GroupNormArgs a) {
  __shared__ float red[kGnThreads / 32];
  const int g = blockIdx.x % a.G, n = blockIdx.x / a.G, D = a.C / a.G;
  const long long count = (long long)a.L * D;
  const size_t base = (size_t)n * a.L * a.C + (size_t)g * D;
  float s = 0.f;
  for (long long e = threadIdx.x; e < count; e += kGnThreads)
    s += load_elem(a.x, base + (size_t)(e / D) * a.C + e % D, a.io_dtype);
  const float mean = block_sum(s, red) / (float)count;
  s = 0.f;
  for (long long e = threadIdx.x; e < count; e += kGnThreads) {
    const float d = load_elem(a.x, base + (size_t)(e / D) * a.C + e % D, a.io_dtype) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = 1.f / sqrtf(block_sum(s, red) / (float)count + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[blockIdx.x] = mean;
    if (a.rstd) a.rstd[blockIdx.x] = rstd;
  }
  for (long long e = threadIdx.x; e < count; e += kGnThreads) {
    const int c = (int)(e % D);
    const size_t at = base + (size_t)(e / D) * a.C + c;
    const float w = a.weight ? load_elem(a.weight, g * D + c, a.wb_dtype) : 1.f;
    const float b = a.bias ? load_elem(a.bias, g * D + c, a.wb_dtype) : 0.f;
    const float u = (load_elem(a.x, at, a.io_dtype) - mean) * rstd * w + b;
    const float y = a.gate ? u * act_value(load_elem(a.gate, at, a.io_dtype), a.act) : act_value(u, a.act);
    store_elem(a.y, at, y, a.io_dtype);
  }
}

// du, xhat (and dz) of one element.
__device__ __forceinline__ float grad_u(const GroupNormArgs& a, size_t at, float mean, float rstd,
                                        float w, float b, float* xhat, float* dz) {
  const float xh = (load_elem(a.x, at, a.io_dtype) - mean) * rstd, u = xh * w + b;
  const float dy = load_elem(a.dy, at, a.io_dtype);
  *xhat = xh;
  if (a.gate) {
    const float z = load_elem(a.gate, at, a.io_dtype);
    *dz = dy * u * act_slope(z, a.act);
    return dy * act_value(z, a.act);
  }
  return dy * act_slope(u, a.act);
}

__global__ void __launch_bounds__(kGnThreads) group_norm_bwd_x_kernel(const GroupNormArgs a) {
  __shared__ float red[kGnThreads / 32];
  const int g = blockIdx.x % a.G, n = blockIdx.x / a.G, D = a.C / a.G;
  const long long count = (long long)a.L * D;
  const size_t base = (size_t)n * a.L * a.C + (size_t)g * D;
  const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  float m1 = 0.f, m2 = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    float s1 = 0.f, s2 = 0.f;
    for (long long e = threadIdx.x; e < count; e += kGnThreads) {
      const int c = (int)(e % D);
      const size_t at = base + (size_t)(e / D) * a.C + c;
      const float w = a.weight ? load_elem(a.weight, g * D + c, a.wb_dtype) : 1.f;
      const float b = a.bias ? load_elem(a.bias, g * D + c, a.wb_dtype) : 0.f;
      float xh, dz = 0.f;
      const float d = grad_u(a, at, mean, rstd, w, b, &xh, &dz) * w;
      if (pass == 0) {
        s1 += d;
        s2 = fmaf(d, xh, s2);
      } else {
        store_elem(a.dx, at, rstd * (d - m1 - xh * m2), a.io_dtype);
        if (a.gate) store_elem(a.dgate, at, dz, a.io_dtype);
      }
    }
    if (pass == 0) {
      m1 = block_sum(s1, red) / (float)count;
      m2 = block_sum(s2, red) / (float)count;
    }
  }
}

// dweight, dbias: one CTA per channel.
__global__ void __launch_bounds__(kGnThreads) group_norm_bwd_w_kernel(const GroupNormArgs a) {
  __shared__ float red[kGnThreads / 32];
  const int c = blockIdx.x, g = c / (a.C / a.G);
  const float w = a.weight ? load_elem(a.weight, c, a.wb_dtype) : 1.f;
  const float b = a.bias ? load_elem(a.bias, c, a.wb_dtype) : 0.f;
  float s1 = 0.f, s2 = 0.f;
  for (long long r = threadIdx.x; r < (long long)a.N * a.L; r += kGnThreads) {
    const long long i = (r / a.L) * a.G + g;
    float xh, dz;
    const float d = grad_u(a, (size_t)r * a.C + c, a.mean[i], a.rstd[i], w, b, &xh, &dz);
    s1 += d;
    s2 = fmaf(d, xh, s2);
  }
  const float db = block_sum(s1, red), dw = block_sum(s2, red);
  if (threadIdx.x == 0) {
    if (a.dweight) a.dweight[c] = dw;
    if (a.dbias) a.dbias[c] = db;
  }
}

}  // namespace

size_t group_norm_fwd_workspace_bytes(int, int, int, int, int) { return 0; }
size_t group_norm_bwd_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a) {
  const long long blocks = (long long)a.N * a.G;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  group_norm_fwd_kernel<<<(unsigned)blocks, kGnThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs& a) {
  const long long blocks = (long long)a.N * a.G;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (blocks > 0) group_norm_bwd_x_kernel<<<(unsigned)blocks, kGnThreads, 0, a.stream>>>(a);
  if (a.dweight || a.dbias) group_norm_bwd_w_kernel<<<(unsigned)a.C, kGnThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn

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
  return gdn::launch_group_norm_fwd(a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
    const bool ok =
        (!dweight || cudaMemsetAsync(dweight, 0, sizeof(float) * C, s) == cudaSuccess) &&
        (!dbias || cudaMemsetAsync(dbias, 0, sizeof(float) * C, s) == cudaSuccess);
    return ok ? GDN_OK : GDN_ERR_CUDA;
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
  return gdn::launch_group_norm_bwd(a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
