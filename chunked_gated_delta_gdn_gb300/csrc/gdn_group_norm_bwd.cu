// gdn_group_norm_bwd.cu -- group norm with an activation, channels last: the backward.
//
// With s the activation, du = dy s'(u) (gate: du = dy s(z), dz = dy u s'(z)):
//   dw_c = sum du xhat,  db_c = sum du   over rows and positions,
//   dx = rstd (du w - m1 - xhat m2),     m1, m2 the group's means of du w and du w xhat.
//
// A thread keeps its channels and sums du and du xhat for each of them (A, B): those are its share
// of db and dw, and sum_c w_c A_c, sum_c w_c B_c its share of m1 and m2.  Every sum is made in a
// fixed order.  Bound by bytes: x, dy (and z) read once, dx (and dz) written once is the floor.
//   L = 1 and groups of up to 512 channels: one launch reads each row once, its groups in
//     registers, and leaves A, B of each set of rows; a second adds the sets.
//   else: a launch for A, B and the slab's share of m1, m2, a second that reads x, dy (and z) again
//     and applies, its last CTAs adding A, B up.
#include "gdn_group_norm.cuh"

namespace gdn {
namespace {

// xhat and du of one element (and dz).
template <bool kGate>
__device__ __forceinline__ float grad_u(float x, float dy, float z, float mean, float rstd, float w, float b,
                                        int act, float* xhat, float* dz) {
  const float xh = (x - mean) * rstd, u = fmaf(xh, w, b);
  *xhat = xh;
  if (kGate) {
    const float2 s = act_both(z, act);
    *dz = dy * u * s.y;
    return dy * s.x;
  }
  return dy * act_both(u, act).y;
}

// Adds up part[set][2][C] over the sets in a fixed order: channel c0 + threadIdx.x % 32, every
// kRows-th set a thread.
template <int kRows>
__device__ void sum_sets(const GroupNormArgs& a, const float* part, int sets, int block) {
  __shared__ float sa[kRows][33], sb[kRows][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, c = block * 32 + lane;
  float A = 0.f, B = 0.f;
  if (c < a.C) {
#pragma unroll 4
    for (int r = row; r < sets; r += kRows) {
      const float* q = part + (size_t)r * 2 * a.C + c;
      A += q[0];
      B += q[a.C];
    }
  }
  sa[row][lane] = A;
  sb[row][lane] = B;
  __syncthreads();
  if (row == 0 && c < a.C) {
    for (int i = 1; i < kRows; ++i) {
      A += sa[i][lane];
      B += sb[i][lane];
    }
    if (a.dbias) a.dbias[c] = A;
    if (a.dweight) a.dweight[c] = B;
  }
}
__global__ void __launch_bounds__(1024) gn_sum_sets_kernel(const GroupNormArgs a, const float* part, int sets) {
  sum_sets<32>(a, part, sets, blockIdx.x);
}

// ------------------------------------------------------------------ L = 1, groups in registers
// A CTA's J lane groups take all G channel groups of J / G rows at a time, or, where J < G, J
// channel groups of one row; then the CTA's next rows.  A, B of the CTA's rows are one set.
struct RowSets {
  int J, across, down, sets;   // lane groups; CTAs across the groups; rows at a time; sets
};

template <typename T, int V, int VPT, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_row_bwd_kernel(const GroupNormArgs a, int lanes, const RowSets q,
                                                                float* part) {
  __shared__ float acc[2][kGnThreads * 16];
  const int D = a.C / a.G, DV = D / V;
  const int l = threadIdx.x & (lanes - 1), j0 = threadIdx.x / lanes;
  const int set = blockIdx.x / q.across;
  const int g_raw = q.across == 1 ? j0 % a.G : (blockIdx.x % q.across) * q.J + j0;
  const int down = q.across == 1 ? j0 / a.G : 0;
  const bool live = g_raw < a.G && down < q.down;
  const int g = live ? g_raw : 0;
  const float inv = 1.f / (float)D;
  float w[VPT][V], b[VPT][V], A[VPT][V], B[VPT][V];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = l + k * lanes, c = g * D + v * V + j;
      w[k][j] = v < DV ? param(a.weight, c, a.wb_dtype, 1.f) : 0.f;
      b[k][j] = v < DV ? param(a.bias, c, a.wb_dtype, 0.f) : 0.f;
      A[k][j] = B[k][j] = 0.f;
    }
  // (every lane of a warp runs the same number of turns: the shuffles want them all)
  const long long step = (long long)q.sets * q.down;
  const int turns = (int)((a.N + step - 1) / step);
  for (int t = 0; t < turns; ++t) {
    const long long n = t * step + (long long)set * q.down + down;
    const bool on = live && n < a.N;
    const size_t at = ((size_t)(on ? n : 0) * a.G + g) * D;   // (n >= N: nothing is touched)
    const float mean = on ? a.mean[(size_t)n * a.G + g] : 0.f, rstd = on ? a.rstd[(size_t)n * a.G + g] : 0.f;
    Pack<T, V> x[VPT], dy[VPT], z[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = l + k * lanes;
      const bool in = on && v < DV;
      x[k] = in ? load_pack<T, V>(a.x, at + (size_t)v * V) : Pack<T, V>{};
      dy[k] = in ? load_pack<T, V>(a.dy, at + (size_t)v * V) : Pack<T, V>{};
      if (kGate) z[k] = in ? load_pack<T, V>(a.gate, at + (size_t)v * V) : Pack<T, V>{};
    }
    float xh[VPT][V], d[VPT][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const bool in = on && l + k * lanes < DV;
      Pack<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float dz = 0.f;
        const float du = grad_u<kGate>(to_f(x[k].e[j]), to_f(dy[k].e[j]), kGate ? to_f(z[k].e[j]) : 0.f, mean,
                                       rstd, w[k][j], b[k][j], a.act, &xh[k][j], &dz);
        if (kGate) from_f(o.e[j], dz);
        if (in) {
          A[k][j] += du;
          B[k][j] = fmaf(du, xh[k][j], B[k][j]);
          d[k][j] = du * w[k][j];
          s1 += d[k][j];
          s2 = fmaf(d[k][j], xh[k][j], s2);
        }
      }
      if (kGate && in) store_pack<T, V>(a.dgate, at + (size_t)(l + k * lanes) * V, o);
    }
    const float m1 = sub_sum(s1, lanes) * inv, m2 = sub_sum(s2, lanes) * inv;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on && l + k * lanes < DV) {
        Pack<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) from_f(o.e[j], rstd * (d[k][j] - m1 - xh[k][j] * m2));
        store_pack<T, V>(a.dx, at + (size_t)(l + k * lanes) * V, o);
      }
  }
  if (!part) return;
  float* out = part + (size_t)set * 2 * a.C;
  if (q.down == 1) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = l + k * lanes;
      if (live && v < DV) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          out[g * D + v * V + j] = A[k][j];
          out[a.C + g * D + v * V + j] = B[k][j];
        }
      }
    }
    return;
  }
  // (down C <= J lanes VPT V <= 256 * 16)
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = l + k * lanes;
    if (live && v < DV) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        acc[0][down * a.C + g * D + v * V + j] = A[k][j];
        acc[1][down * a.C + g * D + v * V + j] = B[k][j];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += kGnThreads) {
    float x = 0.f, y = 0.f;
    for (int r = 0; r < q.down; ++r) {
      x += acc[0][r * a.C + c];
      y += acc[1][r * a.C + c];
    }
    out[c] = x;
    out[a.C + c] = y;
  }
}

// ------------------------------------------------------------------ slabs
// part [n][chunk][2][C]: A, B; share [n][g][chunk][parts]: (sum du w, sum du w xhat) of the slab.
template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_slab_grad_kernel(const GroupNormArgs a, const SlabPlan s,
                                                                  float* part, float2* share) {
  __shared__ float sa[kGnThreads * V], sb[kGnThreads * V];
  const SlabPlace p = slab_place(s, a.C, a.G);
  const int2 rr = slab_rows(s, p, a.L);
  float A[V], B[V];
#pragma unroll
  for (int j = 0; j < V; ++j) A[j] = B[j] = 0.f;
  if (p.on) {
    const float mean = a.mean[(size_t)p.n * a.G + p.g], rstd = a.rstd[(size_t)p.n * a.G + p.g];
    float w[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[j] = param(a.weight, p.c + j, a.wb_dtype, 1.f);
      b[j] = param(a.bias, p.c + j, a.wb_dtype, 0.f);
    }
    const size_t base = (size_t)p.n * a.L * a.C + p.c;
    for (int r = rr.x + p.row; r < rr.y; r += 2 * p.step) {
      Pack<T, V> x[2], dy[2], z[2];
      const int k = min(2, (rr.y - r + p.step - 1) / p.step);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < k) {
          const size_t at = base + (size_t)(r + i * p.step) * a.C;
          x[i] = load_pack<T, V>(a.x, at);
          dy[i] = load_pack<T, V>(a.dy, at);
          if (kGate) z[i] = load_pack<T, V>(a.gate, at);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < k) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float xh, dz;
            const float du = grad_u<kGate>(to_f(x[i].e[j]), to_f(dy[i].e[j]), kGate ? to_f(z[i].e[j]) : 0.f, mean,
                                           rstd, w[j], b[j], a.act, &xh, &dz);
            A[j] += du;
            B[j] = fmaf(du, xh, B[j]);
          }
        }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    sa[j * kGnThreads + threadIdx.x] = A[j];
    sb[j * kGnThreads + threadIdx.x] = B[j];
  }
  __syncthreads();
  // the columns' sums over the CTA's row lanes, in order; each then stands in the first row's place
  if (threadIdx.x < p.cols) {
    float* q = part + ((size_t)p.n * s.chunks + p.chunk) * 2 * a.C + p.c;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float x = 0.f, y = 0.f;
      for (int r = 0; r < p.step; ++r) {
        x += sa[j * kGnThreads + r * p.cols + threadIdx.x];
        y += sb[j * kGnThreads + r * p.cols + threadIdx.x];
      }
      q[j] = x;
      q[a.C + j] = y;
      const float w = param(a.weight, p.c + j, a.wb_dtype, 1.f);
      A[j] = x * w;
      B[j] = y * w;
    }
  }
  __syncthreads();
  if (threadIdx.x < p.cols) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x += A[j];
      y += B[j];
    }
    sa[threadIdx.x] = x;
    sb[threadIdx.x] = y;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, per = s.parts == 1 ? s.DV : p.cols;
  for (int g = threadIdx.x >> 5; g < p.groups; g += kGnThreads / 32) {
    float x = 0.f, y = 0.f;
    for (int m = lane; m < per; m += 32) {
      x += sa[g * per + m];
      y += sb[g * per + m];
    }
    x = warp_sum(x);
    y = warp_sum(y);
    if (lane == 0) {
      const int q = p.chunk * s.parts + (s.parts == 1 ? 0 : p.cb - p.g0 * s.parts);
      share[((size_t)p.n * a.G + p.g0 + g) * (s.chunks * s.parts) + q] = make_float2(x, y);
    }
  }
}

template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_slab_bwd_kernel(const GroupNormArgs a, const SlabPlan s, int slabs,
                                                                 const float* part, const float2* share) {
  if ((int)blockIdx.x >= slabs) {
    sum_sets<kGnThreads / 32>(a, part, a.N * s.chunks, blockIdx.x - slabs);
    return;
  }
  __shared__ float2 means[kGnThreads];
  const SlabPlace p = slab_place(s, a.C, a.G);
  const int lane = threadIdx.x & 31, Q = s.chunks * s.parts;
  const float inv = 1.f / ((float)a.L * (float)(a.C / a.G));
  for (int g = threadIdx.x >> 5; g < p.groups; g += kGnThreads / 32) {
    const float2* q = share + ((size_t)p.n * a.G + p.g0 + g) * Q;
    float x = 0.f, y = 0.f;
    for (int k = lane; k < Q; k += 32) {
      const float2 v = q[k];
      x += v.x;
      y += v.y;
    }
    x = warp_sum(x);
    y = warp_sum(y);
    if (lane == 0) means[g] = make_float2(x * inv, y * inv);
  }
  __syncthreads();
  if (!p.on) return;
  const int2 rr = slab_rows(s, p, a.L);
  const float mean = a.mean[(size_t)p.n * a.G + p.g], rstd = a.rstd[(size_t)p.n * a.G + p.g];
  const float2 m = means[p.g - p.g0];
  float w[V], b[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    w[j] = param(a.weight, p.c + j, a.wb_dtype, 1.f);
    b[j] = param(a.bias, p.c + j, a.wb_dtype, 0.f);
  }
  const size_t base = (size_t)p.n * a.L * a.C + p.c;
  for (int r = rr.x + p.row; r < rr.y; r += 2 * p.step) {
    Pack<T, V> x[2], dy[2], z[2];
    const int k = min(2, (rr.y - r + p.step - 1) / p.step);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < k) {
        const size_t at = base + (size_t)(r + i * p.step) * a.C;
        x[i] = load_pack<T, V>(a.x, at);
        dy[i] = load_pack<T, V>(a.dy, at);
        if (kGate) z[i] = load_pack<T, V>(a.gate, at);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < k) {
        const size_t at = base + (size_t)(r + i * p.step) * a.C;
        Pack<T, V> o, oz;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float xh, dz = 0.f;
          const float du = grad_u<kGate>(to_f(x[i].e[j]), to_f(dy[i].e[j]), kGate ? to_f(z[i].e[j]) : 0.f, mean,
                                         rstd, w[j], b[j], a.act, &xh, &dz);
          from_f(o.e[j], rstd * (du * w[j] - m.x - xh * m.y));
          if (kGate) from_f(oz.e[j], dz);
        }
        store_pack<T, V>(a.dx, at, o);
        if (kGate) store_pack<T, V>(a.dgate, at, oz);
      }
  }
}

constexpr int kRowValues = 16;   // values a lane holds in the row form

// The row form's CTAs: about six an SM, and no more than the rows need.
RowSets row_sets(int N, int G, int lanes) {
  RowSets q;
  q.J = kGnThreads / lanes;
  q.across = q.J >= G ? 1 : (G + q.J - 1) / q.J;
  q.down = q.J >= G ? q.J / G : 1;
  const long long most = ((long long)N + q.down - 1) / q.down, want = 152LL * 6 / q.across + 1;
  q.sets = (int)(want < most ? want : most);
  return q;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T, int V, bool kGate>
void launch_bwd(const GroupNormArgs& a) {
  const bool params = a.dweight || a.dbias;
  const RowPlan r = row_plan(a.C, a.G, a.io_dtype, kRowValues);
  float* part = reinterpret_cast<float*>(a.workspace);
  const unsigned sum_ctas = (unsigned)((a.C + 31) / 32);
  if (a.L == 1 && r.lanes > 0) {
    const RowSets q = row_sets(a.N, a.G, r.lanes);
    const unsigned grid = (unsigned)(q.sets * q.across);
    float* to = params ? part : nullptr;
    if (r.VPT == 1) gn_row_bwd_kernel<T, V, 1, kGate><<<grid, kGnThreads, 0, a.stream>>>(a, r.lanes, q, to);
    else gn_row_bwd_kernel<T, V, kRowValues / V, kGate><<<grid, kGnThreads, 0, a.stream>>>(a, r.lanes, q, to);
    if (params) gn_sum_sets_kernel<<<sum_ctas, 1024, 0, a.stream>>>(a, part, q.sets);
    return;
  }
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  const int slabs = a.N * s.NCB * s.chunks;
  float2* share = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(a.workspace) +
                                            align256((size_t)a.N * s.chunks * 2 * a.C * sizeof(float)));
  gn_slab_grad_kernel<T, V, kGate><<<slabs, kGnThreads, 0, a.stream>>>(a, s, part, share);
  gn_slab_bwd_kernel<T, V, kGate><<<slabs + (params ? sum_ctas : 0), kGnThreads, 0, a.stream>>>(a, s, slabs, part,
                                                                                            share);
}

template <typename T, int V>
void launch_bwd(const GroupNormArgs& a) {
  if (a.gate) launch_bwd<T, V, true>(a);
  else launch_bwd<T, V, false>(a);
}

}  // namespace

size_t group_norm_bwd_workspace_bytes(int N, int L, int C, int G, int io_dtype) {
  if (N == 0 || L == 0) return 0;
  const RowPlan r = row_plan(C, G, io_dtype, kRowValues);
  if (L == 1 && r.lanes > 0) return align256((size_t)row_sets(N, G, r.lanes).sets * 2 * C * sizeof(float));
  const SlabPlan s = slab_plan(N, L, C, G, io_dtype);
  return align256((size_t)N * s.chunks * 2 * C * sizeof(float)) +
         align256((size_t)N * G * s.chunks * s.parts * sizeof(float2));
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs& a) {
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  if ((long long)a.N * s.NCB * s.chunks + a.C > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.io_dtype == GDN_F32) {
    switch (s.V) {
      case 4: launch_bwd<float, 4>(a); break;
      case 2: launch_bwd<float, 2>(a); break;
      default: launch_bwd<float, 1>(a);
    }
  } else {
    switch (s.V) {
      case 8: launch_bwd<__nv_bfloat16, 8>(a); break;
      case 4: launch_bwd<__nv_bfloat16, 4>(a); break;
      case 2: launch_bwd<__nv_bfloat16, 2>(a); break;
      default: launch_bwd<__nv_bfloat16, 1>(a);
    }
  }
  return cudaGetLastError();
}

}  // namespace gdn
