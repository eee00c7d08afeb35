// gdn_group_norm.cu -- group norm with an activation, channels last: the forward.
//
// For each row n and group g of D = C / G channels, over the L positions and the group's channels:
//   xhat = (x - mean) rstd,  u = xhat w + b,  y = act(u), or u act(z) with a gate z.
//
// Bound by bytes: x (and z) read once, y written once is the floor.  Two forms:
//   L = 1 and groups of up to 1024 channels: a group lives in the registers of up to 32 lanes,
//     which read it once, take mean and variance over two register passes and write it.
//   else: a launch for each slab's mean and squared deviations (merged pairwise from batches of
//     registers, never as E[x^2] - E[x]^2), and one that merges the slabs' and applies; the second
//     reading of x comes from L2 where the tensor fits it.
#include "gdn_group_norm.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ L = 1, groups in registers
template <typename T, int V, int VPT, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_row_fwd_kernel(const GroupNormArgs a, int lanes) {
  const int D = a.C / a.G, DV = D / V;
  const int l = threadIdx.x & (lanes - 1);
  const long long items = (long long)a.N * a.G, per = (long long)gridDim.x * (kGnThreads / lanes);
  const float inv = 1.f / (float)D;
  // (every lane of a warp runs the same number of turns: the shuffles want them all)
  const long long first = (long long)blockIdx.x * (kGnThreads / lanes) + threadIdx.x / lanes;
  const long long warp_first = first - (threadIdx.x & 31) / lanes;
  for (long long base = 0; warp_first + base < items; base += per) {
    const long long item = first + base;
    const bool on = item < items;
    const int g = (int)((on ? item : 0) % a.G);
    const size_t at = (size_t)(on ? item : 0) * D;
    float x[VPT][V], z[VPT][V];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = l + k * lanes;
      const bool in = on && v < DV;
      const Pack<T, V> p = in ? load_pack<T, V>(a.x, at + (size_t)v * V) : Pack<T, V>{};
      const Pack<T, V> q = kGate && in ? load_pack<T, V>(a.gate, at + (size_t)v * V) : Pack<T, V>{};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[k][j] = to_f(p.e[j]);
        if (kGate) z[k][j] = to_f(q.e[j]);
      }
    }
    // mean from the first element, then the squared deviations
    const float x0 = __shfl_sync(0xffffffffu, x[0][0], 0, lanes);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (l + k * lanes < DV) {
#pragma unroll
        for (int j = 0; j < V; ++j) s += x[k][j] - x0;
      }
    const float mean = x0 + sub_sum(s, lanes) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (l + k * lanes < DV) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = x[k][j] - mean;
          s = fmaf(d, d, s);
        }
      }
    const float rstd = rsqrtf(fmaf(sub_sum(s, lanes), inv, a.eps));
    if (!on) continue;
    if (l == 0) {
      if (a.mean) a.mean[item] = mean;
      if (a.rstd) a.rstd[item] = rstd;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = l + k * lanes;
      if (v >= DV) continue;
      Pack<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = g * D + v * V + j;
        const float u = fmaf((x[k][j] - mean) * rstd, param(a.weight, c, a.wb_dtype, 1.f),
                             param(a.bias, c, a.wb_dtype, 0.f));
        from_f(o.e[j], kGate ? u * act_value(z[k][j], a.act) : act_value(u, a.act));
      }
      store_pack<T, V>(a.y, at + (size_t)v * V, o);
    }
  }
}

// ------------------------------------------------------------------ slabs
// Mean and squared deviations of `n` values merged with those of `m` more.
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ void merge(Moments& a, float n, float mean, float m2) {
  const float t = a.n + n, d = mean - a.mean, f = n / t;
  a.mean = fmaf(d, f, a.mean);
  a.m2 += m2 + d * d * a.n * f;
  a.n = t;
}

template <typename T, int V>
__global__ void __launch_bounds__(kGnThreads) gn_slab_stats_kernel(const GroupNormArgs a, const SlabPlan s,
                                                                   float2* part) {
  __shared__ float sn[kGnThreads], sm[kGnThreads], sq[kGnThreads];
  const SlabPlace p = slab_place(s, a.C, a.G);
  const int2 rr = slab_rows(s, p, a.L);
  Moments mo{0.f, 0.f, 0.f};
  if (p.on) {
    const size_t base = (size_t)p.n * a.L * a.C + p.c;
    for (int r = rr.x + p.row; r < rr.y; r += 4 * p.step) {
      Pack<T, V> v[4];
      float x[4][V];
      const int k = min(4, (rr.y - r + p.step - 1) / p.step);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < k) v[i] = load_pack<T, V>(a.x, base + (size_t)(r + i * p.step) * a.C);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][j] = i < k ? to_f(v[i].e[j]) : 0.f;
      const float x0 = x[0][0], n = (float)(k * V);
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < k) {
#pragma unroll
          for (int j = 0; j < V; ++j) t += x[i][j] - x0;
        }
      const float mean = x0 + t / n;
      t = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < k) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float d = x[i][j] - mean;
            t = fmaf(d, d, t);
          }
        }
      if (mo.n == 0.f) mo = Moments{n, mean, t};
      else merge(mo, n, mean, t);
    }
  }
  sn[threadIdx.x] = mo.n;
  sm[threadIdx.x] = mo.mean;
  sq[threadIdx.x] = mo.m2;
  __syncthreads();
  // a warp a group: its threads' moments about the first one's mean
  const int lane = threadIdx.x & 31, per = s.parts == 1 ? s.DV : p.cols;
  for (int g = threadIdx.x >> 5; g < p.groups; g += kGnThreads / 32) {
    const int members = per * p.step;
    auto member = [&](int m) { return (m / per) * p.cols + g * per + m % per; };
    const float m0 = sm[member(0)];
    float n = 0.f, t = 0.f;
    for (int m = lane; m < members; m += 32) {
      const int i = member(m);
      if (sn[i] > 0.f) {
        n += sn[i];
        t = fmaf(sn[i], sm[i] - m0, t);
      }
    }
    n = warp_sum(n);
    const float mean = m0 + warp_sum(t) / n;
    t = 0.f;
    for (int m = lane; m < members; m += 32) {
      const int i = member(m);
      if (sn[i] > 0.f) {
        const float d = sm[i] - mean;
        t += sq[i] + sn[i] * d * d;
      }
    }
    t = warp_sum(t);
    if (lane == 0) {
      const int q = p.chunk * s.parts + (s.parts == 1 ? 0 : p.cb - p.g0 * s.parts);
      part[((size_t)p.n * a.G + p.g0 + g) * (s.chunks * s.parts) + q] = make_float2(mean, t);
    }
  }
}

// Values in slab q of a group.
__device__ __forceinline__ float slab_count(const SlabPlan& s, int L, int q) {
  const int chunk = q / s.parts, part = q - chunk * s.parts;
  const int cols = s.parts == 1 ? s.DV : min(kGnThreads, s.DV - part * kGnThreads);
  return (float)(min(s.rows, L - chunk * s.rows)) * (float)(cols * s.V);
}

template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_slab_fwd_kernel(const GroupNormArgs a, const SlabPlan s,
                                                                 const float2* part) {
  __shared__ float2 stats[kGnThreads];   // mean, rstd of the column block's groups
  const SlabPlace p = slab_place(s, a.C, a.G);
  const int lane = threadIdx.x & 31, Q = s.chunks * s.parts;
  const float count = (float)a.L * (float)(a.C / a.G);
  for (int g = threadIdx.x >> 5; g < p.groups; g += kGnThreads / 32) {
    const size_t i = (size_t)p.n * a.G + p.g0 + g;
    const float2* q = part + i * Q;
    const float m0 = q[0].x;
    float t = 0.f;
    for (int k = lane; k < Q; k += 32) t = fmaf(slab_count(s, a.L, k), q[k].x - m0, t);
    const float mean = m0 + warp_sum(t) / count;
    t = 0.f;
    for (int k = lane; k < Q; k += 32) {
      const float d = q[k].x - mean;
      t += q[k].y + slab_count(s, a.L, k) * d * d;
    }
    const float rstd = rsqrtf(warp_sum(t) / count + a.eps);
    if (lane == 0) {
      stats[g] = make_float2(mean, rstd);
      if (p.chunk == 0 && (s.parts == 1 || p.cb == p.g0 * s.parts)) {
        if (a.mean) a.mean[i] = mean;
        if (a.rstd) a.rstd[i] = rstd;
      }
    }
  }
  __syncthreads();
  if (!p.on) return;
  const int2 rr = slab_rows(s, p, a.L);
  const float2 st = stats[p.g - p.g0];
  float w[V], b[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    w[j] = param(a.weight, p.c + j, a.wb_dtype, 1.f);
    b[j] = param(a.bias, p.c + j, a.wb_dtype, 0.f);
  }
  const size_t base = (size_t)p.n * a.L * a.C + p.c;
  for (int r = rr.x + p.row; r < rr.y; r += 4 * p.step) {
    Pack<T, V> v[4], z[4];
    const int k = min(4, (rr.y - r + p.step - 1) / p.step);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < k) {
        v[i] = load_pack<T, V>(a.x, base + (size_t)(r + i * p.step) * a.C);
        if (kGate) z[i] = load_pack<T, V>(a.gate, base + (size_t)(r + i * p.step) * a.C);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < k) {
        Pack<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float u = fmaf((to_f(v[i].e[j]) - st.x) * st.y, w[j], b[j]);
          from_f(o.e[j], kGate ? u * act_value(to_f(z[i].e[j]), a.act) : act_value(u, a.act));
        }
        store_pack<T, V>(a.y, base + (size_t)(r + i * p.step) * a.C, o);
      }
  }
}

constexpr int kRowValues = 32;   // values a lane holds in the row form

template <typename T, int V, bool kGate>
void launch_fwd(const GroupNormArgs& a) {
  const RowPlan r = row_plan(a.C, a.G, a.io_dtype, kRowValues);
  if (a.L == 1 && r.lanes > 0) {
    const long long ctas = ((long long)a.N * a.G * r.lanes + kGnThreads - 1) / kGnThreads;
    const unsigned grid = (unsigned)(ctas < 152 * 32 ? ctas : 152 * 32);
    if (r.VPT == 1) gn_row_fwd_kernel<T, V, 1, kGate><<<grid, kGnThreads, 0, a.stream>>>(a, r.lanes);
    else if (r.VPT <= kRowValues / V / 2)
      gn_row_fwd_kernel<T, V, (kRowValues / V / 2), kGate><<<grid, kGnThreads, 0, a.stream>>>(a, r.lanes);
    else gn_row_fwd_kernel<T, V, kRowValues / V, kGate><<<grid, kGnThreads, 0, a.stream>>>(a, r.lanes);
    return;
  }
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  const unsigned grid = (unsigned)((long long)a.N * s.NCB * s.chunks);
  float2* part = reinterpret_cast<float2*>(a.workspace);
  gn_slab_stats_kernel<T, V><<<grid, kGnThreads, 0, a.stream>>>(a, s, part);
  gn_slab_fwd_kernel<T, V, kGate><<<grid, kGnThreads, 0, a.stream>>>(a, s, part);
}

template <typename T, int V>
void launch_fwd(const GroupNormArgs& a) {
  if (a.gate) launch_fwd<T, V, true>(a);
  else launch_fwd<T, V, false>(a);
}

}  // namespace

size_t group_norm_fwd_workspace_bytes(int N, int L, int C, int G, int io_dtype) {
  if (N == 0 || L == 0 || (L == 1 && row_plan(C, G, io_dtype, kRowValues).lanes > 0)) return 0;
  const SlabPlan s = slab_plan(N, L, C, G, io_dtype);
  return (size_t)N * G * s.chunks * s.parts * sizeof(float2);
}

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a) {
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  if ((long long)a.N * s.NCB * s.chunks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.io_dtype == GDN_F32) {
    switch (s.V) {
      case 4: launch_fwd<float, 4>(a); break;
      case 2: launch_fwd<float, 2>(a); break;
      default: launch_fwd<float, 1>(a);
    }
  } else {
    switch (s.V) {
      case 8: launch_fwd<__nv_bfloat16, 8>(a); break;
      case 4: launch_fwd<__nv_bfloat16, 4>(a); break;
      case 2: launch_fwd<__nv_bfloat16, 2>(a); break;
      default: launch_fwd<__nv_bfloat16, 1>(a);
    }
  }
  return cudaGetLastError();
}

}  // namespace gdn
