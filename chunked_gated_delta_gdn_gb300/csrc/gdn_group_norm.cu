// gdn_group_norm.cu -- group norm with an activation, channels last: the forward.
//
// For each row n and group g of D = C / G channels, over the L positions and the group's channels:
//   xhat = (x - mean) rstd,  u = xhat w + b,  y = act(u), or u act(z) with a gate z.
//
// Bound by bytes: x (and z) read once, y written once is the floor.  Two forms:
//   single positions (and small slabs) with groups of up to 1024 values: a group lives in the
//     registers of up to 32 lanes, which read it once, the next one being on its way meanwhile,
//     take mean and variance over two register passes and write it; each lane keeps its channels'
//     weights.
//   else: a launch for each slab's mean and squared deviations (merged pairwise from registers,
//     never as E[x^2] - E[x]^2), a small one that merges the slabs', and one that applies; the
//     second reading of x comes from L2 where the tensor fits it.
#include "gdn_group_norm.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ groups in registers
constexpr int kRowSteps = 4;

template <typename T, int V, int VPT, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_row_fwd_kernel(const GroupNormArgs a, const RowPlan q) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kIn = kGate ? 2 : 1;
  Ring<T, V, VPT * kIn, kRowSteps> ring(smem);
  const RowPlace p = row_place(q, a.G);
  const RowVectors<V, VPT> at(q, p, a.L, a.C, a.G);
  const float inv = 1.f / ((float)a.L * (float)(a.C / a.G));
  float w[VPT][V], b[VPT][V];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[k][j] = at.in[k] ? param(a.weight, at.c[k] + j, a.wb_dtype, 1.f) : 0.f;
      b[k][j] = at.in[k] ? param(a.bias, at.c[k] + j, a.wb_dtype, 0.f) : 0.f;
    }
  const size_t row = (size_t)a.L * a.C, col = (size_t)p.g * (a.C / a.G);
  const long long step = (long long)q.sets * q.down;
  long long n = (long long)p.set * q.down + p.down;
  auto load = [&](int ahead) {
    const long long m = n + ahead * step;
    if (m < a.N) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (at.in[k]) {
          ring.put(ahead, kIn * k, a.x, m * row + col + at.off[k]);
          if (kGate) ring.put(ahead, kIn * k + kIn - 1, a.gate, m * row + col + at.off[k]);
        }
    }
    ring.commit();
  };
#pragma unroll
  for (int i = 0; i < kRowSteps - 1; ++i) load(i);
  // (every lane of a warp runs the same number of turns: the shuffles want them all)
  const int turns = (int)((a.N + step - 1) / step);
  for (int t = 0; t < turns; ++t, n += step, ring.next()) {
    load(kRowSteps - 1);
    ring.wait();
    float v[VPT][V];
    // mean from the first element, then the squared deviations
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const Pack<T, V> x = ring.get(kIn * k);
#pragma unroll
      for (int j = 0; j < V; ++j) v[k][j] = to_f(x.e[j]);
    }
    const float x0 = __shfl_sync(0xffffffffu, v[0][0], 0, q.lanes);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at.in[k]) {
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[k][j] - x0;
      }
    const float mean = x0 + sub_sum(s, q.lanes) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at.in[k]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[k][j] -= mean;
          s = fmaf(v[k][j], v[k][j], s);
        }
      }
    const float rstd = rsqrtf(fmaf(sub_sum(s, q.lanes), inv, a.eps));
    if (n >= a.N || !p.live) continue;
    if (p.l == 0) {
      if (a.mean) a.mean[n * a.G + p.g] = mean;
      if (a.rstd) a.rstd[n * a.G + p.g] = rstd;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at.in[k]) {
        Pack<T, V> y;
        if (kGate) y = ring.get(kIn * k + kIn - 1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float u = fmaf(v[k][j] * rstd, w[k][j], b[k][j]);
          from_f(y.e[j], kGate ? u * act_value(to_f(y.e[j]), a.act) : act_value(u, a.act));
        }
        store_pack<T, V>(a.y, n * row + col + at.off[k], y);
      }
  }
}

// ------------------------------------------------------------------ slabs
// Mean and squared deviations of values; merged with those of n more (a.n = 0: taken over).
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ void merge(Moments& a, float n, float mean, float m2) {
  const float t = a.n + n, d = mean - a.mean, f = __fdividef(n, t);
  a.mean = fmaf(d, f, a.mean);
  a.m2 += m2 + d * d * a.n * f;
  a.n = t;
}

// Rows of a thread's column in its ring: about 32 KB a CTA.
template <int kPacks>
constexpr int slab_steps = kPacks == 1 ? 8 : 4;

template <typename T, int V>
__global__ void __launch_bounds__(kGnThreads) gn_slab_stats_kernel(const GroupNormArgs a, const SlabPlan s,
                                                                   float2* part) {
  __shared__ float sn[kGnThreads], sm[kGnThreads], sq[kGnThreads];
  extern __shared__ __align__(16) uint8_t smem[];
  const SlabPlace p = slab_place(s, a.C, a.G);
  const int2 rr = slab_rows(s, p, a.L);
  Moments mo{0.f, 0.f, 0.f};
  if (p.on) {
    constexpr int kSlabSteps = slab_steps<1>;
    Ring<T, V, 1, kSlabSteps> ring(smem);
    const size_t base = (size_t)p.n * a.L * a.C + p.c;
    int r = rr.x + p.row;
#pragma unroll
    for (int i = 0; i < kSlabSteps - 1; ++i) {
      if (r + i * p.step < rr.y) ring.put(i, 0, a.x, base + (size_t)(r + i * p.step) * a.C);
      ring.commit();
    }
    for (; r < rr.y; r += p.step, ring.next()) {
      const int ahead = r + (kSlabSteps - 1) * p.step;
      if (ahead < rr.y) ring.put(kSlabSteps - 1, 0, a.x, base + (size_t)ahead * a.C);
      ring.commit();
      ring.wait();
      const Pack<T, V> x = ring.get(0);
      float v[V], t = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j] = to_f(x.e[j]);
        t += v[j];
      }
      const float mean = t * (1.f / V);   // (V is a power of two)
      t = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = v[j] - mean;
        t = fmaf(d, d, t);
      }
      merge(mo, (float)V, mean, t);
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

// Mean and rstd of every group from its slabs, a warp a group.  (Merged by each CTA of the second
// launch instead, 250 slabs of 32 groups took it longer than the rest of its work.)
__global__ void __launch_bounds__(kGnThreads) gn_slab_merge_kernel(const GroupNormArgs a, const SlabPlan s,
                                                                   const float2* part, float2* stats) {
  const int lane = threadIdx.x & 31, Q = s.chunks * s.parts;
  const long long i = (long long)blockIdx.x * (kGnThreads / 32) + (threadIdx.x >> 5);
  if (i >= (long long)a.N * a.G) return;
  const float count = (float)a.L * (float)(a.C / a.G);
  const float2* q = part + i * Q;
  const float m0 = q[0].x;
  float t = 0.f;
#pragma unroll 4
  for (int k = lane; k < Q; k += 32) t = fmaf(slab_count(s, a.L, k), q[k].x - m0, t);
  const float mean = m0 + warp_sum(t) / count;
  t = 0.f;
#pragma unroll 4
  for (int k = lane; k < Q; k += 32) {
    const float2 v = q[k];
    const float d = v.x - mean;
    t += v.y + slab_count(s, a.L, k) * d * d;
  }
  const float rstd = rsqrtf(warp_sum(t) / count + a.eps);
  if (lane == 0) {
    stats[i] = make_float2(mean, rstd);
    if (a.mean) a.mean[i] = mean;
    if (a.rstd) a.rstd[i] = rstd;
  }
}

template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(kGnThreads) gn_slab_fwd_kernel(const GroupNormArgs a, const SlabPlan s,
                                                                 const float2* stats) {
  extern __shared__ __align__(16) uint8_t smem[];
  const SlabPlace p = slab_place(s, a.C, a.G);
  if (!p.on) return;
  const int2 rr = slab_rows(s, p, a.L);
  const float2 st = stats[(size_t)p.n * a.G + p.g];
  float w[V], b[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    w[j] = param(a.weight, p.c + j, a.wb_dtype, 1.f);
    b[j] = param(a.bias, p.c + j, a.wb_dtype, 0.f);
  }
  const size_t base = (size_t)p.n * a.L * a.C + p.c;
  constexpr int kIn = kGate ? 2 : 1, kSlabSteps = slab_steps<kIn>;
  Ring<T, V, kIn, kSlabSteps> ring(smem);
  int r = rr.x + p.row;
  auto load = [&](int i) {
    const int m = r + i * p.step;
    if (m < rr.y) {
      ring.put(i, 0, a.x, base + (size_t)m * a.C);
      if (kGate) ring.put(i, kIn - 1, a.gate, base + (size_t)m * a.C);
    }
    ring.commit();
  };
#pragma unroll
  for (int i = 0; i < kSlabSteps - 1; ++i) load(i);
  for (; r < rr.y; r += p.step, ring.next()) {
    load(kSlabSteps - 1);
    ring.wait();
    const Pack<T, V> x = ring.get(0);
    Pack<T, V> y;
    if (kGate) y = ring.get(kIn - 1);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float u = fmaf((to_f(x.e[j]) - st.x) * st.y, w[j], b[j]);
      from_f(y.e[j], kGate ? u * act_value(to_f(y.e[j]), a.act) : act_value(u, a.act));
    }
    store_pack<T, V>(a.y, base + (size_t)r * a.C, y);
  }
}

constexpr int kRowValues = 32;   // values a lane holds in the row form
constexpr int kRowPerSm = 5;     // its CTAs an SM (registers)

template <typename T, int V, int VPT, bool kGate>
cudaError_t launch_row_fwd(const GroupNormArgs& a, const RowPlan& r) {
  constexpr int kShared = Ring<T, V, VPT * (kGate ? 2 : 1), kRowSteps>::kShared;
  const cudaError_t err = allow_shared<gn_row_fwd_kernel<T, V, VPT, kGate>, kShared>();
  if (err != cudaSuccess) return err;
  gn_row_fwd_kernel<T, V, VPT, kGate><<<(unsigned)(r.sets * r.across), kGnThreads, kShared, a.stream>>>(a, r);
  return cudaGetLastError();
}

template <typename T, int V, bool kGate>
cudaError_t launch_fwd(const GroupNormArgs& a) {
  const RowPlan r = row_plan(a.N, a.L, a.C, a.G, a.io_dtype, kRowValues, kRowPerSm);
  if (r.lanes > 0) {
    if (r.VPT == 1) return launch_row_fwd<T, V, 1, kGate>(a, r);
    if (r.VPT <= kRowValues / V / 2) return launch_row_fwd<T, V, kRowValues / V / 2, kGate>(a, r);
    return launch_row_fwd<T, V, kRowValues / V, kGate>(a, r);
  }
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  const unsigned grid = (unsigned)((long long)a.N * s.NCB * s.chunks);
  float2* part = reinterpret_cast<float2*>(a.workspace);
  constexpr int kStats = Ring<T, V, 1, slab_steps<1>>::kShared;
  constexpr int kApply = Ring<T, V, kGate ? 2 : 1, slab_steps<kGate ? 2 : 1>>::kShared;
  const cudaError_t err = allow_shared<gn_slab_fwd_kernel<T, V, kGate>, kApply>();
  if (err != cudaSuccess) return err;
  gn_slab_stats_kernel<T, V><<<grid, kGnThreads, kStats, a.stream>>>(a, s, part);
  float2* stats = part + (size_t)a.N * a.G * s.chunks * s.parts;
  const unsigned warps = kGnThreads / 32, merge_grid = (unsigned)(((long long)a.N * a.G + warps - 1) / warps);
  gn_slab_merge_kernel<<<merge_grid, kGnThreads, 0, a.stream>>>(a, s, part, stats);
  gn_slab_fwd_kernel<T, V, kGate><<<grid, kGnThreads, kApply, a.stream>>>(a, s, stats);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_fwd(const GroupNormArgs& a) {
  return a.gate ? launch_fwd<T, V, true>(a) : launch_fwd<T, V, false>(a);
}

}  // namespace

size_t group_norm_fwd_workspace_bytes(int N, int L, int C, int G, int io_dtype) {
  if (N == 0 || L == 0 || row_plan(N, L, C, G, io_dtype, kRowValues, kRowPerSm).lanes > 0) return 0;
  const SlabPlan s = slab_plan(N, L, C, G, io_dtype);
  return (size_t)N * G * (s.chunks * s.parts + 1) * sizeof(float2);
}

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a) {
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  if ((long long)a.N * s.NCB * s.chunks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.io_dtype == GDN_F32) {
    switch (s.V) {
      case 4: return launch_fwd<float, 4>(a);
      case 2: return launch_fwd<float, 2>(a);
      default: return launch_fwd<float, 1>(a);
    }
  }
  switch (s.V) {
    case 8: return launch_fwd<__nv_bfloat16, 8>(a);
    case 4: return launch_fwd<__nv_bfloat16, 4>(a);
    case 2: return launch_fwd<__nv_bfloat16, 2>(a);
    default: return launch_fwd<__nv_bfloat16, 1>(a);
  }
}

}  // namespace gdn
