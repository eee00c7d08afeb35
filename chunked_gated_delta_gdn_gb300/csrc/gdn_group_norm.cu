// gdn_group_norm.cu -- group norm with an activation, channels last: the forward.
//
// For each row n and group g of D = C / G channels, over the L positions and the group's channels:
//   xhat = (x - mean) rstd,  u = xhat w + b,  y = act(u), or u act(z) with a gate z.
//
// Bound by bytes: x (and z) read once, y written once is the floor.  Two forms:
//   single positions (and small slabs) with groups of up to 1024 values: a group lives in the
//     registers of up to 32 lanes, which read it once, the next one being on its way meanwhile,
//     take mean and variance over two register passes and write it; each lane keeps its channels'
//     weights.  16384 rows of 4096 with a gate in bf16: 72 us for 403 MB, 5.6 TB/s.
//   else: a launch for each slab's mean and squared deviations (summed about a value of their own,
//     never as E[x^2] - E[x]^2, and merged), a small one that merges the slabs', and one that
//     applies; the second reading of x comes from L2 where the tensor fits it.  8 x 16384
//     positions of 256 channels in bf16: 19 + 3 + 18 us, 67 MB read twice and written once.
// Instructions count as much as bytes here: 16 to 19 an element, in scalar arithmetic, took 88 us
// and 23 + 3 + 25; hence pairs, unrolled rings, and no more CTAs than keep the copies in flight
// (the slabs' 19 + 18 us are 22 + 19 with five CTAs an SM instead of three).
#include "gdn_group_norm.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ groups in registers
constexpr int kRowValues = 32;   // values a lane holds
constexpr int kRowPerSm = 4;     // CTAs an SM (registers)
// Steps of a lane's ring: four, or what a CTA's shared memory holds (three of 64 KB for 32 fp32 values
// a lane with a gate).
template <typename T, int V, int VPT, bool kGate>
constexpr int row_steps = std::min(4, kMaxDynamic / (VPT * (kGate ? 2 : 1) * V * (int)sizeof(T) * kGnThreads));

template <typename T, int V, int VPT, bool kGate>
__global__ void __launch_bounds__(kGnThreads, VPT == 1 ? kRowPerSm : 1)
    gn_row_fwd_kernel(const GroupNormArgs a, const RowPlan q) {
  extern __shared__ __align__(16) uint8_t smem[];
  using P = Pair<V>;
  constexpr int kIn = kGate ? 2 : 1, kP = kPairs<V>;
  const RowPlace p = row_place(q, a.G);
  const RowVectors<V, VPT> at(q, p, a.L, a.C, a.G);
  const float inv = 1.f / ((float)a.L * (float)(a.C / a.G));
  P w[VPT][kP], b[VPT][kP];
  const RowRange rg = row_range(q, p, a.N);
  size_t from[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    from[k] = (size_t)rg.n0 * a.L * a.C + (size_t)p.g * (a.C / a.G) + at.off[k];
    if (at.in[k]) {
      params<V>(a.weight, at.c[k], a.wb_dtype, 1.f, w[k]);
      params<V>(a.bias, at.c[k], a.wb_dtype, 0.f, b[k]);
    }
  }
  const void* src[kIn];
  src[0] = a.x;
  if (kGate) src[kIn - 1] = a.gate;
  const size_t stride = (size_t)rg.step * a.L * a.C;
  walk<T, V, VPT, kIn, row_steps<T, V, VPT, kGate>>(smem, src, from, at.in, stride, rg.mine, rg.turns,
                                                    [&](auto& ring, int u, int t, size_t here) {
    // about the group's first value: the mean, then the squared deviations
    P v[VPT][kP];
#pragma unroll
    for (int k = 0; k < VPT; ++k) unpack<V>(ring.get(u, kIn * k), v[k]);
    float x0;
    if constexpr (V == 1) x0 = v[0][0];
    else x0 = v[0][0].x;
    x0 = __shfl_sync(0xffffffffu, x0, 0, q.lanes);
    P s = both<P>(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at.in[k]) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          v[k][i] = add(v[k][i], both<P>(-x0));
          s = add(s, v[k][i]);
        }
      }
    const float d = sub_sum(sum(s), q.lanes) * inv;
    s = both<P>(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at.in[k]) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          v[k][i] = add(v[k][i], both<P>(-d));
          s = fma(v[k][i], v[k][i], s);
        }
      }
    const float rstd = rsqrtf(fmaf(sub_sum(sum(s), q.lanes), inv, a.eps));
    if (t >= rg.mine || !p.live) return;
    if (p.l == 0) {
      const long long n = rg.n0 + (long long)t * rg.step;
      if (a.mean) a.mean[n * a.G + p.g] = x0 + d;
      if (a.rstd) a.rstd[n * a.G + p.g] = rstd;
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at.in[k]) {
        Pack<T, V> y;
        P z[kP];
        if (kGate) unpack<V>(ring.get(u, kIn * k + kIn - 1), z);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const P h = fma(mul(v[k][i], both<P>(rstd)), w[k][i], b[k][i]);
          pack<V>(y, i, kGate ? mul(h, act_value(z[i], a.act)) : act_value(h, a.act));
        }
        store_pack<T, V>(a.y, from[k] + here, y);
      }
  });
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
__global__ void __launch_bounds__(kGnThreads, kSlabPerSm)
    gn_slab_stats_kernel(const GroupNormArgs a, const SlabPlan s, float2* part) {
  __shared__ float sn[kGnThreads], sm[kGnThreads], sq[kGnThreads];
  extern __shared__ __align__(16) uint8_t smem[];
  using P = Pair<V>;
  constexpr int kP = kPairs<V>;
  const SlabPlace p = slab_place(s, a.C, a.G);
  const SlabRange rr = slab_range(s, p, a.L, a.C);
  next_may_start();
  Moments mo{0.f, 0.f, 0.f};
  if (p.on) {
    // Eight rows at a time: sums and squares about the mean of the first pack (so that squares much
    // larger than the deviations cannot stand in one block), then merged.
    float pivot = 0.f, n = 0.f;
    P s1 = both<P>(0.f), s2 = both<P>(0.f);
    auto close = [&] {
      const float t = sum(s1), f = __fdividef(1.f, n);
      merge(mo, n, fmaf(t, f, pivot), fmaxf(fmaf(-t * f, t, sum(s2)), 0.f));
    };
    const void* src[1] = {a.x};
    const size_t from[1] = {rr.from};
    const bool in[1] = {true};
    walk<T, V, 1, 1, slab_steps<1>>(smem, src, from, in, rr.stride, rr.rows, rr.rows,
                                    [&](auto& ring, int u, int t, size_t) {
      P v[kP];
      unpack<V>(ring.get(u, 0), v);
      if (u == 0) {
        if (t > 0) close();
        P m = v[0];
#pragma unroll
        for (int i = 1; i < kP; ++i) m = add(m, v[i]);
        pivot = sum(m) * (1.f / V);
        s1 = s2 = both<P>(0.f);
        n = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const P d = add(v[i], both<P>(-pivot));
        s1 = add(s1, d);
        s2 = fma(d, d, s2);
      }
      n += (float)V;
    });
    if (rr.rows > 0) close();
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
  next_may_start();
  wait_for_previous();
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
__global__ void __launch_bounds__(kGnThreads, kSlabPerSm)
    gn_slab_fwd_kernel(const GroupNormArgs a, const SlabPlan s, const float2* stats) {
  extern __shared__ __align__(16) uint8_t smem[];
  using P = Pair<V>;
  constexpr int kIn = kGate ? 2 : 1, kP = kPairs<V>;
  const SlabPlace p = slab_place(s, a.C, a.G);
  P w[kP], b[kP];
  if (p.on) {
    params<V>(a.weight, p.c, a.wb_dtype, 1.f, w);
    params<V>(a.bias, p.c, a.wb_dtype, 0.f, b);
  }
  wait_for_previous();
  if (!p.on) return;
  const SlabRange rr = slab_range(s, p, a.L, a.C);
  const float2 st = stats[(size_t)p.n * a.G + p.g];
#pragma unroll
  for (int i = 0; i < kP; ++i) w[i] = mul(w[i], both<P>(st.y));
  const void* src[kIn];
  src[0] = a.x;
  if (kGate) src[kIn - 1] = a.gate;
  const size_t from[1] = {rr.from};
  const bool in[1] = {true};
  walk<T, V, 1, kIn, slab_steps<kIn>>(smem, src, from, in, rr.stride, rr.rows, rr.rows,
                                      [&](auto& ring, int u, int, size_t here) {
    P v[kP], z[kP];
    unpack<V>(ring.get(u, 0), v);
    if (kGate) unpack<V>(ring.get(u, kIn - 1), z);
    Pack<T, V> y;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const P h = fma(add(v[i], both<P>(-st.x)), w[i], b[i]);
      pack<V>(y, i, kGate ? mul(h, act_value(z[i], a.act)) : act_value(h, a.act));
    }
    store_pack<T, V>(a.y, rr.from + here, y);
  });
}


template <typename T, int V, int VPT, bool kGate>
cudaError_t launch_row_fwd(const GroupNormArgs& a, const RowPlan& r) {
  constexpr int kShared = Ring<T, V, VPT * (kGate ? 2 : 1), row_steps<T, V, VPT, kGate>>::kShared;
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
  cudaError_t err = allow_shared<gn_slab_fwd_kernel<T, V, kGate>, kApply>();
  if (err != cudaSuccess) return err;
  gn_slab_stats_kernel<T, V><<<grid, kGnThreads, kStats, a.stream>>>(a, s, part);
  float2* stats = part + (size_t)a.N * a.G * s.chunks * s.parts;
  const unsigned warps = kGnThreads / 32, merge_grid = (unsigned)(((long long)a.N * a.G + warps - 1) / warps);
  if ((err = cudaGetLastError()) != cudaSuccess ||
      (err = launch_behind(gn_slab_merge_kernel, merge_grid, kGnThreads, 0, a.stream, a, s, part, stats)) != cudaSuccess)
    return err;
  return launch_behind(gn_slab_fwd_kernel<T, V, kGate>, grid, kGnThreads, kApply, a.stream, a, s, stats);
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
