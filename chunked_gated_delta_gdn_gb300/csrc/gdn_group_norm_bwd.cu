// gdn_group_norm_bwd.cu -- group norm with an activation, channels last: the backward.
//
// With s the activation, du = dy s'(u) (gate: du = dy s(z), dz = dy u s'(z)):
//   dw_c = sum du xhat,  db_c = sum du   over rows and positions,
//   dx = rstd (du w - m1 - xhat m2),     m1, m2 the group's means of du w and du w xhat.
//
// A thread keeps its channels and sums du and du xhat for each of them (A, B): those are its share
// of db and dw, and sum_c w_c A_c, sum_c w_c B_c its share of m1 and m2.  Every sum is made in a
// fixed order.  Bound by bytes: x, dy (and z) read once, dx (and dz) written once is the floor.
//   single positions (and small slabs) with groups of up to 512 values: one launch reads each row
//     once, its groups in registers, the next row being on its way, and leaves A, B of each set of
//     rows; a second adds the sets.  16384 rows of 4096 with a gate in bf16: 117 + 3 us for 671 MB,
//     5.7 TB/s (three CTAs an SM, whose registers spilled, 140).
//   else: a launch for A, B and the slab's share of m1, m2, a small one that adds the shares up, and
//     one that reads x, dy (and z) again and applies, its last CTAs adding A, B up.
#include "gdn_group_norm.cuh"

namespace gdn {
namespace {

// xhat and du of one element (and dz).
template <bool kGate, typename P>
__device__ __forceinline__ P grad_u(P x, P dy, P z, float mean, float rstd, P w, P b, int act, P* xhat, P* dz) {
  const P xh = mul(add(x, both<P>(-mean)), both<P>(rstd)), u = fma(xh, w, b);
  P slope;
  *xhat = xh;
  const P value = act_both(kGate ? z : u, act, &slope);
  if (!kGate) return mul(dy, slope);
  *dz = mul(mul(dy, u), slope);
  return mul(dy, value);
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
  wait_for_previous();
  sum_sets<32>(a, part, sets, blockIdx.x);
}

// ------------------------------------------------------------------ groups in registers
constexpr int kRowSteps = 3;
constexpr int kRowValues = 16;   // values a lane holds
constexpr int kRowPerSm = 2;     // CTAs an SM (registers)

template <typename T, int V, int VPT, bool kGate>
__global__ void __launch_bounds__(kGnThreads, VPT == 1 ? kRowPerSm : 1)
    gn_row_bwd_kernel(const GroupNormArgs a, const RowPlan q, float* part) {
  extern __shared__ __align__(16) uint8_t smem[];
  using P = Pair<V>;
  constexpr int kIn = kGate ? 3 : 2, kP = kPairs<V>;
  next_may_start();
  const RowPlace p = row_place(q, a.G);
  const RowVectors<V, VPT> at(q, p, a.L, a.C, a.G);
  const int D = a.C / a.G;
  const float inv = 1.f / ((float)a.L * (float)D);
  P w[VPT][kP], b[VPT][kP], A[VPT][kP], B[VPT][kP];
  const RowRange rg = row_range(q, p, a.N);
  size_t from[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    from[k] = (size_t)rg.n0 * a.L * a.C + (size_t)p.g * D + at.off[k];
    if (at.in[k]) {
      params<V>(a.weight, at.c[k], a.wb_dtype, 1.f, w[k]);
      params<V>(a.bias, at.c[k], a.wb_dtype, 0.f, b[k]);
    }
#pragma unroll
    for (int i = 0; i < kP; ++i) A[k][i] = B[k][i] = both<P>(0.f);
  }
  float nmean = 0.f, nrstd = 0.f;
  auto load_stats = [&](int t) {
    if (t < rg.mine && p.live) {
      const long long i = (rg.n0 + t * rg.step) * a.G + p.g;
      nmean = a.mean[i];
      nrstd = a.rstd[i];
    }
  };
  load_stats(0);
  const void* src[kIn];
  src[0] = a.x;
  src[1] = a.dy;
  if (kGate) src[kIn - 1] = a.gate;
  const size_t stride = (size_t)rg.step * a.L * a.C;
  walk<T, V, VPT, kIn, kRowSteps>(smem, src, from, at.in, stride, rg.mine, rg.turns,
                                  [&](auto& ring, int u, int t, size_t here) {
    const bool on = t < rg.mine;
    const float mean = nmean, rstd = nrstd;
    load_stats(t + 1);
    P xh[VPT][kP], d[VPT][kP], s1 = both<P>(0.f), s2 = both<P>(0.f);
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on && at.in[k]) {
        P x[kP], dy[kP], z[kP];
        unpack<V>(ring.get(u, kIn * k), x);
        unpack<V>(ring.get(u, kIn * k + 1), dy);
        if (kGate) unpack<V>(ring.get(u, kIn * k + kIn - 1), z);
        Pack<T, V> o;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          P dz;
          const P du = grad_u<kGate>(x[i], dy[i], z[i], mean, rstd, w[k][i], b[k][i], a.act, &xh[k][i], &dz);
          if (kGate) pack<V>(o, i, dz);
          A[k][i] = add(A[k][i], du);
          B[k][i] = fma(du, xh[k][i], B[k][i]);
          d[k][i] = mul(du, w[k][i]);
          s1 = add(s1, d[k][i]);
          s2 = fma(d[k][i], xh[k][i], s2);
        }
        if (kGate) store_pack<T, V>(a.dgate, from[k] + here, o);
      }
    const float m1 = sub_sum(sum(s1), q.lanes) * inv, m2 = sub_sum(sum(s2), q.lanes) * inv;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (on && at.in[k]) {
        Pack<T, V> o;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const P e = fma(xh[k][i], both<P>(-m2), add(d[k][i], both<P>(-m1)));
          pack<V>(o, i, mul(e, both<P>(rstd)));
        }
        store_pack<T, V>(a.dx, from[k] + here, o);
      }
  });
  if (!part) return;
  // A, B over the CTA's rows and positions: every value through shared memory, summed in order
  // (256 lanes of VPT V values each; the rings are done with).  First channel, channels of the CTA:
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float(*acc)[kGnThreads * VPT * V] = reinterpret_cast<float(*)[kGnThreads * VPT * V]>(smem);
  const int c0 = q.across == 1 ? 0 : (blockIdx.x % q.across) * q.J * D;
  const int nc = q.across == 1 ? a.C : min(q.J * D, a.C - c0);
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    if (at.in[k]) {
      const int r = p.down * a.L + at.off[k] / a.C, e = r * nc + at.c[k] - c0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        acc[0][e + j] = reinterpret_cast<const float*>(A[k])[j];
        acc[1][e + j] = reinterpret_cast<const float*>(B[k])[j];
      }
    }
  __syncthreads();
  float* out = part + (size_t)p.set * 2 * a.C + c0;
  for (int c = threadIdx.x; c < nc; c += kGnThreads) {
    float x = 0.f, y = 0.f;
    for (int r = 0; r < q.down * a.L; ++r) {
      x += acc[0][r * nc + c];
      y += acc[1][r * nc + c];
    }
    out[c] = x;
    out[a.C + c] = y;
  }
}

// ------------------------------------------------------------------ slabs
constexpr int kSlabSteps = 4;   // rows of a thread's column in its ring

// Walks down a thread's column: f(x, dy, z, distance).
template <typename T, int V, bool kGate, class F>
__device__ __forceinline__ void walk_slab(const GroupNormArgs& a, const SlabRange& rr, void* smem, F&& f) {
  constexpr int kIn = kGate ? 3 : 2, kP = kPairs<V>;
  const void* src[kIn];
  src[0] = a.x;
  src[1] = a.dy;
  if (kGate) src[kIn - 1] = a.gate;
  const size_t from[1] = {rr.from};
  const bool in[1] = {true};
  walk<T, V, 1, kIn, kSlabSteps>(smem, src, from, in, rr.stride, rr.rows, rr.rows,
                                 [&](auto& ring, int u, int, size_t here) {
    Pair<V> x[kP], dy[kP], z[kP];
    unpack<V>(ring.get(u, 0), x);
    unpack<V>(ring.get(u, 1), dy);
    if (kGate) unpack<V>(ring.get(u, kIn - 1), z);
    f(x, dy, z, here);
  });
}

// part [n][chunk][2][C]: A, B; share [n][g][chunk][parts]: (sum du w, sum du w xhat) of the slab.
template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(kGnThreads, kSlabPerSm)
    gn_slab_grad_kernel(const GroupNormArgs a, const SlabPlan s, float* part, float2* share) {
  extern __shared__ __align__(16) uint8_t smem[];
  const SlabPlace p = slab_place(s, a.C, a.G);
  using P = Pair<V>;
  constexpr int kP = kPairs<V>;
  next_may_start();
  P Ap[kP], Bp[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) Ap[i] = Bp[i] = both<P>(0.f);
  if (p.on) {
    const float mean = a.mean[(size_t)p.n * a.G + p.g], rstd = a.rstd[(size_t)p.n * a.G + p.g];
    P w[kP], b[kP];
    params<V>(a.weight, p.c, a.wb_dtype, 1.f, w);
    params<V>(a.bias, p.c, a.wb_dtype, 0.f, b);
    walk_slab<T, V, kGate>(a, slab_range(s, p, a.L, a.C), smem, [&](P(&x)[kP], P(&dy)[kP], P(&z)[kP], size_t) {
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        P xh, dz;
        const P du = grad_u<kGate>(x[i], dy[i], z[i], mean, rstd, w[i], b[i], a.act, &xh, &dz);
        Ap[i] = add(Ap[i], du);
        Bp[i] = fma(du, xh, Bp[i]);
      }
    });
  }
  float A[V], B[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    A[j] = reinterpret_cast<const float*>(Ap)[j];
    B[j] = reinterpret_cast<const float*>(Bp)[j];
  }
  // (the rings are done with; a thread's own copies have landed)
  __syncthreads();
  float* sa = reinterpret_cast<float*>(smem);
  float* sb = sa + kGnThreads * V;
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
      const float w = a.weight ? load_elem(a.weight, p.c + j, a.wb_dtype) : 1.f;
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

// m1, m2 of every group from its slabs' shares, a warp a group.
__global__ void __launch_bounds__(kGnThreads) gn_slab_means_kernel(const GroupNormArgs a, int Q, const float2* share,
                                                                   float2* means) {
  next_may_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * (kGnThreads / 32) + (threadIdx.x >> 5);
  if (i >= (long long)a.N * a.G) return;
  const float inv = 1.f / ((float)a.L * (float)(a.C / a.G));
  float x = 0.f, y = 0.f;
#pragma unroll 4
  for (int k = lane; k < Q; k += 32) {
    const float2 v = share[i * Q + k];
    x += v.x;
    y += v.y;
  }
  x = warp_sum(x);
  y = warp_sum(y);
  if (lane == 0) means[i] = make_float2(x * inv, y * inv);
}

template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(kGnThreads, kSlabPerSm)
    gn_slab_bwd_kernel(const GroupNormArgs a, const SlabPlan s, int slabs, const float* part, const float2* means) {
  wait_for_previous();
  if ((int)blockIdx.x >= slabs) {
    sum_sets<kGnThreads / 32>(a, part, a.N * s.chunks, blockIdx.x - slabs);
    return;
  }
  extern __shared__ __align__(16) uint8_t smem[];
  const SlabPlace p = slab_place(s, a.C, a.G);
  if (!p.on) return;
  using P = Pair<V>;
  constexpr int kP = kPairs<V>;
  const SlabRange rr = slab_range(s, p, a.L, a.C);
  const float mean = a.mean[(size_t)p.n * a.G + p.g], rstd = a.rstd[(size_t)p.n * a.G + p.g];
  const float2 m = means[(size_t)p.n * a.G + p.g];
  P w[kP], b[kP];
  params<V>(a.weight, p.c, a.wb_dtype, 1.f, w);
  params<V>(a.bias, p.c, a.wb_dtype, 0.f, b);
  walk_slab<T, V, kGate>(a, rr, smem, [&](P(&x)[kP], P(&dy)[kP], P(&z)[kP], size_t here) {
    Pack<T, V> o, oz;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      P xh, dz;
      const P du = grad_u<kGate>(x[i], dy[i], z[i], mean, rstd, w[i], b[i], a.act, &xh, &dz);
      const P e = fma(xh, both<P>(-m.y), fma(du, w[i], both<P>(-m.x)));
      pack<V>(o, i, mul(e, both<P>(rstd)));
      if (kGate) pack<V>(oz, i, dz);
    }
    store_pack<T, V>(a.dx, rr.from + here, o);
    if (kGate) store_pack<T, V>(a.dgate, rr.from + here, oz);
  });
}


size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T, int V, int VPT, bool kGate>
cudaError_t launch_row_bwd(const GroupNormArgs& a, const RowPlan& r, float* part) {
  constexpr int kRing = Ring<T, V, VPT * (kGate ? 3 : 2), kRowSteps>::kShared;
  constexpr int kSums = 2 * kGnThreads * VPT * V * (int)sizeof(float);
  constexpr int kShared = kRing > kSums ? kRing : kSums;
  const cudaError_t err = allow_shared<gn_row_bwd_kernel<T, V, VPT, kGate>, kShared>();
  if (err != cudaSuccess) return err;
  gn_row_bwd_kernel<T, V, VPT, kGate><<<(unsigned)(r.sets * r.across), kGnThreads, kShared, a.stream>>>(a, r, part);
  return cudaGetLastError();
}

template <typename T, int V, bool kGate>
cudaError_t launch_bwd(const GroupNormArgs& a) {
  const bool params = a.dweight || a.dbias;
  const RowPlan r = row_plan(a.N, a.L, a.C, a.G, a.io_dtype, kRowValues, kRowPerSm);
  float* part = reinterpret_cast<float*>(a.workspace);
  const unsigned sum_ctas = (unsigned)((a.C + 31) / 32);
  cudaError_t err;
  if (r.lanes > 0) {
    float* to = params ? part : nullptr;
    err = r.VPT == 1 ? launch_row_bwd<T, V, 1, kGate>(a, r, to)
                     : launch_row_bwd<T, V, kRowValues / V, kGate>(a, r, to);
    if (err != cudaSuccess || !params) return err;
    return launch_behind(gn_sum_sets_kernel, sum_ctas, 1024, 0, a.stream, a, part, r.sets);
  }
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  const int slabs = a.N * s.NCB * s.chunks;
  float2* share = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(a.workspace) +
                                            align256((size_t)a.N * s.chunks * 2 * a.C * sizeof(float)));
  constexpr int kRing = Ring<T, V, kGate ? 3 : 2, kSlabSteps>::kShared;
  constexpr int kSums = 2 * kGnThreads * V * (int)sizeof(float);
  constexpr int kGrad = kRing > kSums ? kRing : kSums;
  if ((err = allow_shared<gn_slab_grad_kernel<T, V, kGate>, kGrad>()) != cudaSuccess ||
      (err = allow_shared<gn_slab_bwd_kernel<T, V, kGate>, kRing>()) != cudaSuccess)
    return err;
  gn_slab_grad_kernel<T, V, kGate><<<slabs, kGnThreads, kGrad, a.stream>>>(a, s, part, share);
  const int Q = s.chunks * s.parts;
  float2* means = share + (size_t)a.N * a.G * Q;
  const unsigned warps = kGnThreads / 32, means_grid = (unsigned)(((long long)a.N * a.G + warps - 1) / warps);
  if ((err = cudaGetLastError()) != cudaSuccess ||
      (err = launch_behind(gn_slab_means_kernel, means_grid, kGnThreads, 0, a.stream, a, Q, share, means)) !=
          cudaSuccess)
    return err;
  return launch_behind(gn_slab_bwd_kernel<T, V, kGate>, slabs + (params ? sum_ctas : 0), kGnThreads, kRing, a.stream,
                       a, s, slabs, part, means);
}

template <typename T, int V>
cudaError_t launch_bwd(const GroupNormArgs& a) {
  return a.gate ? launch_bwd<T, V, true>(a) : launch_bwd<T, V, false>(a);
}

}  // namespace

size_t group_norm_bwd_workspace_bytes(int N, int L, int C, int G, int io_dtype) {
  if (N == 0 || L == 0) return 0;
  const RowPlan r = row_plan(N, L, C, G, io_dtype, kRowValues, kRowPerSm);
  if (r.lanes > 0) return align256((size_t)r.sets * 2 * C * sizeof(float));
  const SlabPlan s = slab_plan(N, L, C, G, io_dtype);
  return align256((size_t)N * s.chunks * 2 * C * sizeof(float)) +
         align256((size_t)N * G * (s.chunks * s.parts + 1) * sizeof(float2));
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs& a) {
  const SlabPlan s = slab_plan(a.N, a.L, a.C, a.G, a.io_dtype);
  if ((long long)a.N * s.NCB * s.chunks + a.C > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.io_dtype == GDN_F32) {
    switch (s.V) {
      case 4: return launch_bwd<float, 4>(a);
      case 2: return launch_bwd<float, 2>(a);
      default: return launch_bwd<float, 1>(a);
    }
  }
  switch (s.V) {
    case 8: return launch_bwd<__nv_bfloat16, 8>(a);
    case 4: return launch_bwd<__nv_bfloat16, 4>(a);
    case 2: return launch_bwd<__nv_bfloat16, 2>(a);
    default: return launch_bwd<__nv_bfloat16, 1>(a);
  }
}

}  // namespace gdn
