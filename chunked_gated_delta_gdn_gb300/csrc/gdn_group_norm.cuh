// gdn_group_norm.cuh -- what the forward and backward kernels of group norm share.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_group_norm.h"
#include "gdn_launch.cuh"

namespace gdn {
namespace {

constexpr int kGnThreads = 256;
constexpr int kSlabPerSm = 3;   // CTAs an SM in the slab form (registers)

// V consecutive elements in one load: V sizeof(T) is 2, 4, 8 or 16 bytes.
template <int kBytes> struct Raw;
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T e[V];
};
// The arithmetic, on pairs (two values an instruction), or on one where a pack holds one.
template <int V> using Pair = std::conditional_t<V == 1, float, float2>;
template <int V> constexpr int kPairs = V == 1 ? 1 : V / 2;
__device__ __forceinline__ unsigned long long bits(float2 a) { return *reinterpret_cast<unsigned long long*>(&a); }
__device__ __forceinline__ float2 pair_of(unsigned long long a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair_of(d);
}
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair_of(d);
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair_of(d);
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float sum(float a) { return a; }
template <typename P> __device__ __forceinline__ P both(float x);
template <> __device__ __forceinline__ float2 both<float2>(float x) { return make_float2(x, x); }
template <> __device__ __forceinline__ float both<float>(float x) { return x; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }

// 1 / (1 + 2^(-x log2 e)); and the activation's value and slope s (1 + x (1 - s)).
template <typename P>
__device__ __forceinline__ P sigmoid(P x) {
  return rcp(add(ex2(mul(x, both<P>(-1.4426950408889634f))), both<P>(1.f)));
}
template <typename P>
__device__ __forceinline__ P act_value(P x, int act) {
  return act == GDN_ACT_SILU ? mul(x, sigmoid(x)) : x;
}
template <typename P>
__device__ __forceinline__ P act_both(P x, int act, P* slope) {
  if (act != GDN_ACT_SILU) {
    *slope = both<P>(1.f);
    return x;
  }
  const P s = sigmoid(x), v = mul(x, s);
  *slope = fma(v, fma(s, both<P>(-1.f), both<P>(1.f)), s);
  return v;
}

template <int V>
__device__ __forceinline__ void unpack(const Pack<float, V>& p, Pair<V> (&v)[kPairs<V>]) {
  if constexpr (V == 1) v[0] = p.e[0];
  else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = make_float2(p.e[2 * i], p.e[2 * i + 1]);
  }
}
template <int V>
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, V>& p, Pair<V> (&v)[kPairs<V>]) {
  if constexpr (V == 1) v[0] = __bfloat162float(p.e[0]);
  else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const uint32_t u = reinterpret_cast<const uint32_t*>(p.e)[i];
      v[i] = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
  }
}
template <int V>
__device__ __forceinline__ void pack(Pack<float, V>& p, int i, Pair<V> v) {
  if constexpr (V == 1) p.e[0] = v;
  else {
    p.e[2 * i] = v.x;
    p.e[2 * i + 1] = v.y;
  }
}
template <int V>
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, V>& p, int i, Pair<V> v) {
  if constexpr (V == 1) p.e[0] = __float2bfloat16_rn(v);
  else reinterpret_cast<__nv_bfloat162*>(p.e)[i] = __float22bfloat162_rn(v);
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const void* base, size_t at) {
  Pack<T, V> p;
  using R = typename Raw<V * sizeof(T)>::type;
  *reinterpret_cast<R*>(&p) = *reinterpret_cast<const R*>(reinterpret_cast<const T*>(base) + at);
  return p;
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(void* base, size_t at, const Pack<T, V>& p) {
  using R = typename Raw<V * sizeof(T)>::type;
  *reinterpret_cast<R*>(reinterpret_cast<T*>(base) + at) = *reinterpret_cast<const R*>(&p);
}

// A thread's own ring of packs in shared memory, filled by asynchronous copies (no registers and
// no other thread involved: only its own group count is waited for).  kPacks packs a step, kSteps
// steps deep.  2-byte packs, which such copies do not move, are copied at once.
template <typename T, int V, int kPacks, int kSteps>
struct Ring {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int kShared = kSteps * kPacks * kBytes * kGnThreads;
  uint8_t* mine;
  __device__ __forceinline__ explicit Ring(void* smem)
      : mine(reinterpret_cast<uint8_t*>(smem) + threadIdx.x * kBytes) {}
  __device__ __forceinline__ uint8_t* slot(int step, int i) const {
    return mine + (step * kPacks + i) * kBytes * kGnThreads;
  }
  __device__ __forceinline__ void put(int step, int i, const T* src) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot(step, i));
    if (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (kBytes >= 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes < 4 ? 4 : kBytes)
                   : "memory");
    else *reinterpret_cast<Pack<T, V>*>(slot(step, i)) = load_pack<T, V>(src, 0);
  }
  __device__ __forceinline__ Pack<T, V> get(int step, int i) const { return load_pack<T, V>(slot(step, i), 0); }
};

// Walks over `turns` turns of VPT places, `stride` elements from one turn to the next, with kIn
// tensors a place: f(ring, step, turn, distance) finds tensor i of place k as ring.get(step, kIn k
// + i).  Of each place `mine` turns are read, and only where in[k]; the copies run kSteps - 1 turns
// ahead.  (Unrolled over the ring, so that its steps are constants.)
template <typename T, int V, int VPT, int kIn, int kSteps, class F>
__device__ __forceinline__ void walk(void* smem, const void* const (&src)[kIn], const size_t (&at)[VPT],
                                     const bool (&in)[VPT], size_t stride, int mine, int turns, F&& f) {
  Ring<T, V, VPT * kIn, kSteps> ring(smem);
  size_t ahead = 0, here = 0;   // distances of the next copies, and of the turn at hand
  auto load = [&](int step, int t) {
    if (t < mine) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        if (in[k]) {
#pragma unroll
          for (int i = 0; i < kIn; ++i)
            ring.put(step, kIn * k + i, reinterpret_cast<const T*>(src[i]) + (at[k] + ahead));
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += stride;
  };
#pragma unroll
  for (int i = 0; i < kSteps - 1; ++i) load(i, i);
  for (int t0 = 0; t0 < turns; t0 += kSteps) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      if (t0 + u >= turns) break;
      load((u + kSteps - 1) % kSteps, t0 + u + kSteps - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kSteps - 1) : "memory");
      f(ring, u, t0 + u, here);
      here += stride;
    }
  }
}

// weight (default 1) or bias (default 0) of the V channels from c.
template <int V>
__device__ __forceinline__ void params(const void* p, int c, int dtype, float none, Pair<V> (&v)[kPairs<V>]) {
  float x[V];
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = p ? load_elem(p, c + j, dtype) : none;
  if constexpr (V == 1) v[0] = x[0];
  else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = make_float2(x[2 * i], x[2 * i + 1]);
  }
}

// How the slabs of L > 1 positions (or groups too wide for a warp) are cut.  A CTA takes `rows`
// positions of one n and one column block: up to 256 vectors of V channels, whole groups of DV
// vectors each, or, where a group alone is wider, a part of one.  A thread keeps its column and
// walks down the rows.
struct SlabPlan {
  int V, DV;          // channels a vector, vectors a group
  int GPB, parts;     // groups a column block; or column blocks a group
  int NCB;            // column blocks
  int rows, chunks;   // positions a CTA; CTAs down the positions
};

// The largest power of two that divides D, at most `most`.
inline int vector_width(int D, int most) {
  int v = 1;
  while (v < most && D % (2 * v) == 0) v *= 2;
  return v;
}

inline SlabPlan slab_plan(int N, int L, int C, int G, int io_dtype) {
  SlabPlan s;
  const int D = C / G;
  s.V = vector_width(D, io_dtype == GDN_BF16 ? 8 : 4);
  s.DV = D / s.V;
  if (s.DV <= kGnThreads) {
    s.GPB = kGnThreads / s.DV < G ? kGnThreads / s.DV : G;
    s.parts = 1;
    s.NCB = (G + s.GPB - 1) / s.GPB;
  } else {
    s.GPB = 1;
    s.parts = (s.DV + kGnThreads - 1) / kGnThreads;
    s.NCB = G * s.parts;
  }
  const int cols = s.parts == 1 ? s.GPB * s.DV : kGnThreads;
  const int step = kGnThreads / cols;               // rows that a CTA takes at a time
  // one wave, each thread at least four rows
  const long long want = std::max(1LL, (long long)current_sm_count() * kSlabPerSm / ((long long)N * s.NCB));
  const long long most = (L + 4LL * step - 1) / (4LL * step);
  const long long chunks = want < most ? want : most;
  s.rows = (int)((L + chunks - 1) / chunks);
  s.chunks = (L + s.rows - 1) / s.rows;
  return s;
}

// A thread's place in its CTA's slab.
struct SlabPlace {
  int n, cb, chunk;
  int g0, groups;      // the first group of the column block, and how many it holds
  int cols;            // vectors in the column block
  int col, row, step;  // this thread's vector and first row (from the chunk's), rows to the next
  int c;               // its first channel
  int g;               // its group
  bool on;
};
__device__ __forceinline__ SlabPlace slab_place(const SlabPlan& s, int C, int G) {
  SlabPlace p;
  int b = blockIdx.x;
  p.cb = b % s.NCB;
  b /= s.NCB;
  p.chunk = b % s.chunks;
  p.n = b / s.chunks;
  int first;   // the block's first vector
  if (s.parts == 1) {
    p.g0 = p.cb * s.GPB;
    p.groups = min(s.GPB, G - p.g0);
    p.cols = p.groups * s.DV;
    first = p.g0 * s.DV;
  } else {
    p.g0 = p.cb / s.parts;
    p.groups = 1;
    const int part = p.cb - p.g0 * s.parts;
    p.cols = min(kGnThreads, s.DV - part * kGnThreads);
    first = p.g0 * s.DV + part * kGnThreads;
  }
  p.step = kGnThreads / p.cols;
  p.col = threadIdx.x % p.cols;
  p.row = threadIdx.x / p.cols;
  p.on = p.row < p.step;
  p.c = (first + p.col) * s.V;
  p.g = s.parts == 1 ? p.g0 + p.col / s.DV : p.g0;
  return p;
}
// A thread's rows: its first element, elements from a row to its next, how many.
struct SlabRange {
  size_t from, stride;
  int rows;
};
__device__ __forceinline__ SlabRange slab_range(const SlabPlan& s, const SlabPlace& p, int L, int C) {
  const int r = p.chunk * s.rows + p.row, end = min(L, (p.chunk + 1) * s.rows);
  return SlabRange{((size_t)p.n * L + r) * C + p.c, (size_t)p.step * C, r < end ? (end - r + p.step - 1) / p.step : 0};
}

// Groups that up to 32 lanes hold in registers: lanes a group (a power of two), vectors a lane
// (the group's L DV vectors in order); 0 lanes where that does not serve.
struct RowPlan {
  int V, lanes, VPT;
  // A CTA's J lane groups take all G channel groups of `down` rows n at a time, or, where J < G, J
  // channel groups of one row; then the CTA's next rows.  What a CTA sums over its rows is a set.
  int J, across, down, sets;   // lane groups; CTAs across the groups; rows at a time; sets
};
// It serves groups of up to `most` values a lane, for one position, or for slabs so small that a
// CTA of the slab form would stand mostly idle on one.
inline RowPlan row_plan(int N, int L, int C, int G, int io_dtype, int most, int per_sm) {
  RowPlan r{vector_width(C / G, io_dtype == GDN_BF16 ? 8 : 4), 0, 1, 0, 0, 0, 0};
  if (L > 1 && (long long)L * C > 8192) return r;
  const long long vecs = (long long)L * (C / G / r.V);
  int lanes = 1;
  while (lanes < 32 && lanes < vecs) lanes *= 2;
  if ((vecs + lanes - 1) / lanes * r.V > most) return r;
  r.lanes = lanes;
  r.VPT = (int)((vecs + lanes - 1) / lanes);
  r.J = kGnThreads / lanes;
  r.across = r.J >= G ? 1 : (G + r.J - 1) / r.J;
  r.down = r.J >= G ? r.J / G : 1;
  // one wave of `per_sm` CTAs an SM, and no more than the rows need
  const long long need = ((long long)N + r.down - 1) / r.down, want = std::max(1, current_sm_count() * per_sm / r.across);
  r.sets = (int)std::min(need, want);
  return r;
}

// A thread's place in the row form.
struct RowPlace {
  int l, set, down, g;
  bool live;
};
__device__ __forceinline__ RowPlace row_place(const RowPlan& q, int G) {
  RowPlace p;
  const int j = threadIdx.x / q.lanes;
  p.l = threadIdx.x & (q.lanes - 1);
  p.set = blockIdx.x / q.across;
  p.g = q.across == 1 ? j % G : (blockIdx.x % q.across) * q.J + j;
  p.down = q.across == 1 ? j / G : 0;
  p.live = p.g < G && p.down < q.down;
  if (!p.live) p.g = 0;
  return p;
}
// Its rows n0, n0 + step, ...: how many, and how many turns its CTA takes (every lane of a warp runs
// the same number of them: the shuffles want them all).
struct RowRange {
  long long n0, step;
  int mine, turns;
};
__device__ __forceinline__ RowRange row_range(const RowPlan& q, const RowPlace& p, int N) {
  RowRange r;
  r.step = (long long)q.sets * q.down;
  r.n0 = (long long)p.set * q.down + p.down;
  r.turns = (int)((N + r.step - 1) / r.step);
  r.mine = r.n0 < N ? (int)((N - r.n0 + r.step - 1) / r.step) : 0;
  return r;
}
// Where this lane's vectors stand in a group (from its first element), their channels, and whether
// they are in it.
template <int V, int VPT>
struct RowVectors {
  int off[VPT], c[VPT];
  bool in[VPT];
  __device__ __forceinline__ RowVectors(const RowPlan& q, const RowPlace& p, int L, int C, int G) {
    const int D = C / G, DV = D / V;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = p.l + k * q.lanes, r = v / DV, e = (v - r * DV) * V;
      in[k] = p.live && r < L;
      off[k] = r * C + e;
      c[k] = p.g * D + e;
    }
  }
};

// Lets a kernel have kBytes of dynamic shared memory beside its static arrays of up to 8 KB (set
// once a device and kernel).
constexpr int kMaxDynamic = 232448 - 8 * 1024;
template <auto kKernel, int kBytes>
cudaError_t allow_shared() {
  static_assert(kBytes <= kMaxDynamic, "more shared memory than a CTA can have");
  if (kBytes <= 40 * 1024) return cudaSuccess;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed))) return err;
  err = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (err == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return err;
}

__device__ __forceinline__ float sub_sum(float x, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace
}  // namespace gdn
