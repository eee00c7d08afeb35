// gdn_group_norm.cuh -- what the forward and backward kernels of group norm share.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_group_norm.h"

namespace gdn {
namespace {

constexpr int kGnThreads = 256;

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
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

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
// steps deep, of which kSteps - 1 are on their way while one is used.  2-byte packs, which such
// copies do not move, are copied at once.
template <typename T, int V, int kPacks, int kSteps>
struct Ring {
  static constexpr int kBytes = V * (int)sizeof(T);
  static constexpr int kShared = kSteps * kPacks * kBytes * kGnThreads;
  uint8_t* mine;
  int at = 0;   // the step that `get` reads and the next `put` ends up behind
  __device__ __forceinline__ explicit Ring(void* smem) : mine(reinterpret_cast<uint8_t*>(smem) + threadIdx.x * kBytes) {}
  __device__ __forceinline__ uint8_t* slot(int step, int i) const {
    return mine + (step * kPacks + i) * kBytes * kGnThreads;
  }
  // Pack i of a step that is `ahead` steps behind the one read now.
  __device__ __forceinline__ void put(int ahead, int i, const void* base, size_t elem) {
    int st = at + ahead;
    if (st >= kSteps) st -= kSteps;
    const T* src = reinterpret_cast<const T*>(base) + elem;
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot(st, i));
    if (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (kBytes >= 4) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes < 4 ? 4 : kBytes) : "memory");
    else *reinterpret_cast<Pack<T, V>*>(slot(st, i)) = load_pack<T, V>(base, elem);
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Waits for the step to be read (all but the kSteps - 1 newest groups).
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kSteps - 1) : "memory"); }
  __device__ __forceinline__ Pack<T, V> get(int i) const {
    Pack<T, V> p;
    using R = typename Raw<kBytes>::type;
    *reinterpret_cast<R*>(&p) = *reinterpret_cast<const R*>(slot(at, i));
    return p;
  }
  __device__ __forceinline__ void next() { at = at + 1 == kSteps ? 0 : at + 1; }
};

// weight (default 1) or bias (default 0) of channel c.
__device__ __forceinline__ float param(const void* p, int c, int dtype, float none) {
  return p ? load_elem(p, c, dtype) : none;
}

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float act_value(float x, int act) {
  return act == GDN_ACT_SILU ? x * sigmoid_fast(x) : x;
}
// Value and slope.
__device__ __forceinline__ float2 act_both(float x, int act) {
  if (act != GDN_ACT_SILU) return make_float2(x, 1.f);
  const float s = sigmoid_fast(x);
  return make_float2(x * s, s * (1.f + x * (1.f - s)));
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
  // one wave of five CTAs an SM, each thread at least four rows
  const long long want = std::max(1LL, 152LL * 5 / ((long long)N * s.NCB));
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
// Positions [r0, r1) of a chunk.
__device__ __forceinline__ int2 slab_rows(const SlabPlan& s, const SlabPlace& p, int L) {
  return make_int2(p.chunk * s.rows, min(L, (p.chunk + 1) * s.rows));
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
  const long long need = ((long long)N + r.down - 1) / r.down, want = std::max(1, 152 * per_sm / r.across);
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
template <auto kKernel, int kBytes>
cudaError_t allow_shared() {
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
  for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace
}  // namespace gdn
