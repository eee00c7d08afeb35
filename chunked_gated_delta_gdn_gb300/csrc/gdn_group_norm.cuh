// gdn_group_norm.cuh -- what the forward and backward kernels of group norm share.
#pragma once

#include <stdint.h>

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
  // about four CTAs an SM, each thread at least four rows
  const long long want = 152LL * 4 / ((long long)N * s.NCB) + 1;
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

// Groups that a warp (or part of one) holds in registers, for L = 1: lanes a group (a power of
// two), vectors a lane; 0 lanes where the group is too wide.
struct RowPlan {
  int V, lanes, VPT;
};
inline RowPlan row_plan(int C, int G, int io_dtype, int most_values) {
  RowPlan r{vector_width(C / G, io_dtype == GDN_BF16 ? 8 : 4), 0, 1};
  const int DV = C / G / r.V;
  int lanes = 1;
  while (lanes < 32 && lanes < DV) lanes *= 2;
  const int vpt = (DV + lanes - 1) / lanes;
  if (vpt * r.V <= most_values) {
    r.lanes = lanes;
    r.VPT = vpt;
  }
  return r;
}

__device__ __forceinline__ float sub_sum(float x, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

}  // namespace
}  // namespace gdn
