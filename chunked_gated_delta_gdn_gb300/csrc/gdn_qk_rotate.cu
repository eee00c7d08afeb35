// gdn_qk_rotate.cu -- the norm of each head's queries and keys with the rotation of their positions.
//
//     n = x r w,  r = 1 / sqrt(mean(x^2) + eps) (or the sum, or 1);  y = n, its pairs turned by phi.
//     backward, with d the gradient turned back and xh = x r:
//     dw = sum over tokens and heads of d xh,   dx = r (d w - xh mean(d w xh)).
//
// Bound by bytes: one reading, one writing.  G lanes hold a head and walk the heads of a token (or a run of
// them, where tokens are few), whose sines and cosines they make once; the 32 / G groups of a warp have
// tokens of their own.  CTAs work on queries or on keys, in proportion, so that weights and their
// gradients stay in registers.  A lane's unit is two vectors of V values whose pairs are complete: of the two
// halves, or, interleaved, any two.  Lanes copy heads ahead into rings of their own in shared memory
// (asynchronous copies, no barrier).  bf16, heads of 128: forward of 4 x 32768 x (16 + 16) 320 us, 6.7 TB/s;
// 2 x 8192 x (32 + 8) 64 us forward, 91 us backward, 5.2 and 5.5 TB/s, of which launch, first loads and the weights'
// sums (7 us) are what is missing; three axes, 2 x 9731 x (12 + 12): 45 us, 5.3 TB/s.  fp32,
// 4 x 8192 x (16 + 16): 170 us forward, 269 backward, 6.3 and 6.0 TB/s.  Three CTAs an SM instead
// of two, or streaming stores, were slower.
//
// Angles: phi / 2 pi as a fraction of 2^64, position * floor(2^64 frac(inv_freq / 2 pi)) in integers that wrap,
// of which the upper 32 bits are kept: off by less than 2^-31 of a turn for every position and finite frequency.
// What is left is rounded to fp32 and less than half a turn: there the hardware's sine and cosine are off by
// 2^-21 of a unit at most, which is enough for bf16; fp32 takes the full functions.
#include "gdn_common.cuh"
#include "gdn_launch.cuh"
#include "gdn_qk_rotate.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSm = 2;
constexpr int kMaxParts = 1024;   // CTAs of a backward that sums weights' gradients
constexpr double kAngles = 1.5;   // the time of a token's angles, in heads

template <typename T, int V> struct alignas(V * sizeof(T)) Vec { T e[V]; };

template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& raw, float (&x)[V]) {
  if constexpr (sizeof(T) == 2 && V > 1) {
    const unsigned* const two = reinterpret_cast<const unsigned*>(&raw);
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      x[j] = __uint_as_float(two[j / 2] << 16);
      x[j + 1] = __uint_as_float(two[j / 2] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = (float)raw.e[j];
  }
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&x)[V]) {
  Vec<T, V> v;
  if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
    for (int j = 0; j < V; j += 2) reinterpret_cast<__nv_bfloat162*>(&v)[j / 2] = __floats2bfloat162_rn(x[j], x[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v.e[j] = (T)x[j];
  }
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// V values from global to shared memory, asynchronously.
template <typename T, int V>
__device__ __forceinline__ void copy_ahead(Vec<T, V>* dst, const T* src) {
  constexpr int kBytes = V * sizeof(T);
  static_assert(kBytes >= 4, "asynchronous copies have at least four bytes");
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src), "n"(kBytes)
                 : "memory");
}

// What a lane holds of a head: unit u's two vectors start at o1 and o2, so that neighbouring lanes' vectors
// are neighbours in memory.  (V = 1, interleaved: the two values of a pair.)
struct Unit {
  int o1, o2;
  bool on, second, turns;
};
template <int V>
__device__ __forceinline__ Unit unit_of(const QkRotateArgs& a, int u) {
  const int turning = a.R / (2 * V), behind = ((a.K - a.R) / V + 1) / 2;
  Unit r;
  r.turns = u < turning;
  if (r.turns) {
    const bool apart = V > 1 || !a.interleaved;
    r.o1 = apart ? u * V : 2 * u;
    r.o2 = apart ? r.o1 + a.R / 2 : r.o1 + 1;
    r.on = r.second = true;
  } else {
    r.o1 = a.R + (u - turning) * V;
    r.o2 = r.o1 + behind * V;
    r.on = u - turning < behind;
    r.second = r.on && r.o2 < a.K;
  }
  return r;
}
// The j-th of a unit's V pairs.
template <int V, bool kInVector>
__device__ __forceinline__ int pair_of(const Unit& u, int j) {
  return kInVector ? (j < V / 2 ? u.o1 / 2 + j : u.o2 / 2 + j - V / 2) : V == 1 && u.o2 == u.o1 + 1 ? u.o1 / 2 : u.o1 + j;
}

// frac(f / 2 pi) in units of 2^-64, to one of them, for every finite f = m 2^e: m (24 bits) times the 96 bits of
// 1 / 2 pi behind its first e ones, all that matters (after Payne and Hanek, "Radian reduction for trigonometric
// functions", 1983; the bits are those of Machin's formula for pi).
__constant__ unsigned kTurnsPerRadian[7] = {0x28be60dbu, 0x9391054au, 0x7f09d5f4u, 0x7d4d3770u,
                                            0x36d8a566u, 0x4f10e410u, 0x7f9458eau};
__device__ __forceinline__ unsigned long long turn_rate(float f) {
  const unsigned bits = __float_as_uint(f), exponent = bits >> 23 & 0xff;
  const unsigned long long m = (bits & 0x7fffff) | (exponent ? 0x800000 : 0);
  const int e = (int)max(exponent, 1u) - 150, word = e >> 5, shift = e & 31;
  unsigned w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = (unsigned)(word + k) < 7u ? kTurnsPerRadian[word + k] : 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) w[k] = __funnelshift_l(w[k + 1], w[k], shift);
  const unsigned long long rate = (m * w[0] << 32) + m * w[1] + (m * w[2] >> 32);
  return bits >> 31 ? 0 - rate : rate;
}

// The angle of a position, as sine and cosine.
template <bool kFast>
__device__ __forceinline__ void angle(unsigned long long rate, int position, float* s, float* c) {
  const unsigned p = (unsigned)position, lo = (unsigned)rate;
  unsigned turn = p * (unsigned)(rate >> 32) + __umulhi(p, lo);   // the product's upper half
  if (position < 0) turn -= lo;
  if (kFast) {
    const float phi = (float)(int)turn * 1.4629180792671596e-9f;   // 2 pi / 2^32
    *s = __sinf(phi);
    *c = __cosf(phi);
  } else {
    sincospif((float)(int)turn * 4.656612873077393e-10f, s, c);    // half turns
  }
}

__device__ __forceinline__ float group_sum(float x, int G) {
  for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One side's share of a launch: CTAs [first, first + ctas).  Tokens [from, to) in items of nh heads, `splits` of them
// a token; then the tokens that do not fill a turn of all groups, in smaller items.
struct Run {
  int from, to, splits, nh;
};
struct SidePlan {
  int first, ctas;
  Run run[2];
};
struct Plan {
  int G;
  SidePlan side[2];
};

template <typename T, int V, int NU, bool kBwd>
struct Ring {
  static constexpr int kDepth = 3;   // (deeper, DRAM does less: 4 x 32768 x 32 x 128 forward 328 us with 3, 375 with 4 or 6)
  static constexpr int kVecs = NU * 2 * (kBwd ? 2 : 1);
  Vec<T, V> slot[kWarps][kDepth][kVecs][32];
};

template <typename T, int V, int NU, bool kAdjacent, bool kBwd>
__global__ void __launch_bounds__(kThreads, kPerSm) qk_rotate_kernel(QkRotateArgs a, Plan plan, float* part) {
  constexpr bool kFast = sizeof(T) == 2;
  constexpr bool kInVector = kAdjacent && V > 1;   // a pair's two values stand in one vector
  using R = Ring<T, V, NU, kBwd>;
  extern __shared__ __align__(16) char shared_bytes[];
  R& ring = *reinterpret_cast<R*>(shared_bytes);
  __shared__ unsigned long long rates[GDN_MAX_ROTATE_DIM / 2];
  for (int j = threadIdx.x; j < a.R / 2; j += kThreads) rates[j] = turn_rate(a.inv_freq[j]);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sd = (int)blockIdx.x >= plan.side[1].first;
  const QkSide side = sd ? a.side[1] : a.side[0];
  const SidePlan sp = sd ? plan.side[1] : plan.side[0];
  const int G = plan.G, sub = lane & (G - 1), hs = lane / G, groups = 32 / G;
  Unit unit[NU];
  float w[NU][2][V];
#pragma unroll
  for (int m = 0; m < NU; ++m) {
    unit[m] = unit_of<V>(a, sub + G * m);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[m][0][j] = side.w && unit[m].on ? load_elem(side.w, unit[m].o1 + j, a.w_dtype) : 1.f;
      w[m][1][j] = side.w && unit[m].second ? load_elem(side.w, unit[m].o2 + j, a.w_dtype) : 1.f;
    }
  }
  for (int k = 0; k < R::kDepth * R::kVecs; ++k) {   // what no copy writes is zero
    const int v = k % R::kVecs % (2 * NU);
    bool on = false;
#pragma unroll
    for (int m = 0; m < NU; ++m) on |= v == 2 * m ? unit[m].on : v == 2 * m + 1 && unit[m].second;
    if (!on) ring.slot[warp][k / R::kVecs][k % R::kVecs][lane] = Vec<T, V>{};
  }
  const float mean = a.norm == GDN_NORM_RMS ? 1.f / (float)a.K : 1.f;
  const long long tokens = (long long)a.B * a.T, stride = (long long)sp.ctas * kWarps * groups;
  const long long base0 = ((long long)(blockIdx.x - sp.first) * kWarps + warp) * groups;
  float acc[NU][2][V];
#pragma unroll
  for (int m = 0; m < NU; ++m)
#pragma unroll
    for (int j = 0; j < V; ++j) acc[m][0][j] = acc[m][1][j] = 0.f;
  for (int which = 0; which < 2; ++which) {
    const Run run = which ? sp.run[1] : sp.run[0];
    const long long items = (long long)(run.to - run.from) * run.splits;
    const long long turns = base0 < items ? (items - base0 + stride - 1) / stride : 0;   // items of the warp's first group

    // the copies run kDepth - 1 heads ahead of the work
    long long ahead_item = base0 + hs;
    int ahead_h = 0, ahead_slot = 0;
    long long ahead_left = turns * run.nh;
    const T* ahead_x = nullptr;
    const T* ahead_dy = nullptr;
    auto copy_head = [&]() {
      if (ahead_left > 0) {
        if (ahead_h == 0) {
          const long long item = ahead_item < items ? ahead_item : items - 1;   // (a spare group reads the last one)
          const int part = run.splits == 1 ? 0 : (int)(item % run.splits), h0 = part * run.nh;
          const long long token = run.from + (run.splits == 1 ? item : item / run.splits);
          const int b = (int)token / a.T, t = (int)token - b * a.T;
          ahead_x = static_cast<const T*>(side.x) + b * side.sb + t * side.st + h0 * side.sh;
          if (kBwd) ahead_dy = static_cast<const T*>(side.dy) + (token * side.H + h0) * a.K;
        }
        Vec<T, V>(*const to)[32] = ring.slot[warp][ahead_slot];
        if constexpr (V * sizeof(T) >= 4) {
  #pragma unroll
          for (int m = 0; m < NU; ++m) {
            if (unit[m].on) copy_ahead<T, V>(&to[2 * m][lane], ahead_x + unit[m].o1);
            if (unit[m].second) copy_ahead<T, V>(&to[2 * m + 1][lane], ahead_x + unit[m].o2);
            if (kBwd) {
              if (unit[m].on) copy_ahead<T, V>(&to[2 * (NU + m)][lane], ahead_dy + unit[m].o1);
              if (unit[m].second) copy_ahead<T, V>(&to[2 * (NU + m) + 1][lane], ahead_dy + unit[m].o2);
            }
          }
        } else {   // two bytes: by loads, all of them before the first store
          T one[R::kVecs];
  #pragma unroll
          for (int v = 0; v < R::kVecs; ++v) {
            const Unit& u = unit[v % (2 * NU) / 2];
            const T* const from = v < 2 * NU ? ahead_x : ahead_dy;
            one[v] = (v & 1 ? u.second : u.on) ? from[v & 1 ? u.o2 : u.o1] : (T)0.f;
          }
  #pragma unroll
          for (int v = 0; v < R::kVecs; ++v) to[v][lane].e[0] = one[v];
        }
        ahead_x += side.sh;
        if (kBwd) ahead_dy += a.K;
        if (++ahead_h == run.nh) {
          ahead_h = 0;
          ahead_item += stride;
        }
        if (++ahead_slot == R::kDepth) ahead_slot = 0;
        --ahead_left;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int k = 0; k < R::kDepth - 1; ++k) copy_head();

    // the positions of an item's token on every axis, read an item ahead
    int at[GDN_MAX_AXES] = {0, 0, 0, 0};
    auto positions_of = [&](long long item) {
      if (item >= items) return;
      const long long token = run.from + (run.splits == 1 ? item : item / run.splits);
      if (!a.positions) {
  #pragma unroll
        for (int i = 0; i < GDN_MAX_AXES; ++i) at[i] = (int)token % a.T;
      } else {
  #pragma unroll
        for (int i = 0; i < GDN_MAX_AXES; ++i)
          if (i < a.num_axes) at[i] = a.positions[i * tokens + token];
      }
    };
    positions_of(base0 + hs);
    int slot = 0;
    for (long long n = 0; n < turns; ++n) {
      const long long item = base0 + hs + n * stride;
      const bool here = item < items;
      const long long token = here ? run.from + (run.splits == 1 ? item : item / run.splits) : 0;
      const int h0 = here && run.splits > 1 ? (int)(item % run.splits) * run.nh : 0;
      float c[NU][V], s[NU][V];
  #pragma unroll
      for (int m = 0; m < NU; ++m)
  #pragma unroll
        for (int j = 0; j < V; ++j) {
          c[m][j] = 1.f;
          s[m][j] = 0.f;
          if (unit[m].turns) {
            const int pair = pair_of<V, kInVector>(unit[m], j);
            int position = at[0];
  #pragma unroll
            for (int i = 1; i < GDN_MAX_AXES; ++i) position = pair >= a.axis_end[i - 1] ? at[i] : position;
            angle<kFast>(rates[pair], position, &s[m][j], &c[m][j]);
          }
        }
      // forward: the turn's factors with the weights in them, y1 = r (x1 f1 - x2 f2), y2 = r (x2 f3 + x1 f4)
      float f[kBwd ? 1 : NU][4][V];
      if constexpr (!kBwd) {
  #pragma unroll
        for (int m = 0; m < NU; ++m)
  #pragma unroll
          for (int j = 0; j < V; ++j) {
            const float w1 = kInVector ? w[m][2 * j / V][2 * j % V] : w[m][0][j];
            const float w2 = kInVector ? w[m][2 * j / V][2 * j % V + 1] : w[m][1][j];
            f[m][0][j] = w1 * c[m][j];
            f[m][1][j] = w2 * s[m][j];
            f[m][2][j] = w2 * c[m][j];
            f[m][3][j] = w1 * s[m][j];
          }
      }
      positions_of(item + stride);
      T* out = static_cast<T*>(side.out) + (token * side.H + h0) * a.K;
      for (int h = 0; h < run.nh; ++h, out += a.K) {
        copy_head();
        asm volatile("cp.async.wait_group %0;" ::"n"(R::kDepth - 1) : "memory");
        float x[NU][2][V], ss = 0.f;
  #pragma unroll
        for (int m = 0; m < NU; ++m)
  #pragma unroll
          for (int v = 0; v < 2; ++v) {
            unpack<T, V>(ring.slot[warp][slot][2 * m + v][lane], x[m][v]);
  #pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(x[m][v][j], x[m][v][j], ss);
          }
        const float inv = a.norm == GDN_NORM_NONE ? 1.f : rsqrtf(fmaf(group_sum(ss, G), mean, a.eps));
        if constexpr (!kBwd) {
  #pragma unroll
          for (int m = 0; m < NU; ++m) {
            float y[2][V];
  #pragma unroll
            for (int j = 0; j < V; ++j) {   // pair j (behind the rotated part: an angle of 0)
              const int v1 = kInVector ? 2 * j / V : 0, v2 = kInVector ? v1 : 1, j1 = kInVector ? 2 * j % V : j,
                        j2 = kInVector ? j1 + 1 : j;
              y[v1][j1] = inv * fmaf(x[m][v1][j1], f[m][0][j], -x[m][v2][j2] * f[m][1][j]);
              y[v2][j2] = inv * fmaf(x[m][v2][j2], f[m][2][j], x[m][v1][j1] * f[m][3][j]);
            }
            if (here && unit[m].on) store<T, V>(out + unit[m].o1, y[0]);
            if (here && unit[m].second) store<T, V>(out + unit[m].o2, y[1]);
          }
        } else {
          // with d r in d's place: dw += d x,  dx = d w - x r^2 mean(d w x)
          float d[NU][2][V], dot = 0.f;
  #pragma unroll
          for (int m = 0; m < NU; ++m) {
            float r[2][V];
  #pragma unroll
            for (int v = 0; v < 2; ++v) {
              unpack<T, V>(ring.slot[warp][slot][2 * (NU + m) + v][lane], r[v]);
  #pragma unroll
              for (int j = 0; j < V; ++j) r[v][j] *= inv;
            }
  #pragma unroll
            for (int j = 0; j < V; ++j) {
              const int v1 = kInVector ? 2 * j / V : 0, v2 = kInVector ? v1 : 1, j1 = kInVector ? 2 * j % V : j,
                        j2 = kInVector ? j1 + 1 : j;
              d[m][v1][j1] = fmaf(r[v1][j1], c[m][j], r[v2][j2] * s[m][j]);
              d[m][v2][j2] = fmaf(r[v2][j2], c[m][j], -r[v1][j1] * s[m][j]);
            }
  #pragma unroll
            for (int v = 0; v < 2; ++v)
  #pragma unroll
              for (int j = 0; j < V; ++j) {
                if (here) acc[m][v][j] = fmaf(d[m][v][j], x[m][v][j], acc[m][v][j]);
                d[m][v][j] *= w[m][v][j];
                dot = fmaf(d[m][v][j], x[m][v][j], dot);
              }
          }
          const float k = a.norm == GDN_NORM_NONE ? 0.f : group_sum(dot, G) * mean * inv * inv;
  #pragma unroll
          for (int m = 0; m < NU; ++m) {
            if (a.norm != GDN_NORM_NONE) {
  #pragma unroll
              for (int v = 0; v < 2; ++v)
  #pragma unroll
                for (int j = 0; j < V; ++j) d[m][v][j] = fmaf(-x[m][v][j], k, d[m][v][j]);
            }
            if (here && unit[m].on) store<T, V>(out + unit[m].o1, d[m][0]);
            if (here && unit[m].second) store<T, V>(out + unit[m].o2, d[m][1]);
          }
        }
        if (++slot == R::kDepth) slot = 0;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if (!kBwd || !part) return;
  // this CTA's sums: over the groups of a warp, then over the warps in order
  __syncthreads();
  float(*const total)[GDN_MAX_ROTATE_DIM] = reinterpret_cast<float(*)[GDN_MAX_ROTATE_DIM]>(shared_bytes);
  static_assert(sizeof(R) >= kWarps * GDN_MAX_ROTATE_DIM * sizeof(float) || !kBwd, "the ring holds the sums");
#pragma unroll
  for (int m = 0; m < NU; ++m)
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float x = acc[m][v][j];
        for (int o = 16; o >= G; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (hs == 0 && (v ? unit[m].second : unit[m].on)) total[warp][(v ? unit[m].o2 : unit[m].o1) + j] = x;
      }
  __syncthreads();
  for (int d = threadIdx.x; d < a.K; d += kThreads) {
    float x = 0.f;
    for (int k = 0; k < kWarps; ++k) x += total[k][d];
    part[(size_t)blockIdx.x * a.K + d] = x;
  }
}

// The weights' gradients: CTAs' parts, 32 runs of them side by side, added in order.
__global__ void __launch_bounds__(1024) qk_rotate_dw_kernel(QkRotateArgs a, Plan plan, const float* part) {
  __shared__ float run[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, d = blockIdx.x * 32 + lane, sd = blockIdx.y;
  const SidePlan& sp = plan.side[sd];
  next_may_start();
  wait_for_previous();
  float x = 0.f;
  if (d < a.K)
    for (int p = sp.ctas * w / 32; p < sp.ctas * (w + 1) / 32; ++p) x += part[(size_t)(sp.first + p) * a.K + d];
  run[w][lane] = x;
  __syncthreads();
  if (w > 0 || d >= a.K || !a.side[sd].dw) return;
  x = 0.f;
  for (int k = 0; k < 32; ++k) x += run[k][lane];
  a.side[sd].dw[d] = x;
}

// The widest vectors that every row and pair allows.
int vector_width(const QkRotateArgs& a, bool bwd) {
  const int eb = a.io_dtype == GDN_BF16 ? 2 : 4;
  for (int v = 16 / eb; v > 1; v >>= 1) {
    bool fits = a.K % v == 0 && a.R % (2 * v) == 0;
    for (const QkSide& s : a.side) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(s.x) | reinterpret_cast<uintptr_t>(s.out) |
                           (bwd ? reinterpret_cast<uintptr_t>(s.dy) : 0);
      fits = fits && at % (v * eb) == 0 && (a.B == 1 || s.sb % v == 0) && (a.T == 1 || s.st % v == 0) &&
             (s.H == 1 || s.sh % v == 0);
    }
    if (fits) return v;
  }
  return 1;
}

// CTAs for queries and keys in proportion to their heads (a token's angles count as kAngles more); a token's
// heads are shared out as far as the longest run of a group of lanes gets shorter by it (19462 tokens of
// 12 heads: 65 us with a fifth turn for 6 of them, see run[1]).
Plan plan_of(const QkRotateArgs& a, int v) {
  Plan p;
  const int units = a.R / (2 * v) + (a.K - a.R + 2 * v - 1) / (2 * v);
  p.G = 1;
  while (p.G < units && p.G < 32) p.G *= 2;
  const int sms = current_sm_count();
  const long long tokens = (long long)a.B * a.T, per_cta = (long long)kWarps * (32 / p.G);
  int ctas = (sms > 0 ? sms : 1) * kPerSm;
  if (ctas > kMaxParts) ctas = kMaxParts;
  const double q = a.side[0].H + kAngles, k = a.side[1].H + kAngles;
  int share[2];
  share[0] = (int)(ctas * q / (q + k) + 0.5);
  share[0] = share[0] < 1 ? 1 : share[0] > ctas - 1 ? ctas - 1 : share[0];
  if (share[0] < 1) share[0] = 1;
  share[1] = ctas - share[0] < 1 ? 1 : ctas - share[0];
  for (int i = 0; i < 2; ++i) {
    const int H = a.side[i].H;
    SidePlan& s = p.side[i];
    // tokens in full turns of n items each, and those behind them in items of their own
    const long long groups = per_cta * share[i];
    int divisors[64], count = 0;
    for (int n = 1; n <= H / n && count < 63; ++n)
      if (H % n == 0) {
        divisors[count++] = n;
        if (n != H / n) divisors[count++] = H / n;
      }
    auto turn = [&](int n) { return H / n + kAngles; };
    auto turns = [&](long long items) { return (double)((items + groups - 1) / groups); };
    auto rest = [&](long long left, int* best) {
      double least = left ? 1e300 : 0.;
      *best = 1;
      for (int d = 0; d < count && left; ++d) {
        const int n = divisors[d];
        const double time = turns(left * n) * turn(n);
        if (time < 0.99 * least) {
          least = time;
          *best = n;
        }
      }
      return least;
    };
    double least = 1e300;
    for (int d = 0; d < count; ++d) {
      const int n = divisors[d];
      const long long full = tokens * n / groups * groups / n;
      int n2;
      const double time = turns(full * n) * turn(n) + rest(tokens - full, &n2);
      if (time < 0.99 * least) {
        least = time;
        s.run[0] = Run{0, (int)full, n, H / n};
        s.run[1] = Run{(int)full, (int)tokens, n2, H / n2};
      }
    }
    long long need = 0;
    for (const Run& r : s.run) {
      const long long ctas_of = ((long long)(r.to - r.from) * r.splits + per_cta - 1) / per_cta;
      need = ctas_of > need ? ctas_of : need;
    }
    s.ctas = (int)(need < share[i] ? need : share[i]);
  }
  p.side[0].first = 0;
  p.side[1].first = p.side[0].ctas;
  return p;
}

template <typename T, int V, int NU, bool kAdjacent, bool kBwd>
cudaError_t launch(const QkRotateArgs& a, const Plan& p, float* part) {
  constexpr auto kernel = qk_rotate_kernel<T, V, NU, kAdjacent, kBwd>;
  const size_t shared = sizeof(Ring<T, V, NU, kBwd>);
  const cudaError_t err = allow_shared<kernel>(shared);
  if (err != cudaSuccess) return err;
  kernel<<<p.side[0].ctas + p.side[1].ctas, kThreads, shared, a.stream>>>(a, p, part);
  return cudaGetLastError();
}

template <typename T, int V, int NU, bool kBwd>
cudaError_t launch(const QkRotateArgs& a, const Plan& p, float* part) {
  return a.interleaved ? launch<T, V, NU, true, kBwd>(a, p, part) : launch<T, V, NU, false, kBwd>(a, p, part);
}

template <typename T, bool kBwd>
cudaError_t launch(const QkRotateArgs& a) {
  const int v = vector_width(a, kBwd);
  const Plan p = plan_of(a, v);
  float* const part = kBwd && (a.side[0].dw || a.side[1].dw) ? static_cast<float*>(a.workspace) : nullptr;
  cudaError_t err;
  if (v == 8 && sizeof(T) == 2) err = launch<T, sizeof(T) == 2 ? 8 : 4, 1, kBwd>(a, p, part);
  else if (v == 4) err = launch<T, 4, 1, kBwd>(a, p, part);
  else if (v == 2) err = launch<T, 2, 2, kBwd>(a, p, part);
  else err = launch<T, 1, 4, kBwd>(a, p, part);
  if (err != cudaSuccess || !part) return err;
  return launch_behind(qk_rotate_dw_kernel, dim3((a.K + 31) / 32, 2), 1024, 0, a.stream, a, p, (const float*)part);
}

}  // namespace

size_t qk_rotate_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int K, bool need_weights) {
  if (!need_weights || (long long)B * T == 0) return 0;
  return (size_t)kMaxParts * K * sizeof(float);
}

cudaError_t launch_qk_rotate_fwd(const QkRotateArgs& a) {
  return a.io_dtype == GDN_BF16 ? launch<__nv_bfloat16, false>(a) : launch<float, false>(a);
}
cudaError_t launch_qk_rotate_bwd(const QkRotateArgs& a) {
  return a.io_dtype == GDN_BF16 ? launch<__nv_bfloat16, true>(a) : launch<float, true>(a);
}

}  // namespace gdn
