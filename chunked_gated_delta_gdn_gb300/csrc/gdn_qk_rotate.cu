// gdn_qk_rotate.cu -- the norm of each head's queries and keys with the rotation of their positions.
//
//     n = x r w,  r = 1 / sqrt(mean(x^2) + eps) (or the sum, or 1);  y = n, its pairs turned by phi.
//     backward, with d the gradient turned back and xh = x r:
//     dw = sum over tokens and heads of d xh,   dx = r (d w - xh mean(d w xh)).
//
// A token's heads share its angles, so a warp takes a token (or a part of its heads, where tokens are
// few), makes the sines and cosines of its own pairs once and walks the heads.  G lanes hold a head,
// 32 / G heads pass at a time.  A lane's unit is two vectors of V values whose pairs are complete: of
// the two halves, or, interleaved, two in a row; behind the rotated part two in a row.
//
// Angles: phi / 2 pi as a fraction of 2^64, position * round(2^64 frac(inv_freq / 2 pi)) in integers
// that wrap, is exact to 2^-11 of fp32's rounding for every position.
#include "gdn_common.cuh"
#include "gdn_launch.cuh"
#include "gdn_qk_rotate.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 1024;   // CTAs of a backward that sums weights' gradients

template <typename T, int V> struct alignas(V * sizeof(T)) Vec { T e[V]; };

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float (&x)[V]) {
  const Vec<T, V> v = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = (float)v.e[j];
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&x)[V]) {
  Vec<T, V> v;
#pragma unroll
  for (int j = 0; j < V; ++j) v.e[j] = (T)x[j];
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// What a lane holds of a head: unit u's two vectors start at o1 and o2.
struct Unit {
  int o1, o2;
  bool on, second, turns;
  int pair;
};
template <int V>
__device__ __forceinline__ Unit unit_of(const QkRotateArgs& a, int u) {
  const int turning = a.R / (2 * V);
  Unit r;
  r.turns = u < turning;
  if (r.turns) {
    r.o1 = a.interleaved ? 2 * u * V : u * V;
    r.o2 = a.interleaved ? r.o1 + V : r.o1 + a.R / 2;
  } else {
    r.o1 = a.R + 2 * (u - turning) * V;
    r.o2 = r.o1 + V;
  }
  r.pair = u * V;
  r.on = r.o1 < a.K;
  r.second = r.on && r.o2 < a.K;
  return r;
}

// frac(f / 2 pi) in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_rate(float f) {
  const double t = (double)f * 0.15915494309189533577;
  return (unsigned long long)((t - floor(t)) * 18446744073709551616.0);
}

// The angle of a position on pair j, as sine and cosine.
__device__ __forceinline__ void angle(unsigned long long rate, int position, float* s, float* c) {
  const unsigned long long turn = rate * (unsigned long long)(long long)position;
  sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, s, c);   // 2^-31: half turns
}

// Turns the pairs of a unit (back: by the negative angle).
template <int V>
__device__ __forceinline__ void rotate(float (&x)[V], float (&y)[V], const float (&c)[V], const float (&s)[V],
                                       bool adjacent, float sign) {
  if (V > 1 && adjacent) {
#pragma unroll
    for (int j = 0; j + 1 < V; j += 2) {
      const float s1 = sign * s[j / 2], s2 = sign * s[V / 2 + j / 2];
      const float u = x[j], v = x[j + 1];
      x[j] = u * c[j / 2] - v * s1;
      x[j + 1] = v * c[j / 2] + u * s1;
      const float p = y[j], q = y[j + 1];
      y[j] = p * c[V / 2 + j / 2] - q * s2;
      y[j + 1] = q * c[V / 2 + j / 2] + p * s2;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float u = x[j], v = y[j], w = sign * s[j];
      x[j] = u * c[j] - v * w;
      y[j] = v * c[j] + u * w;
    }
  }
}

__device__ __forceinline__ float group_sum(float x, int G) {
  for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T, int V, int NU, bool kBwd>
__global__ void __launch_bounds__(kThreads) qk_rotate_kernel(QkRotateArgs a, int G, int splits, float* part) {
  __shared__ float total[kBwd ? kWarps * 2 * GDN_MAX_ROTATE_DIM : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (G - 1), hs = lane / G, heads = 32 / G;
  Unit unit[NU];
  unsigned long long rate[NU][V];
#pragma unroll
  for (int m = 0; m < NU; ++m) {
    unit[m] = unit_of<V>(a, sub + G * m);
#pragma unroll
    for (int j = 0; j < V; ++j) rate[m][j] = unit[m].turns ? turn_rate(a.inv_freq[unit[m].pair + j]) : 0;
  }
  const int passes[2] = {(a.side[0].H + heads - 1) / heads, (a.side[1].H + heads - 1) / heads};
  const int all = passes[0] + passes[1];
  const float mean = a.norm == GDN_NORM_RMS ? 1.f / (float)a.K : 1.f;
  float acc[2][NU][2][V];
  if (kBwd) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < NU; ++m)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[s][m][0][j] = acc[s][m][1][j] = 0.f;
  }
  const long long tokens = (long long)a.B * a.T, items = tokens * splits;
  for (long long item = (long long)blockIdx.x * kWarps + warp; item < items; item += (long long)gridDim.x * kWarps) {
    const int token = (int)(item / splits), split = (int)(item - (long long)token * splits);
    const int b = token / a.T, t = token - b * a.T;
    float c[NU][V], s[NU][V];
#pragma unroll
    for (int m = 0; m < NU; ++m)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        c[m][j] = 1.f;
        s[m][j] = 0.f;
        if (unit[m].turns) {
          const int pair = unit[m].pair + j;
          const int axis = (pair >= a.axis_end[0]) + (pair >= a.axis_end[1]) + (pair >= a.axis_end[2]);
          angle(rate[m][j], a.positions ? a.positions[axis * tokens + token] : t, &s[m][j], &c[m][j]);
        }
      }
    const int p0 = (int)((long long)all * split / splits), p1 = (int)((long long)all * (split + 1) / splits);
#pragma unroll
    for (int sd = 0; sd < 2; ++sd) {
      const QkSide& side = a.side[sd];
      const int from = sd ? max(p0 - passes[0], 0) : p0, to = sd ? p1 - passes[0] : min(p1, passes[0]);
      if (from >= to) continue;
      float w[NU][2][V];
#pragma unroll
      for (int m = 0; m < NU; ++m)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          w[m][0][j] = side.w && unit[m].on ? load_elem(side.w, unit[m].o1 + j, a.w_dtype) : 1.f;
          w[m][1][j] = side.w && unit[m].second ? load_elem(side.w, unit[m].o2 + j, a.w_dtype) : 1.f;
        }
      const T* const x0 = static_cast<const T*>(side.x) + b * side.sb + t * side.st;
      for (int p = from; p < to; ++p) {
        const int h = p * heads + hs;
        const bool here = h < side.H;
        const T* const xh = x0 + h * side.sh;
        const size_t at = ((size_t)token * side.H + h) * a.K;
        float x[NU][2][V], d[NU][2][V], ss = 0.f;
#pragma unroll
        for (int m = 0; m < NU; ++m) {
#pragma unroll
          for (int j = 0; j < V; ++j) x[m][0][j] = x[m][1][j] = d[m][0][j] = d[m][1][j] = 0.f;
          if (here && unit[m].on) load<T, V>(xh + unit[m].o1, x[m][0]);
          if (here && unit[m].second) load<T, V>(xh + unit[m].o2, x[m][1]);
          if (kBwd) {
            const T* const dy = static_cast<const T*>(side.dy) + at;
            if (here && unit[m].on) load<T, V>(dy + unit[m].o1, d[m][0]);
            if (here && unit[m].second) load<T, V>(dy + unit[m].o2, d[m][1]);
          }
#pragma unroll
          for (int j = 0; j < V; ++j) ss += x[m][0][j] * x[m][0][j] + x[m][1][j] * x[m][1][j];
        }
        const float inv = a.norm == GDN_NORM_NONE ? 1.f : 1.f / sqrtf(group_sum(ss, G) * mean + a.eps);
        T* const out = static_cast<T*>(side.out) + at;
        if (!kBwd) {
#pragma unroll
          for (int m = 0; m < NU; ++m) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              x[m][0][j] *= inv * w[m][0][j];
              x[m][1][j] *= inv * w[m][1][j];
            }
            if (unit[m].turns) rotate<V>(x[m][0], x[m][1], c[m], s[m], a.interleaved, 1.f);
            if (here && unit[m].on) store<T, V>(out + unit[m].o1, x[m][0]);
            if (here && unit[m].second) store<T, V>(out + unit[m].o2, x[m][1]);
          }
        } else {
          float dot = 0.f;
#pragma unroll
          for (int m = 0; m < NU; ++m) {
            if (unit[m].turns) rotate<V>(d[m][0], d[m][1], c[m], s[m], a.interleaved, -1.f);
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
              for (int j = 0; j < V; ++j) {
                x[m][v][j] *= inv;
                acc[sd][m][v][j] += d[m][v][j] * x[m][v][j];
                d[m][v][j] *= w[m][v][j];
                dot += d[m][v][j] * x[m][v][j];
              }
          }
          dot = a.norm == GDN_NORM_NONE ? 0.f : group_sum(dot, G) * mean;
#pragma unroll
          for (int m = 0; m < NU; ++m) {
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
              for (int j = 0; j < V; ++j) d[m][v][j] = inv * (d[m][v][j] - x[m][v][j] * dot);
            if (here && unit[m].on) store<T, V>(out + unit[m].o1, d[m][0]);
            if (here && unit[m].second) store<T, V>(out + unit[m].o2, d[m][1]);
          }
        }
      }
    }
  }
  if (!kBwd || !part) return;
  // this CTA's sums: over the heads side by side in a warp, then over the warps in order
#pragma unroll
  for (int sd = 0; sd < 2; ++sd)
#pragma unroll
    for (int m = 0; m < NU; ++m)
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float x = acc[sd][m][v][j];
          for (int o = 16; o >= G; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (hs == 0 && (v ? unit[m].second : unit[m].on))
            total[(warp * 2 + sd) * GDN_MAX_ROTATE_DIM + (v ? unit[m].o2 : unit[m].o1) + j] = x;
        }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * a.K; e += kThreads) {
    const int sd = e >= a.K, d = e - sd * a.K;
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += total[(w * 2 + sd) * GDN_MAX_ROTATE_DIM + d];
    part[(size_t)blockIdx.x * 2 * a.K + e] = x;
  }
}

// The weights' gradients: CTAs' parts, eight runs of them side by side, added in order.
__global__ void __launch_bounds__(kThreads) qk_rotate_dw_kernel(QkRotateArgs a, const float* part, int parts) {
  __shared__ float run[kWarps][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float x = 0.f;
  if (e < 2 * a.K) {
    const int from = (int)((long long)parts * w / kWarps), to = (int)((long long)parts * (w + 1) / kWarps);
    for (int p = from; p < to; ++p) x += part[(size_t)p * 2 * a.K + e];
  }
  run[w][threadIdx.x & 31] = x;
  __syncthreads();
  if (w > 0 || e >= 2 * a.K) return;
  x = 0.f;
  for (int i = 0; i < kWarps; ++i) x += run[i][threadIdx.x];
  float* const dw = a.side[e >= a.K].dw;
  if (dw) dw[e >= a.K ? e - a.K : e] = x;
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

struct Plan {
  int G, splits;
  unsigned ctas;
};

Plan plan_of(const QkRotateArgs& a, int v) {
  Plan p;
  const int units = a.R / (2 * v) + (a.K - a.R + 2 * v - 1) / (2 * v);
  p.G = 1;
  while (p.G < units && p.G < 32) p.G *= 2;
  const int heads = 32 / p.G;
  const int all = (a.side[0].H + heads - 1) / heads + (a.side[1].H + heads - 1) / heads;
  const long long tokens = (long long)a.B * a.T;
  const int sms = current_sm_count();
  // a token's heads are shared out where tokens do not fill the SMs' warps
  const long long want = (long long)(sms > 0 ? sms : 1) * 16;
  p.splits = tokens >= want ? 1 : (int)((want + tokens - 1) / tokens);
  if (p.splits > all) p.splits = all;
  const long long ctas = (tokens * p.splits + kWarps - 1) / kWarps;
  const long long most = (sms > 0 ? sms : 1) * 4 < kMaxParts ? (sms > 0 ? sms : 1) * 4 : kMaxParts;
  p.ctas = (unsigned)(ctas < most ? ctas : most);
  return p;
}

template <typename T, bool kBwd>
cudaError_t launch(const QkRotateArgs& a) {
  const int v = vector_width(a, kBwd);
  const Plan p = plan_of(a, v);
  float* const part = kBwd && (a.side[0].dw || a.side[1].dw) ? static_cast<float*>(a.workspace) : nullptr;
  switch (v) {
    case 8:
      if constexpr (sizeof(T) == 2)
        qk_rotate_kernel<T, 8, 1, kBwd><<<p.ctas, kThreads, 0, a.stream>>>(a, p.G, p.splits, part);
      break;
    case 4: qk_rotate_kernel<T, 4, 1, kBwd><<<p.ctas, kThreads, 0, a.stream>>>(a, p.G, p.splits, part); break;
    case 2: qk_rotate_kernel<T, 2, 2, kBwd><<<p.ctas, kThreads, 0, a.stream>>>(a, p.G, p.splits, part); break;
    default: qk_rotate_kernel<T, 1, 4, kBwd><<<p.ctas, kThreads, 0, a.stream>>>(a, p.G, p.splits, part);
  }
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !part) return err;
  qk_rotate_dw_kernel<<<(2 * a.K + 31) / 32, kThreads, 0, a.stream>>>(a, part, (int)p.ctas);
  return cudaGetLastError();
}

}  // namespace

size_t qk_rotate_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int K, bool need_weights) {
  if (!need_weights || (long long)B * T == 0) return 0;
  return (size_t)kMaxParts * 2 * K * sizeof(float);
}

cudaError_t launch_qk_rotate_fwd(const QkRotateArgs& a) {
  return a.io_dtype == GDN_BF16 ? launch<__nv_bfloat16, false>(a) : launch<float, false>(a);
}
cudaError_t launch_qk_rotate_bwd(const QkRotateArgs& a) {
  return a.io_dtype == GDN_BF16 ? launch<__nv_bfloat16, true>(a) : launch<float, true>(a);
}

}  // namespace gdn
