// gdn_recurrence.cuh -- what the kernels of the gated linear recurrence share: the gates, packed
// lengths, a warp's window of tokens and its copies, what CTAs of a cluster tell one another.
//
// The tokens of all sequences stand on one axis.  A CTA holds W = 32 kCh channels (a lane kCh of them)
// and walks tiles of it; a warp has kTau successive tokens of a tile.  What a window does to a state is
// h -> A h + H, A = exp(L): windows are joined by that, and sequences' starts by "reset", which
// takes H alone (a NaN in front of it stays there).  L is a sum of logarithms: A is rounded once for
// all the tokens that it stands for, not once a token, and an error that always has the same sign
// does not add up over a long memory.
#pragma once

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_launch.cuh"
#include "gdn_recurrence.h"

namespace gdn {
namespace {

constexpr int kTau = 16;   // tokens of a warp's window

// ---------------------------------------------------------------- gates

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Logarithms of decays are to base 2 where the outputs are bf16 (the hardware's exponential, off by
// 2^-22, is enough for them), natural ones with the full functions for fp32.
template <bool kFast> __device__ __forceinline__ float decay_of(float l) { return kFast ? ex2_approx(l) : expf(l); }
template <bool kFast> __device__ __forceinline__ float gate_sigmoid(float x) {
  return kFast ? rcp_approx(1.f + ex2_approx(x * -kLog2e)) : sigmoid_f(x);
}

// 1 - a^2 of a = decay_of(l): a short series where a is near 1 and the difference would lose its digits.
template <bool kFast>
__device__ __forceinline__ float one_minus_square(float l, float a) {
  if (!kFast) return -expm1f(2.f * l);
  const float z = l * (2.f * kLn2);
  float p = fmaf(z, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(z, p, 1.f / 24.f);
  p = fmaf(z, p, 1.f / 6.f);
  p = fmaf(z, p, 0.5f);
  p = fmaf(z, p, 1.f);
  return z > -0.25f ? -z * p : fmaf(-a, a, 1.f);
}

// Everything that one token of one channel has from its fused gates; rate is a_t's logarithm at an
// open recurrence gate.
template <bool kFast>
struct FusedGate {
  float l, a, sr, si, s;
  __device__ __forceinline__ FusedGate(float r, float i, float rate) {
    sr = gate_sigmoid<kFast>(r);
    si = gate_sigmoid<kFast>(i);
    l = rate * sr;
    a = decay_of<kFast>(l);
    const float q = one_minus_square<kFast>(l, a);
    s = kFast ? sqrt_approx(q) : sqrtf(q);
  }
};
__device__ __forceinline__ float gate_rate(float c, float lam, bool fast) {
  return -c * softplus_f(lam) * (fast ? kLog2e : 1.f);
}

// a h + b, a = exp(la), for a state that is rounded at every token (decode): without the error that
// rounding a makes in the same direction at every token of a long memory (1 - a to 24 bits instead of
// a); short memories take a itself, as h + (a - 1) h would lose what is left of h there.
__device__ __forceinline__ float decayed(float la, float h, float b) {
  if (la < -0.7f) return fmaf(expf(la), h, b);
  return h + fmaf(expm1f(la), h, b);
}

// ---------------------------------------------------------------- sequences

// Whether cu_seqlens [N + 1] starts at 0 and rises to at most T; called by every thread of the CTA.
__device__ __forceinline__ bool packed_lengths_fit(const int32_t* cu, int N, int T) {
  int bad = 0;
  for (int n = threadIdx.x; n <= N; n += blockDim.x) {
    const int at = cu[n];
    bad |= at > T || at < (n == 0 ? 0 : cu[n - 1]) || (n == 0 && at != 0);
  }
  return __syncthreads_or(bad) == 0;
}

// The batch's sequences on the one token axis.
struct Sequences {
  const int32_t* cu;   // NULL: rows of T tokens
  int N, T, tokens;    // tokens: of the whole axis

  __device__ __forceinline__ int begin(int n) const { return cu ? cu[n] : n * T; }
  __device__ __forceinline__ int end(int n) const { return cu ? cu[n + 1] : (n + 1) * T; }
  // The first n in [0, N] that begins at q or behind it.
  __device__ __forceinline__ int first_from(int q) const {
    if (!cu) return T ? min(N, (q + T - 1) / T) : 0;
    int lo = 0, hi = N;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] < q) lo = mid + 1; else hi = mid;
    }
    return lo;
  }
  // The sequence that token t belongs to, -1 behind the last one.
  __device__ __forceinline__ int of(int t) const {
    if (!cu) return t / T;
    int lo = 0, hi = N;   // the first n in [0, N] that begins behind t
    if (cu[N] <= t) return -1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= t) lo = mid + 1; else hi = mid;
    }
    return lo - 1;
  }
};

// A run of whole sequences [n0, n1) and their tokens [t0, t1), the part of one cluster.  The last part
// has the tokens behind the last sequence too.
struct Part {
  int n0, n1, t0, t1;
};
__device__ __forceinline__ Part part_of(const Sequences& s, int p, int parts) {
  Part r;
  r.n0 = p == 0 ? 0 : s.first_from((int)((long long)s.tokens * p / parts));
  r.n1 = p == parts - 1 ? s.N : s.first_from((int)((long long)s.tokens * (p + 1) / parts));
  r.t0 = p == 0 ? 0 : r.n0 < s.N ? s.begin(r.n0) : s.cu ? s.cu[s.N] : s.tokens;
  r.t1 = p == parts - 1 ? s.tokens : r.n1 < s.N ? s.begin(r.n1) : s.cu ? s.cu[s.N] : s.tokens;
  return r;
}

// What a warp knows of its window's tokens [w0, w0 + kTau), one bit a token.
struct Window {
  unsigned in;      // of this part
  unsigned dead;    // not in this part, in no sequence, or in a padding one: its row is zero
  unsigned first;   // a sequence's first token
  unsigned last;    // ... last token
  int row;          // lane j: the state of token j's sequence
  bool plain;       // inside one sequence: none of the above but `in`
};

// Finds windows one after the other, remembering the sequence that the last one ended in.
struct WindowFinder {
  Sequences seq;
  Part part;
  const int32_t* slots;   // NULL: states are the sequences'
  int num_slots;
  int* dev_status;
  int bos = 0, eos = 0;   // of the sequence that a neighbouring window lies in

  template <bool kLeftwards>
  __device__ __forceinline__ Window find(int w0, int lane) {
    Window w;
    w.plain = w0 > bos && w0 + kTau < eos;
    if (w.plain) {
      w.in = (1u << kTau) - 1;
      w.dead = w.first = w.last = 0;
      w.row = 0;
      return w;
    }
    const int t = w0 + (lane & (kTau - 1));
    const bool in = t >= part.t0 && t < part.t1;
    const int n = in ? seq.of(t) : -1;
    int b = 0, e = 0, row = n;
    if (n >= 0) {
      b = seq.begin(n);
      e = seq.end(n);
      if (slots) {
        row = slots[n];
        if (row < 0 || row >= num_slots) row = -1;
      }
    }
    w.in = __ballot_sync(~0u, in) & ((1u << kTau) - 1);
    w.dead = __ballot_sync(~0u, row < 0) & ((1u << kTau) - 1);
    w.first = __ballot_sync(~0u, row >= 0 && t == b) & ((1u << kTau) - 1);
    w.last = __ballot_sync(~0u, row >= 0 && t + 1 == e) & ((1u << kTau) - 1);
    w.row = row;
    const int at = kLeftwards ? 0 : kTau - 1;
    const bool live = __shfl_sync(~0u, row, at) >= 0;
    bos = __shfl_sync(~0u, b, at);
    eos = live ? __shfl_sync(~0u, e, at) : 0;
    return w;
  }
};

// ---------------------------------------------------------------- copies

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// One warp's window of one tensor: rows lo <= j < hi of kTau, kRow bytes each (`left` of them inside the
// tensor), to dst [kTau][kRow].  unit: the bytes that every row's start and end is a multiple of, 16,
// 4 or 2 (then by loads and stores: asynchronous copies have at least four bytes).
template <int kRow>
__device__ __forceinline__ void copy_window(char* dst, const char* src, long long pitch, int lo, int hi, int left,
                                            int unit, int lane) {
  if (unit == 16) {
    constexpr int kPer = kRow / 16;
    const int c = lane % kPer * 16;
#pragma unroll
    for (int k = 0; k < kTau * kPer / 32; ++k) {
      const int row = lane / kPer + k * (32 / kPer);
      if (row >= lo && row < hi && c < left) copy_async16(dst + row * kRow + c, src + row * pitch + c);
    }
  } else if (unit == 4) {
    constexpr int kPer = kRow / 4;
    constexpr int kStep = kPer >= 32 ? 1 : 32 / kPer;
#pragma unroll
    for (int k = 0; k < kTau / kStep; ++k) {
      const int row = lane / kPer + k * kStep, c = lane % kPer * 4;
      if (row >= lo && row < hi && c < left) copy_async4(dst + row * kRow + c, src + row * pitch + c);
    }
  } else {
#pragma unroll 4
    for (int row = lo; row < hi; ++row)
#pragma unroll
      for (int c = lane * 2; c < kRow; c += 64)
        if (c < left)
          *reinterpret_cast<uint16_t*>(dst + row * kRow + c) = *reinterpret_cast<const uint16_t*>(src + row * pitch + c);
  }
}

// A lane's kCh values of a row in shared memory.
template <typename T, int kCh>
__device__ __forceinline__ void read_row(const char* row, int lane, float (&x)[kCh]) {
  if constexpr (sizeof(T) == 2 && kCh == 2) {
    const float2 v = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(row)[lane]);
    x[0] = v.x;
    x[1] = v.y;
  } else {
#pragma unroll
    for (int c = 0; c < kCh; ++c) x[c] = (float)reinterpret_cast<const T*>(row)[lane * kCh + c];
  }
}
// ... to global memory; n: how many of them are inside the tensor, whole: they may go in one store.
template <typename T, int kCh>
__device__ __forceinline__ void write_row(T* row, const float (&x)[kCh], int n, bool whole) {
  if constexpr (sizeof(T) == 2 && kCh == 2) {
    if (whole) {
      *reinterpret_cast<__nv_bfloat162*>(row) = __floats2bfloat162_rn(x[0], x[1]);
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < kCh; ++c)
    if (c < n) row[c] = (T)x[c];
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// p's counterpart in the CTA of that rank.
__device__ __forceinline__ unsigned peer_address(const void* p, int rank) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((unsigned)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_peer(unsigned at, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(x) : "memory");
}
__device__ __forceinline__ void store_peer(unsigned at, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

// ---------------------------------------------------------------- launches

// How the work is shared out: parts of whole sequences, clusters of S CTAs along each part's tokens.
struct RecurrencePlan {
  int blocks, parts, S;
};

// For kernels of `width` channels and `tile` tokens a CTA, `per_sm` CTAs an SM.
inline RecurrencePlan recurrence_plan(long long tokens, int D, int N, bool packed, int width, int tile, int max_S,
                                      int per_sm) {
  const long long want = (long long)std::max(1, current_sm_count()) * per_sm;
  RecurrencePlan p;
  p.blocks = (D + width - 1) / width;
  N = std::max(1, N);
  const long long tiles = std::max(1LL, (tokens + tile - 1) / tile);
  auto parts_for = [&](long long ctas) {   // of all blocks together
    return (int)std::min<long long>({(long long)N, tiles, std::max(1LL, (ctas + p.blocks - 1) / p.blocks)});
  };
  p.S = 1;
  if (!packed) {
    p.parts = parts_for(2 * want);
    while (p.S < max_S && (long long)p.blocks * p.parts * p.S < want && 2LL * p.S * p.parts <= tiles) p.S *= 2;
  } else {
    while (p.S < max_S && 2 * p.S <= tiles) p.S *= 2;
    p.parts = std::min<long long>(parts_for((want + p.S - 1) / p.S), std::max(1LL, tiles / p.S));
  }
  return p;
}

inline int copy_unit(const void* p, long long pitch, int D, int elem) {
  const unsigned long long all = reinterpret_cast<uintptr_t>(p) | (unsigned long long)pitch * elem |
                                 (unsigned long long)D * elem;
  return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 2;
}

}  // namespace
}  // namespace gdn
