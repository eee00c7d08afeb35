// gdn_recurrence.cuh -- what the kernels of the gated linear recurrence share: the gates, packed
// lengths, a warp's window of tokens and its copies, what warps and CTAs tell one another.
//
// The tokens of all sequences stand on one axis.  A CTA holds W = 32 kCh channels (a lane kCh of them,
// bf16 in pairs) and walks tiles of the axis; a warp has kTau successive tokens of a tile, its window.
// What a window does to a state is h -> 2^L h + H: windows are joined by that, and sequences' starts by
// "reset", which takes H alone (a NaN in front of it stays there).  L is a sum of logarithms: its power is
// rounded once for all the tokens that it stands for, not once a token.  From tile to tile a state goes as
// h + ((2^L - 1) h + H), and what the last sum rounds off goes into the next tile's H: where decays are the same
// all the time every tile's rounding is, too, and would add up over a long memory (2^19 tokens: a state was 7.3e-5
// off after 2048 tiles and e, backwards, 1.3e-4 after 4096; 3.0e-6 and 1.8e-6 now, in the same time).
//
// A window's warp knows L and H without its neighbours.  It then gets what is in front of it from the
// warp of the window before, passes on what is behind it, and walks its tokens: no barrier of the
// CTA, a chain of short hand-overs through shared memory that runs ahead of the walking.
#pragma once

#include <algorithm>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_recurrence.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

// ---------------------------------------------------------------- gates

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A lane's values of a token, one for each of its channels.
template <int N>
struct Lanes {
  float v[N];
};
template <typename F, int N, typename... More>
__device__ __forceinline__ Lanes<N> each(F f, const Lanes<N>& x, const More&... more) {
  Lanes<N> r;
#pragma unroll
  for (int c = 0; c < N; ++c) r.v[c] = f(x.v[c], more.v[c]...);
  return r;
}
template <int N> __device__ __forceinline__ Lanes<N> fill(float x) {
  Lanes<N> r;
#pragma unroll
  for (int c = 0; c < N; ++c) r.v[c] = x;
  return r;
}
template <int N> __device__ __forceinline__ Lanes<N> operator+(const Lanes<N>& a, const Lanes<N>& b) {
  return each([](float x, float y) { return x + y; }, a, b);
}
template <int N> __device__ __forceinline__ Lanes<N> operator*(const Lanes<N>& a, const Lanes<N>& b) {
  return each([](float x, float y) { return x * y; }, a, b);
}
template <int N> __device__ __forceinline__ Lanes<N> operator*(const Lanes<N>& a, float b) {
  return each([=](float x) { return x * b; }, a);
}
template <int N>
__device__ __forceinline__ Lanes<N> fma(const Lanes<N>& a, const Lanes<N>& b, const Lanes<N>& c) {
  return each([](float x, float y, float z) { return fmaf(x, y, z); }, a, b, c);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int N> __device__ __forceinline__ Lanes<N> ex2(const Lanes<N>& x) {
  return each([](float v) { return ex2(v); }, x);
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-x).
__device__ __forceinline__ float gate_sigmoid(float x) { return rcp(1.f + ex2(x * -kLog2e)); }

// 1 - a^2 of a = 2^l.  Where a is near 1 the difference would lose its digits: there (1 - e^-z) / z, z = -2 ln a
// in [0, 1/2], as the polynomial of degree 4 with the least relative error (8e-8), here in powers of l.
// Behind the border a's own error, 2^-22, makes at most 8e-7 of it.  (Its root has half of either.)
__device__ __forceinline__ float one_minus_square(float l, float a) {
  const float near = l * fmaf(l, fmaf(l, fmaf(l, fmaf(l, -0.034668292f, -0.15143253f), -0.44371712f), -0.96089161f), -1.3862943f);
  return l > -0.36067376f ? near : fmaf(-a, a, 1.f);
}

// The gates' arithmetic of a lane's channels, packed where there are two (the rest is not: pairs that live long
// spill).
__device__ __forceinline__ float2 pair(const Lanes<2>& x) { return make_float2(x.v[0], x.v[1]); }
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
__device__ __forceinline__ Lanes<2> lanes(float2 x) { return Lanes<2>{{x.x, x.y}}; }
template <int N> __device__ __forceinline__ Lanes<N> times(const Lanes<N>& a, const Lanes<N>& b) {
  if constexpr (N == 2) return lanes(__fmul2_rn(pair(a), pair(b)));
  else return a * b;
}
template <int N> __device__ __forceinline__ Lanes<N> gate_sigmoid(const Lanes<N>& x) {
  if constexpr (N == 2) {
    const float2 y = __fmul2_rn(pair(x), pair(-kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2(y.x), ex2(y.y)), pair(1.f));
    return lanes(make_float2(rcp(d.x), rcp(d.y)));
  } else {
    return each([](float v) { return gate_sigmoid(v); }, x);
  }
}
template <int N> __device__ __forceinline__ Lanes<N> one_minus_square(const Lanes<N>& l, const Lanes<N>& a) {
  if constexpr (N == 2) {
    const float2 z = pair(l);
    float2 p = __ffma2_rn(z, pair(-0.034668292f), pair(-0.15143253f));
    p = __ffma2_rn(z, p, pair(-0.44371712f));
    p = __ffma2_rn(z, p, pair(-0.96089161f));
    p = __ffma2_rn(z, p, pair(-1.3862943f));
    p = __fmul2_rn(z, p);
    const float2 far = __ffma2_rn(make_float2(-a.v[0], -a.v[1]), pair(a), pair(1.f));
    return lanes(make_float2(z.x > -0.36067376f ? p.x : far.x, z.y > -0.36067376f ? p.y : far.y));
  } else {
    return each([](float l, float a) { return one_minus_square(l, a); }, l, a);
  }
}

// The logarithm (to base 2) of a_t at an open recurrence gate.
__device__ __forceinline__ float gate_rate(float c, float lam) { return -c * softplus_f(lam) * kLog2e; }

// 2^l - 1 of |l| < 1/2: (2^l - 1) / l as the polynomial of degree 5 with the least relative error (2e-8).
__device__ __forceinline__ float ex2_less_one(float l) {
  return l * fmaf(l, fmaf(l, fmaf(l, fmaf(l, fmaf(l, 0.000154035122f, 0.00133907353f), 0.00961823761f), 0.0555035733f), 0.240226492f), 0.693147182f);
}
// base <- 2^l base + h; returns what its rounding leaves out where |l| < 1/2.  (Otherwise it is forgotten before it
// adds up.)
__device__ __forceinline__ float pass(float l, float h, float* base) {
  const bool near = fabsf(l) < 0.5f;
  const float kept = near ? *base : 0.f, d = fmaf(near ? ex2_less_one(l) : ex2(l), *base, h);
  *base = kept + d;
  return d - (*base - kept);
}
template <int N> __device__ __forceinline__ Lanes<N> pass(const Lanes<N>& L, const Lanes<N>& H, Lanes<N>* base) {
  Lanes<N> left;
#pragma unroll
  for (int c = 0; c < N; ++c) left.v[c] = pass(L.v[c], H.v[c], &base->v[c]);
  return left;
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

// A run of whole sequences [n0, n1) and their tokens [t0, t1): what one CTA of a block of channels walks, or
// several, a segment each.  The last part has the tokens behind the last sequence too.
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

// What a warp knows of its window's tokens [w0, w0 + kTau), one bit a token (kTau 8 or 16).
struct Window {
  unsigned in;      // of this part
  unsigned dead;    // not in this part, in no sequence, or in a padding one: its row is zero
  unsigned first;   // a sequence's first token
  unsigned last;    // ... last token
  int row;          // lane j: the state of token j's sequence
  int n;            // lane j: that sequence
  bool plain;       // inside one sequence: none of the above but `in`
};

// Finds windows one after the other, remembering the sequence that the last one ended in.
struct WindowFinder {
  Sequences seq;
  Part part;
  const int32_t* slots;   // NULL: states are the sequences'
  int num_slots;
  int bos = 0, eos = 0;   // of the sequence that a neighbouring window lies in

  template <int kTau, bool kLeftwards>
  __device__ __forceinline__ Window find(int w0, int lane) {
    Window w;
    w.plain = w0 > bos && w0 + kTau < eos;
    w.in = (1u << kTau) - 1;
    w.dead = w.first = w.last = 0;
    w.row = w.n = 0;
    if (!w.plain) look<kTau, kLeftwards>(w0, lane, &w);
    return w;
  }

  template <int kTau, bool kLeftwards>
  __device__ __forceinline__ void look(int w0, int lane, Window* w) {
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
    constexpr unsigned all = (1u << kTau) - 1;
    w->in = __ballot_sync(~0u, in) & all;
    w->dead = __ballot_sync(~0u, row < 0) & all;
    w->first = __ballot_sync(~0u, row >= 0 && t == b) & all;
    w->last = __ballot_sync(~0u, row >= 0 && t + 1 == e) & all;
    w->row = row;
    w->n = n;
    const int at = kLeftwards ? 0 : kTau - 1;
    const bool live = __shfl_sync(~0u, row, at) >= 0;
    bos = __shfl_sync(~0u, b, at);
    eos = __shfl_sync(~0u, live ? e : 0, at);
  }
};

// ---------------------------------------------------------------- copies

// The lanes that have channels: where rows do not start on 16 bytes, 28, so that the 16-byte blocks that a row of
// bf16 pairs or fp32 values lies in are no more than the 128 bytes of a whole one.
template <bool kBoxes> constexpr int kLanes = kBoxes ? 32 : 28;
// What a row of E, N a lane, takes in shared memory.
template <typename E, int N, bool kBoxes>
constexpr int kRowBytes = kBoxes ? 32 * N * (int)sizeof(E) : (kLanes<false> * N * (int)sizeof(E) + 30 - (int)sizeof(E) + 1) / 16 * 16;

// A tensor's rows where they do not come in boxes.  (bf16 with fused gates, 4 x 8192 x 1001: forward 134 us, backward
// 214; a bulk copy a row 151 and 234; copies of 4 bytes, 2 where rows are odd, 275 and 408.  1000 channels, in
// boxes: 88 and 152.)
struct Rows {
  const char* base;
  long long pitch;   // bytes
  const char* end;   // of the last row

  template <typename E>
  static __device__ __forceinline__ Rows of(const void* p, long long pitch, int tokens, int D) {
    const char* const base = static_cast<const char*>(p);
    return Rows{base, pitch * (long long)sizeof(E), base + ((tokens - 1) * pitch + D) * (long long)sizeof(E)};
  }
  // Where in its 16-byte block row `token` has its byte `at`.
  __device__ __forceinline__ int shift(int token, int at) const {
    return (int)((reinterpret_cast<uintptr_t>(base) + token * pitch + at) & 15);
  }
  // Bytes [at, at + bytes) of the rows of tokens w0 <= t < w0 + kTau that are in [t0, t1), to dst [kTau][kRow]: the
  // 16-byte blocks that they lie in, asynchronously; one warp.  Of blocks that reach beyond the tensor, the row's
  // values alone.
  template <typename E, int kTau, int kRow>
  __device__ __forceinline__ void copy(char* dst, int w0, int t0, int t1, int at, int bytes, int lane) const {
    constexpr int kBlocks = kRow / 16;
#pragma unroll 2
    for (int k = lane; k < kTau * kBlocks; k += 32) {
      const int row = k / kBlocks, token = w0 + row;
      const char* const from = base + token * pitch + at;
      const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15), c = k % kBlocks * 16 - shift;   // in the row
      if (token < t0 || token >= t1 || c >= bytes) continue;
      char* const to = dst + row * kRow + shift;
      if (from + c >= base && from + c + 16 <= end) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + c)), "l"(from + c) : "memory");
      } else {
        for (int v = max(c, 0); v < min(c + 16, bytes); v += sizeof(E))
          *reinterpret_cast<E*>(to + v) = *reinterpret_cast<const E*>(from + v);
      }
    }
  }
};
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Rows that start and end on 16 bytes: the box [kTau][W] of a map made by rows_map; one thread.
__device__ __forceinline__ void tma_window(char* dst, const CUtensorMap* map, uint64_t* bar, int channel, int token) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(channel), "r"(token)
      : "memory");
}

// A lane's values of a row in shared memory, and to global memory: n of them are inside the tensor; whole:
// all or none, and they may go in one access.
template <bool kWhole, typename T, int N>
__device__ __forceinline__ Lanes<N> read_row(const char* row, int lane) {
  Lanes<N> x;
  if constexpr (kWhole && N == 2 && sizeof(T) == 2) {
    const float2 v = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(row)[lane]);
    x.v[0] = v.x;
    x.v[1] = v.y;
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) x.v[c] = (float)reinterpret_cast<const T*>(row)[lane * N + c];
  }
  return x;
}
template <bool kWhole, typename T, int N>
__device__ __forceinline__ void write_row(T* row, const Lanes<N>& x, int n) {
  if constexpr (kWhole && N == 2 && sizeof(T) == 2) {
    if (n > 0) *reinterpret_cast<__nv_bfloat162*>(row) = __floats2bfloat162_rn(x.v[0], x.v[1]);
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c)
      if (c < n) row[c] = (T)x.v[c];
  }
}
// ... of fp32 states; zero where there is no tensor.
template <int N>
__device__ __forceinline__ Lanes<N> read_state(const float* row, int n) {
  Lanes<N> x;
#pragma unroll
  for (int c = 0; c < N; ++c) x.v[c] = row && c < n ? row[c] : 0.f;
  return x;
}
template <int N>
__device__ __forceinline__ void write_state(float* row, const Lanes<N>& x, int n) {
#pragma unroll
  for (int c = 0; c < N; ++c)
    if (c < n) row[c] = x.v[c];
}

// ---------------------------------------------------------------- hand-overs

// A wait of at most this many tries, 2 s: the hardware gives one that finds nothing 3.8 us.  One that has run out is
// reported, and none of its kind follows it: what the launch writes is then not to be used.
constexpr int kTries = 1 << 19;
__device__ __forceinline__ bool wait_some(uint64_t* bar, unsigned parity, int tries = kTries) {
  for (int k = 0; k < tries; ++k)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
constexpr unsigned kMessage = 1, kCopy = 2;   // the kinds
__device__ __forceinline__ void wait_or_report(uint64_t* bar, unsigned parity, unsigned* lost, int* dev_status,
                                               int tries = kTries) {
  if (*lost & kMessage || wait_some(bar, parity, tries)) return;
  *lost |= kMessage;
  report(dev_status, GDN_DEV_TIMEOUT);
}
// A round's copies.  Behind one that does not arrive nothing is fetched any more, and those under way are given the
// same time again: no copy outlives its CTA.
template <int kStages, int kWarps>
__device__ __forceinline__ void wait_for_copies(uint64_t (*arrived)[kWarps], int warp, int round, int rounds, unsigned* lost,
                                                int* dev_status, int tries = kTries) {
  if (*lost & kCopy || wait_some(&arrived[round % kStages][warp], round / kStages & 1, tries)) return;
  *lost |= kCopy;
  report(dev_status, GDN_DEV_TIMEOUT);
  for (int k = round; k < min(round + kStages, rounds); ++k)
    wait_some(&arrived[k % kStages][warp], k / kStages & 1, tries);
}

// The state in front of a window: 2^L base + H.
template <int N>
struct Front {
  Lanes<N> base, L, H;
  __device__ __forceinline__ Lanes<N> value() const { return fma(ex2(L), base, H); }
};

// A CTA's windows stand in one chain: `Front` goes from warp to warp and from the last one to the first one's
// next round.  A slot is written again one round later, by a warp that has had its own message of that
// round, for which the ring of messages has gone round since the slot was read.
template <int kWarps, int N>
struct Chain {
  Front<N> slot[kWarps][32];
  Lanes<N> last[32];   // what is behind the last window
  alignas(8) uint64_t full[kWarps];

  __device__ __forceinline__ void init() {   // one thread; a barrier follows
    for (int k = 0; k < kWarps; ++k) mbar_init(&full[k], 1);
    fence_mbar_init();
  }

  // One warp: what is in front of the first window.
  __device__ __forceinline__ void start(int lane, const Lanes<N>& state) {
    send(0, lane, Front<N>{state, fill<N>(0.f), fill<N>(0.f)});
  }

  // The state in front of this warp's window (L, H), after handing on what is behind it.  `order`: the
  // window's place in its tile.
  __device__ __forceinline__ Lanes<N> hand_over(int order, int round, int rounds, int lane, const Lanes<N>& L,
                                                const Lanes<N>& H, bool reset, unsigned* lost,
                                                int* dev_status) {
    const Lanes<N> A = ex2(L);   // (the way from message to message is what the chain's speed depends on)
    wait_or_report(&full[order], round & 1, lost, dev_status);
    const Front<N> f = slot[order][lane];
    Front<N> behind{f.base, f.L + L, fma(A, f.H, H)};
    if (reset) {
      behind.H = H;
      behind.L = behind.base = fill<N>(0.f);
    }
    if (order + 1 < kWarps) {
      send(order + 1, lane, behind);
    } else {
      behind.H = pass(behind.L, behind.H, &behind.base);
      behind.L = fill<N>(0.f);
      if (round + 1 < rounds) send(0, lane, behind);
      else last[lane] = behind.base;
    }
    return f.value();
  }

  // Behind the last of `rounds`, for the last window's warp.
  __device__ __forceinline__ Lanes<N> end(int rounds, int lane) const { return rounds > 0 ? last[lane] : fill<N>(0.f); }

 private:
  __device__ __forceinline__ void send(int to, int lane, const Front<N>& f) {
    slot[to][lane] = f;
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[to]);
  }
};

// ---------------------------------------------------------------- segments

constexpr int kMaxSegments = 160;
constexpr float kReset = __builtin_huge_valf();   // in L's place: "reset"

// Where parts are too few for the SMs their tiles are cut into segments.  A first launch runs segment 0 of each,
// which has nothing in front of it; beside it a second one makes the steps (L, H) of the others but the
// last from nothing in front of them; a third one runs those and the last from the steps of the
// segments before them.  Steps: [parts][segments][2][D].  (Clusters of up to 16 CTAs with the chain in their shared
// memory: 103 us against 102 for one 32768 x 2048, but two to four times as slow where a cluster's CTAs
// have little to do, and of no use to more than 16 segments.)
struct Segments {
  int count, from, here;   // of a part; this launch's: [from, from + here)
  float first;             // segment 0's length, of another's: what making a step takes, of running

  // The first of a part's tiles that segment s has, of `tiles` from 0.
  __host__ __device__ __forceinline__ int tile(int s, int tiles) const {
    if (s == 0) return 0;
    return s == count ? tiles : (int)((float)tiles * (first + (float)(s - 1)) / (first + (float)(count - 1)));
  }
};
template <int N>
__device__ __forceinline__ void write_step(float* steps, int D, int ch, const Lanes<N>& L, const Lanes<N>& H, bool reset,
                                           int mine) {
  write_state(steps + ch, reset ? fill<N>(kReset) : L, mine);
  write_state(steps + D + ch, H, mine);
}
// The state behind the first `count` segments, for the warp that starts the chain (`starts`; nothing for the others):
// every warp joins a share of the steps, which stand in the chain's slots until that warp sends its first message.
template <int kWarps, int N>
__device__ __forceinline__ Lanes<N> behind_steps(Chain<kWarps, N>& chain, const float* first, int count, int D, int ch, int mine,
                                                 int warp, int lane, bool starts) {
  Lanes<N> L = fill<N>(0.f), H = fill<N>(0.f);
  auto behind = [](const Lanes<N>& l, const Lanes<N>& x, const Lanes<N>& h) {   // a step
    return each([](float l, float x, float h) {
      pass(l, x, &h);
      return l == kReset ? x : h;
    }, l, x, h);
  };
#pragma unroll 4
  for (int k = count * warp / kWarps; k < count * (warp + 1) / kWarps; ++k) {
    const float* const at = first + (size_t)k * 2 * D + ch;
    const Lanes<N> l = read_state<N>(at, mine), x = read_state<N>(at + D, mine);
    H = behind(l, x, H);
    L = each([](float l, float s) { return l == kReset || s == kReset ? kReset : s + l; }, l, L);
  }
  chain.slot[warp][lane].L = L;
  chain.slot[warp][lane].H = H;
  __syncthreads();
  H = fill<N>(0.f);
  for (int k = 0; k < kWarps && starts; ++k)
    H = behind(chain.slot[k][lane].L, chain.slot[k][lane].H, H);
  return H;
}

// ---------------------------------------------------------------- launches

// How the work is shared out: blocks of channels, parts of whole sequences, segments of a part's tiles.
struct RecurrencePlan {
  int blocks, parts, segments;
};

// The plan with the least time, for CTAs (one an SM) of `width` channels and tiles of `tile` tokens: waves of CTAs, each as
// many rounds as its longest part has and one more to start.  Parts are whole sequences: of equal ones the
// longest part is known, of packed ones (whose lengths the host does not know) it is taken to be longer
// than the mean by half a mean sequence.  With segments the launches side by side take `first` of the third
// one's time; two more launches take some six rounds, most of it on the host (a call on 1 x 1024 x 256 and its end:
// 37 us whole, 48 cut, of a captured graph 12 either way; 1 x 2048 x 256: 46 whole, 44 cut, 18 and 13 of a graph).
inline RecurrencePlan recurrence_plan(long long tokens, int D, int N, bool packed, int width, int tile, double first) {
  const long long sms = std::max(1, current_sm_count());
  RecurrencePlan best{(D + width - 1) / width, 1, 1};
  double least = 1e300;
  N = std::max(1, N);
  const int most_parts =
      (int)std::min<long long>({(long long)N, 64, std::max(1LL, 4 * sms / best.blocks), std::max(1LL, tokens / tile)});
  for (int parts = 1; parts <= most_parts; parts += parts < 8 ? 1 : parts / 4) {
    const double each = packed ? (double)tokens / parts + (parts > 1 ? 0.5 * (double)tokens / N : 0.)
                               : (double)tokens / N * ((N + parts - 1) / parts);
    const long long tiles = (long long)(each / tile) + 1;
    for (int waves = 0; waves <= 4; ++waves) {   // as many segments a launch as fill so many waves
      const long long fill = waves * sms / ((long long)best.blocks * parts);
      const int segments = fill < 2 ? 1 : (int)std::min<long long>({fill + 1, tiles, (long long)kMaxSegments});
      const long long ctas = (long long)best.blocks * parts * (segments > 1 ? segments - 1 : 1);
      const double turns = (double)((ctas + sms - 1) / sms);
      const double time = segments > 1 ? turns * (tiles * (1. + first) / (segments - 1 + first) + 2.) + 6. : turns * (double)(tiles + 1);
      if (time < 0.98 * least) {
        least = time;
        best.parts = parts;
        best.segments = segments;
      }
    }
  }
  return best;
}

// Every width of a CTA that a call may have.
constexpr int kWidths[] = {28, 32, 56, 64};

inline size_t steps_bytes(const RecurrencePlan& p, int D) {
  return p.segments > 1 ? (size_t)p.parts * p.segments * 2 * D * sizeof(float) : 0;
}
// The launches of a plan: `run` and `make_steps` take a RecurrenceArgs, the parts, the Segments and what follows.
template <auto run, auto make_steps, typename... Args>
cudaError_t launch_segments(const RecurrenceArgs& a, const RecurrencePlan& p, double first, int threads, size_t shared,
                            const Args&... args) {
  cudaError_t err = allow_shared<run>(shared);
  if (err != cudaSuccess) return err;
  const long long chains = (long long)p.blocks * p.parts;
  Segments s{p.segments, 0, 1, (float)first};
  run<<<(unsigned)chains, threads, shared, a.stream>>>(a, p.parts, s, args...);
  err = cudaGetLastError();
  if (err != cudaSuccess || p.segments == 1) return err;
  err = allow_shared<make_steps>(shared);
  if (err != cudaSuccess) return err;
  s.from = 1;
  s.here = p.segments - 2;
  if (s.here > 0) {
    err = launch_behind(make_steps, (unsigned)(chains * s.here), threads, shared, a.stream, a, p.parts, s, args...);
    if (err != cudaSuccess) return err;
  }
  s.here = p.segments - 1;
  return launch_behind(run, (unsigned)(chains * s.here), threads, shared, a.stream, a, p.parts, s, args...);
}

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Whether rows start and end on 16 bytes, as boxes of them have to.
inline bool box_rows(const void* p, long long pitch, int D, int elem) {
  const unsigned long long all = reinterpret_cast<uintptr_t>(p) | (unsigned long long)pitch * elem |
                                 (unsigned long long)D * elem;
  return all % 16 == 0 && pitch * elem < (1LL << 40);
}

// The map of rows [tokens, D] `pitch` elements apart for boxes of `box` tokens of `width` channels.
inline bool rows_map(CUtensorMap* m, const void* p, long long tokens, int D, long long pitch, int elem, int width, int box) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode_tiled = tensor_map_encoder();
  if (!encode_tiled) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)tokens}, strides[1] = {(cuuint64_t)pitch * elem};
  const cuuint32_t size[2] = {(cuuint32_t)width, (cuuint32_t)box}, step[2] = {1, 1};
  auto encode = [&]() {
    return encode_tiled(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                        const_cast<void*>(p), dims, strides, size, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // a thread that has made no runtime call yet (autograd's, say) has no current context
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

}  // namespace
}  // namespace gdn
