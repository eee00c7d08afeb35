// gdn_recurrence.cu -- the gated linear recurrence: forward and single-token decode.
//
//     h_t = a_t h_{t-1} + b_t   per channel, with a_t = exp(g_t), b_t = x_t, or
//     a_t = exp(-c softplus(lam) sigmoid(r_t)),  b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t.
//
// Forward: one reading of the inputs where there are channels and sequences for all SMs.  A CTA walks a part's
// tokens a tile of kWarps windows at a time.  Each warp turns its window's inputs, which were copied ahead
// into shared memory, into a and b in registers and into the window's (L, H), is handed the state in front
// of its window and walks its tokens.  Few parts are cut into segments, whose steps a launch of their own
// (kSteps) makes.
//
// Bound by bytes: 3 or (fused) 4 values an element.  bf16, 4 x 32768 x 4096: given 473 us, 6.8 TB/s (a plain copy's
// rate); fused 690 us, 6.2 TB/s.  2 x 8192 x 4096 has 128 CTAs for 152 SMs; with fused gates what they issue
// counts, too (three exponentials, two reciprocals and a root among 31 instructions an element; 68% of the issue
// slots): 101 us, 5.3 TB/s; given 66 us, 6.1 TB/s.  fp32: 4 x 32768 x 4096 fused 1.24 ms, 6.9 TB/s; given 0.99 ms, 6.5.  One channel a lane (twice the CTAs, half as wide rows): 122 and
// 107 us; three stages with given gates, 523 and 68 us; 8-token windows with three CTAs an SM, and all of it in
// packed arithmetic (113 us, spilled registers), were slower too.  In segments, one 32768 x 2048 given: 101 us for
// 59 us of bytes, some of which are read twice.
#include <algorithm>

#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

constexpr int kTau = 16;
constexpr int kWarps = 16;
constexpr int kTile = kWarps * kTau;
constexpr double kFirst = 0.7;   // the time of a step, of running
constexpr int kStages = 2;

template <typename T, typename G, bool kFused, int N, bool kBoxes>
struct FwdShared {
  static constexpr int kRowX = kRowBytes<T, N, kBoxes>, kRowG = kRowBytes<G, N, kBoxes>;
  static constexpr int kAtG = kTau * kRowX, kAtI = kAtG + kTau * kRowG;
  static constexpr int kWindow = kAtG + (kFused ? 2 : 1) * kTau * kRowG;
  alignas(128) char ring[kStages][kWarps][kWindow];
  Chain<kWarps, N> chain;
  uint64_t arrived[kStages][kWarps];   // the copy engine's
};

// kBoxes: a window's inputs come in boxes, and outputs go out whole; else row by row.  states: where the steps' launch
// keeps sequences' initial states for the later one, whose final states may take their place.
template <typename T, typename G, bool kFused, int N, bool kBoxes, bool kSteps>
__global__ void __launch_bounds__(kWarps * 32, 1)
    recurrence_fwd_kernel(RecurrenceArgs a, int parts, Segments segments, float* steps, float* states,
                          const __grid_constant__ CUtensorMap x_map, const __grid_constant__ CUtensorMap g_map,
                          const __grid_constant__ CUtensorMap i_map) {
  using Shared = FwdShared<T, G, kFused, N, kBoxes>;
  using Values = Lanes<N>;
  constexpr int W = kLanes<kBoxes> * N;
  extern __shared__ __align__(1024) char shared_bytes[];
  Shared& sh = *reinterpret_cast<Shared*>(shared_bytes);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  // blocks next to one another read the same tokens' rows at about the same time (32 packed prompts of 100 to 4096
  // tokens: 388 us; with the parts next to one another 430)
  const int blocks = (a.D + W - 1) / W, block = blockIdx.x % blocks, segment = segments.from + blockIdx.x / blocks % segments.here,
            part_index = blockIdx.x / blocks / segments.here;
  const int ch = block * W + lane * N;   // this lane's first channel
  const int mine = lane < kLanes<kBoxes> ? max(0, min(N, a.D - ch)) : 0;
  WindowFinder finder;
  finder.seq = Sequences{a.cu_seqlens, a.num_seqs, a.T, a.cu_seqlens ? a.T : a.B * a.T};
  finder.slots = a.state_indices;
  finder.num_slots = a.num_slots;
  if (a.cu_seqlens && !packed_lengths_fit(a.cu_seqlens, a.num_seqs, a.T)) {   // every row is zero
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    for (long long t = (part_index * segments.count + segment) * kWarps + warp; t < a.T && a.y && !kSteps;
         t += parts * segments.count * kWarps)
      write_row<false>(static_cast<T*>(a.y) + (size_t)t * a.D + ch, fill<N>(0.f), mine);
    wait_for_previous();
    return;
  }
  finder.part = part_of(finder.seq, part_index, parts);
  const Part part = finder.part;
  // empty sequences' states, and bad slots
  for (long long n = part.n0 + segment * kWarps + warp; n < part.n1 && !kSteps; n += segments.count * kWarps) {
    int row = (int)n;
    if (a.state_indices) {
      row = a.state_indices[n];
      if (row < 0 || row >= a.num_slots) {
        if (row != -1 && block == 0 && lane == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
        continue;
      }
    }
    if (finder.seq.end((int)n) > finder.seq.begin((int)n) || !a.final_state) continue;
    const size_t at = (size_t)row * a.D + ch;
    write_state(a.final_state + at, read_state<N>(a.initial_state ? a.initial_state + at : nullptr, mine), mine);
  }
  const Values rate = each([&](float lam) { return gate_rate(a.c, lam); }, read_state<N>(kFused ? a.lam + ch : nullptr, mine));

  const int tile0 = part.t0 / kTile, tiles = part.t1 > part.t0 ? (part.t1 - 1) / kTile - tile0 + 1 : 0;
  const int first = tile0 + segments.tile(segment, tiles), rounds = tile0 + segments.tile(segment + 1, tiles) - first;
  auto window_start = [&](int round) { return (first + round) * kTile + warp * kTau; };
  unsigned lost = 0;   // kinds of waits that have run out
  const Rows rows_x = Rows::of<T>(a.x, a.x_pitch, finder.seq.tokens, a.D), rows_g = Rows::of<G>(a.g, a.g_pitch, finder.seq.tokens, a.D),
             rows_i = Rows::of<G>(a.i, a.i_pitch, finder.seq.tokens, a.D);
  auto shift = [&](const Rows& rows, int token, int elem) { return kBoxes ? 0 : rows.shift(token, block * W * elem); };
  auto fetch = [&](int round) {
    char* const to = sh.ring[round % kStages][warp];
    if constexpr (kBoxes) {
      if (round < rounds && lane == 0 && !(lost & kCopy)) {
        uint64_t* const bar = &sh.arrived[round % kStages][warp];
        const int w0 = window_start(round);
        mbar_arrive_expect_tx(bar, Shared::kWindow);
        tma_window(to, &x_map, bar, block * W, w0);
        tma_window(to + Shared::kAtG, &g_map, bar, block * W, w0);
        if (kFused) tma_window(to + Shared::kAtI, &i_map, bar, block * W, w0);
      }
    } else {
      if (round < rounds) {
        const int start = window_start(round), values = min(W, a.D - block * W);
        auto copy = [&](auto elem, const Rows& rows, int at) {
          using E = decltype(elem);
          rows.template copy<E, kTau, kRowBytes<E, N, kBoxes>>(to + at, start, part.t0, part.t1, block * W * (int)sizeof(E),
                                                               values * (int)sizeof(E), lane);
        };
        copy(T{}, rows_x, 0);
        copy(G{}, rows_g, Shared::kAtG);
        if (kFused) copy(G{}, rows_i, Shared::kAtI);
      }
      copies_close();
    }
  };
  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages * kWarps; ++k) mbar_init(&sh.arrived[0][k], 1);
    sh.chain.init();
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(k);

  next_may_start();
  Values start = fill<N>(0.f);
  if (!kSteps && segment > 0) {
    wait_for_previous();
    start = behind_steps(sh.chain, steps + (size_t)part_index * segments.count * 2 * a.D, segment, a.D, ch, mine, warp, lane,
                         warp == 0);
  }
  if (warp == 0) sh.chain.start(lane, start);
  Values sum = fill<N>(0.f);   // of a segment's logarithms
  bool any_reset = false;
  // a first token's initial state: lane j's sequence, of which lanes know the cache's row and the number
  const bool saved = !kSteps && states && segment > 0 && segment + 1 < segments.count;
  auto initial = [&](const Window& w, int j) {
    const int row = __shfl_sync(~0u, saved ? w.n : w.row, j);
    const float* const from = saved ? states : a.initial_state;
    const Values h = read_state<N>(from ? from + (size_t)row * a.D + ch : nullptr, mine);
    if (kSteps && states) write_state(states + (size_t)__shfl_sync(~0u, w.n, j) * a.D + ch, h, mine);
    return h;
  };
  for (int round = 0; round < rounds; ++round) {
    const int w0 = window_start(round);
    const Window w = finder.template find<kTau, false>(w0, lane);
    const unsigned reset = w.first | w.dead;
    if constexpr (kBoxes) {
      wait_for_copies<kStages>(sh.arrived, warp, round, rounds, &lost, a.dev_status);
    } else {
      copies_wait<kStages - 1>();
      __syncwarp();
    }
    // a and b of the window's tokens, and what they do together
    Values da[kTau], db[kTau], L = fill<N>(0.f), H = fill<N>(0.f);
    const char* const from = sh.ring[round % kStages][warp];
#pragma unroll
    for (int j = 0; j < kTau; ++j) {
      const Values x = read_row<kBoxes, T, N>(from + j * Shared::kRowX + shift(rows_x, w0 + j, sizeof(T)), lane);
      const Values g = read_row<kBoxes, G, N>(from + Shared::kAtG + j * Shared::kRowG + shift(rows_g, w0 + j, sizeof(G)), lane);
      Values l;
      if (kFused) {
        const Values i = read_row<kBoxes, G, N>(from + Shared::kAtI + j * Shared::kRowG + shift(rows_i, w0 + j, sizeof(G)), lane);
        l = times(rate, gate_sigmoid(g));
        da[j] = ex2(l);
        db[j] = times(times(each(sqrt_approx, one_minus_square(l, da[j])), gate_sigmoid(i)), x);
      } else {
        l = g * kLog2e;
        da[j] = ex2(l);
        db[j] = x;
      }
      L = L + l;
      H = fma(da[j], H, db[j]);
    }
    if (kSteps) {
      __syncwarp();
      fetch(round + kStages);
    }
    if (reset) {   // a first token takes its sequence's state in, a dead one nothing
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
        if (reset >> j & 1) {
          db[j] = w.dead >> j & 1 ? fill<N>(0.f) : fma(da[j], initial(w, j), db[j]);
          H = db[j];
        } else {
          H = fma(da[j], H, db[j]);
        }
      }
    }
    Values h = sh.chain.hand_over(warp, round, rounds, lane, L, H, reset != 0, &lost, a.dev_status);
    if (kSteps) {
      sum = sum + L;
      any_reset |= reset != 0;
      continue;
    }
    // the window's tokens from the state in front of it
    if (a.carries && w0 % kRecCarry == 0 && (w.in & 1)) write_state(a.carries + (size_t)(w0 / kRecCarry) * a.D + ch, h, mine);
    T* const y = static_cast<T*>(a.y) + (size_t)w0 * a.D + ch;
    if (w.plain && a.y) {
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
        h = fma(da[j], h, db[j]);
        write_row<kBoxes>(y + (size_t)j * a.D, h, mine);
      }
    } else if (!w.plain) {
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
        h = reset >> j & 1 ? db[j] : fma(da[j], h, db[j]);
        if (a.y && (w.in >> j & 1)) write_row<kBoxes>(y + (size_t)j * a.D, h, mine);
        if (w.last >> j & 1) {
          const int row = __shfl_sync(~0u, w.row, j);
          if (a.final_state) write_state(a.final_state + (size_t)row * a.D + ch, h, mine);
        }
      }
    }
    // (before the hand-over, as soon as its slot is free, the copy is too early where there are outputs: CTAs run
    // apart, and DRAM does less: 4 x 32768 x 4096 given 590 us against 473, 2 x 8192 77 against 66)
    __syncwarp();
    fetch(round + kStages);
  }
  if (!kBoxes) copies_wait<0>();
  if (!kSteps && segment + 1 < segments.count && segment == 0 && warp + 1 == kWarps)   // (nothing is in front of it)
    write_step(steps + (size_t)part_index * segments.count * 2 * a.D, a.D, ch, sum, sh.chain.end(rounds, lane), true, mine);
  if (kSteps) {   // (a segment that resets takes nothing from in front of it, whatever L says)
    Values(*const sums)[32] = reinterpret_cast<Values(*)[32]>(sh.ring);
    any_reset = __syncthreads_or(any_reset);
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp + 1 < kWarps) return;
    sum = fill<N>(0.f);
    for (int k = 0; k < kWarps; ++k) sum = sum + sums[k][lane];
    write_step(steps + ((size_t)part_index * segments.count + segment) * 2 * a.D, a.D, ch, sum, sh.chain.end(rounds, lane),
               any_reset, mine);
    wait_for_previous();
  }
}

RecurrencePlan plan_of(int B, int T, int D, int N, bool packed, int width) {
  return recurrence_plan((long long)B * T, D, N, packed, width, kTile, kFirst);
}

template <typename T, typename G, bool kFused, int N, bool kBoxes, typename... Args>
cudaError_t launch_fwd(const RecurrenceArgs& a, const RecurrencePlan& p, const Args&... args) {
  float* const steps = static_cast<float*>(a.workspace);
  float* const states = p.segments > 1 && a.initial_state && a.final_state
                            ? reinterpret_cast<float*>(static_cast<char*>(a.workspace) + up256(steps_bytes(p, a.D)))
                            : nullptr;
  return launch_segments<recurrence_fwd_kernel<T, G, kFused, N, kBoxes, false>, recurrence_fwd_kernel<T, G, kFused, N, kBoxes, true>>(
      a, p, kFirst, kWarps * 32, sizeof(FwdShared<T, G, kFused, N, kBoxes>), steps, states, args...);
}

template <typename T, typename G, bool kFused, int N>
cudaError_t launch_fwd(const RecurrenceArgs& a) {
  const long long tokens = (long long)a.B * a.T;
  const bool boxes = tokens > 0 && box_rows(a.x, a.x_pitch, a.D, sizeof(T)) && box_rows(a.g, a.g_pitch, a.D, sizeof(G)) &&
                     (!kFused || box_rows(a.i, a.i_pitch, a.D, sizeof(G))) &&
                     reinterpret_cast<uintptr_t>(a.y) % (N * sizeof(T)) == 0;
  const int W = (boxes ? kLanes<true> : kLanes<false>)*N;
  const RecurrencePlan p = plan_of(a.B, a.T, a.D, a.num_seqs, a.cu_seqlens != nullptr, W);
  CUtensorMap mx{}, mg{}, mi{};
  if (!boxes) return launch_fwd<T, G, kFused, N, false>(a, p, mx, mg, mi);
  if (!rows_map(&mx, a.x, tokens, a.D, a.x_pitch, sizeof(T), W, kTau) ||
      !rows_map(&mg, a.g, tokens, a.D, a.g_pitch, sizeof(G), W, kTau) ||
      (kFused && !rows_map(&mi, a.i, tokens, a.D, a.i_pitch, sizeof(G), W, kTau)))
    return cudaErrorInvalidValue;
  return launch_fwd<T, G, kFused, N, true>(a, p, mx, mg, mi);
}

template <typename T, typename G, int N>
cudaError_t launch_fwd(const RecurrenceArgs& a) {
  return a.lam ? launch_fwd<T, G, true, N>(a) : launch_fwd<T, G, false, N>(a);
}

constexpr int kDecodeThreads = 128;

// 8 bytes a state and 6 or 8 (bf16) of the token's.  2048 x 4096 takes 32 us given and 34 fused of a captured graph, of
// which one small kernel takes 7: 3.7 TB/s, 4.7 without those 7, so not the bytes' rate (17 us).  A thread has two
// requests under way, each of them a slot's index and, behind it, the state.  256 x 4096 takes 11 us.
// A thread has V channels of a few requests; what a channel's gates have in common it makes once.
template <typename T, typename G, bool kFused, int V>
__global__ void __launch_bounds__(kDecodeThreads) recurrence_decode_kernel(RecurrenceArgs a, int requests) {
  const int ch = (blockIdx.x * kDecodeThreads + threadIdx.x) * V;
  if (ch >= a.D) return;
  struct alignas(V * sizeof(T)) PackT { T e[V]; };
  struct alignas(V * sizeof(G)) PackG { G e[V]; };
  struct alignas(V * sizeof(float)) PackF { float e[V]; };
  float rate[V];
#pragma unroll
  for (int j = 0; j < V; ++j) rate[j] = kFused ? -a.c * softplus_f(a.lam[ch + j]) : 0.f;
  const int first = blockIdx.y * requests;
#pragma unroll 2
  for (int n = first; n < min(first + requests, a.n); ++n) {
    const int slot = a.batch_indices ? a.batch_indices[n] : n;
    PackT out;
    if (slot < 0 || slot >= a.num_slots) {
      if (slot != -1 && ch == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
#pragma unroll
      for (int j = 0; j < V; ++j) out.e[j] = (T)0.f;
    } else {
      PackF* const at = reinterpret_cast<PackF*>(a.state + (size_t)slot * a.D + ch);
      PackF h = *at;
      const PackT x = *reinterpret_cast<const PackT*>(static_cast<const T*>(a.x) + (size_t)n * a.x_pitch + ch);
      const PackG g = *reinterpret_cast<const PackG*>(static_cast<const G*>(a.g) + (size_t)n * a.g_pitch + ch);
      PackG i = g;
      if (kFused) i = *reinterpret_cast<const PackG*>(static_cast<const G*>(a.i) + (size_t)n * a.i_pitch + ch);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float la = (float)g.e[j], b = (float)x.e[j];
        if (kFused) la = rate[j] * gate_sigmoid(la);
        // a - 1, not a: rounding a would err in the same direction at every token of a long memory.  Short
        // memories take a itself, as h + (a - 1) h would lose what is left of h there.
        const float less = expm1f(la);
        if (kFused) b *= sqrtf(-less * (2.f + less)) * gate_sigmoid((float)i.e[j]);
        h.e[j] = la < -0.7f ? fmaf(expf(la), h.e[j], b) : h.e[j] + fmaf(less, h.e[j], b);
        out.e[j] = (T)h.e[j];
      }
      *at = h;
    }
    *reinterpret_cast<PackT*>(static_cast<T*>(a.y) + (size_t)n * a.D + ch) = out;
  }
}

template <typename T, typename G, bool kFused>
cudaError_t launch_decode(const RecurrenceArgs& a) {
  const bool four = a.D % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.x) % (4 * sizeof(T)) == 0 && a.x_pitch % 4 == 0 &&
                    reinterpret_cast<uintptr_t>(a.y) % (4 * sizeof(T)) == 0 &&
                    reinterpret_cast<uintptr_t>(a.g) % (4 * sizeof(G)) == 0 && a.g_pitch % 4 == 0 &&
                    (!kFused || (reinterpret_cast<uintptr_t>(a.i) % (4 * sizeof(G)) == 0 && a.i_pitch % 4 == 0));
  const int per = kDecodeThreads * (four ? 4 : 1);
  const unsigned blocks = (unsigned)(((long long)a.D + per - 1) / per);
  // as many requests a CTA as leave eight CTAs an SM, and no more than 65535 rows of them
  const long long want = std::max(1LL, 8LL * std::max(1, current_sm_count()) / blocks);
  const int requests = (int)std::max<long long>((a.n + want - 1) / want, (a.n + 65534) / 65535);
  const dim3 grid(blocks, (unsigned)((a.n + requests - 1) / requests));
  if (four) recurrence_decode_kernel<T, G, kFused, 4><<<grid, kDecodeThreads, 0, a.stream>>>(a, requests);
  else recurrence_decode_kernel<T, G, kFused, 1><<<grid, kDecodeThreads, 0, a.stream>>>(a, requests);
  return cudaGetLastError();
}

template <typename T, typename G>
cudaError_t launch_decode(const RecurrenceArgs& a) {
  return a.lam ? launch_decode<T, G, true>(a) : launch_decode<T, G, false>(a);
}

}  // namespace

size_t recurrence_carries_bytes(long long tokens, int D) {
  return (size_t)((tokens + kRecCarry - 1) / kRecCarry) * D * sizeof(float);
}

// Segments' steps, then the initial states of the sequences, for whichever plan the call will have.
size_t recurrence_fwd_workspace_bytes(int B, int T, int D, int num_seqs) {
  size_t most = 0;
  for (int packed = 0; packed < 2; ++packed)
    for (int width : kWidths) {
      const RecurrencePlan p = plan_of(B, T, D, num_seqs, packed, width);
      if (p.segments > 1) most = std::max(most, up256(steps_bytes(p, D)) + (size_t)num_seqs * D * sizeof(float));
    }
  return most;
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
  if (a.io_dtype == GDN_F32) return launch_fwd<float, float, 1>(a);
  return a.g_dtype == GDN_F32 ? launch_fwd<__nv_bfloat16, float, 1>(a) : launch_fwd<__nv_bfloat16, __nv_bfloat16, 2>(a);
}

cudaError_t launch_recurrence_decode(const RecurrenceArgs& a) {
  if (a.io_dtype == GDN_F32) return launch_decode<float, float>(a);
  return a.g_dtype == GDN_F32 ? launch_decode<__nv_bfloat16, float>(a) : launch_decode<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace gdn
