// gdn_recurrence_bwd.cu -- gradients of the gated linear recurrence.
//
//     delta_t = dy_t + e_{t+1},  e_t = a_t delta_t   (the final state's gradient behind the last token),
//     dx_t = delta_t,   d(log a_t) = e_t h_{t-1},   d h_0 = e_1,
//
// and through the fused gates, with s = sqrt(1 - a^2) and u = sigmoid(i) x:
//     d(log a) = e (h_{t-1} - u a / s),   dr = d(log a) log a (1 - sigmoid(r)),
//     dx = delta s sigmoid(i),   di = delta s u (1 - sigmoid(i)),
//     dlam = sum of d(log a) sigmoid(r), times -c sigmoid(lam).
//
// The forward's shape from right to left, one reading of the inputs: a CTA walks tiles of kWarps windows,
// with the states that the forward saved in front of every fourth one (every 32nd token: 1/16 of a bf16 tensor's
// bytes).  A window hands on its effects on the state (to the right, up to the next saved one) and on e (to
// the left).  The gates' sigmoids and s stay in shared memory for the second half.  Each lane sums its
// channels' dlam over its CTA's tokens; a second launch adds the CTAs up in order.
//
// 5 or (fused) 7 values an element to read and write; with fused gates bound by what an SM issues, 76
// instructions an element.  bf16, 2 x 8192 x 4096 (128 CTAs on 152 SMs): fused 210 us, 4.5 TB/s, 74% of the
// issue slots used; given 140 us, 4.8 TB/s.  4 x 32768 x 4096 given: 1.02 ms, 5.3 TB/s; fp32 given 1.87 ms, 5.7, fused
// 2.39 ms, 6.3 TB/s.  Given gates leave the chain in sight: 8192 tokens are 1024 windows one after the other, and a
// message takes 0.1 us.  With s made
// again from a in the second half instead of kept it took 258 us.
#include <algorithm>

#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

constexpr int kTau = 8;
constexpr int kWarps = 16;
constexpr int kTile = kWarps * kTau;
constexpr double kFirst = 0.4;   // the time of a step, of running
constexpr int kStages = 2;
constexpr int kGroup = kRecCarry / kTau;   // windows from one saved state to the next
static_assert(kRecCarry % kTau == 0 && kTile % kRecCarry == 0, "saved states stand in front of windows");

template <typename T, typename G, bool kFused, int N, bool kBoxes>
struct BwdShared {
  static constexpr int kRowX = kRowBytes<T, N, kBoxes>, kRowG = kRowBytes<G, N, kBoxes>;
  static constexpr int kAtDy = kTau * kRowX, kAtG = 2 * kTau * kRowX, kAtI = kAtG + kTau * kRowG;
  static constexpr int kWindow = kAtG + (kFused ? 2 : 1) * kTau * kRowG;
  alignas(128) char ring[kStages][kWarps][kWindow];
  Lanes<N> sigmoid[kFused ? kWarps : 1][2][kFused ? kTau : 1][32];   // (dlam's sums in the end)
  Chain<kWarps, N> chain;              // of e, right to left
  Lanes<N> state[kWarps][32];          // the state in front of each window, left to right in a tile
  uint64_t state_full[kWarps];
  uint64_t arrived[kStages][kWarps];   // the copy engine's
};

// kBoxes: a window's inputs come in boxes, and outputs go out whole; else row by row.
template <typename T, typename G, bool kFused, int N, bool kBoxes, bool kSteps>
__global__ void __launch_bounds__(kWarps * 32, 1)
    recurrence_bwd_kernel(RecurrenceArgs a, int parts, Segments segments, float* steps, float* dlam_part, const __grid_constant__ CUtensorMap x_map,
                          const __grid_constant__ CUtensorMap dy_map, const __grid_constant__ CUtensorMap g_map,
                          const __grid_constant__ CUtensorMap i_map) {
  using Shared = BwdShared<T, G, kFused, N, kBoxes>;
  using Values = Lanes<N>;
  constexpr int W = kLanes<kBoxes> * N;
  extern __shared__ __align__(1024) char shared_bytes[];
  Shared& sh = *reinterpret_cast<Shared*>(shared_bytes);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  const int blocks = (a.D + W - 1) / W, block = blockIdx.x % blocks, segment = segments.from + blockIdx.x / blocks % segments.here,
            part_index = blockIdx.x / blocks / segments.here;
  const int ch = block * W + lane * N;
  const int mine = lane < kLanes<kBoxes> ? max(0, min(N, a.D - ch)) : 0;
  WindowFinder finder;
  finder.seq = Sequences{a.cu_seqlens, a.num_seqs, a.T, a.cu_seqlens ? a.T : a.B * a.T};
  finder.slots = nullptr;
  finder.num_slots = 0;
  float* const dlam_row = dlam_part ? dlam_part + ((size_t)part_index * segments.count + segment) * a.D + ch : nullptr;
  if (a.cu_seqlens && !packed_lengths_fit(a.cu_seqlens, a.num_seqs, a.T)) {   // every gradient is zero
    wait_for_previous();
    if (kSteps) return;
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    const int step = parts * segments.count * kWarps, first = (part_index * segments.count + segment) * kWarps + warp;
    const Values zero = fill<N>(0.f);
    for (long long t = first; t < a.T; t += step) {
      const size_t at = (size_t)t * a.D + ch;
      write_row<false>(static_cast<T*>(a.dx) + at, zero, mine);
      write_row<false>(static_cast<G*>(a.dg) + at, zero, mine);
      if (kFused) write_row<false>(static_cast<G*>(a.di) + at, zero, mine);
    }
    for (long long n = first; n < a.num_seqs && a.d_initial_state; n += step)
      write_state(a.d_initial_state + (size_t)n * a.D + ch, zero, mine);
    if (dlam_row && warp == 0) write_state(dlam_row, zero, mine);
    return;
  }
  finder.part = part_of(finder.seq, part_index, parts);
  const Part part = finder.part;
  if (a.d_initial_state && !kSteps) {   // empty sequences
    for (long long n = part.n0 + segment * kWarps + warp; n < part.n1; n += segments.count * kWarps) {
      if (finder.seq.end((int)n) > finder.seq.begin((int)n)) continue;
      const size_t at = (size_t)n * a.D + ch;
      write_state(a.d_initial_state + at, read_state<N>(a.d_final_state ? a.d_final_state + at : nullptr, mine), mine);
    }
  }
  const Values rate = each([&](float lam) { return gate_rate(a.c, lam); }, read_state<N>(kFused ? a.lam + ch : nullptr, mine));
  const Values rate_e = rate * kLn2;   // of the natural logarithm
  Values dlam = fill<N>(0.f);
  auto state_of = [&](const float* states, int row) {   // of a sequence
    return read_state<N>(states ? states + (size_t)row * a.D + ch : nullptr, mine);
  };

  // segment 0 is the rightmost one
  const int tile0 = part.t0 / kTile, tiles = part.t1 > part.t0 ? (part.t1 - 1) / kTile - tile0 + 1 : 0;
  const int first = tile0 + tiles - 1 - segments.tile(segment, tiles);
  const int rounds = segments.tile(segment + 1, tiles) - segments.tile(segment, tiles);
  auto tile_of = [&](int round) { return first - round; };
  unsigned lost = 0;   // kinds of waits that have run out
  const int tokens = finder.seq.tokens;
  const Rows rows_x = Rows::of<T>(a.x, a.x_pitch, tokens, a.D), rows_dy = Rows::of<T>(a.dy, a.D, tokens, a.D),
             rows_g = Rows::of<G>(a.g, a.g_pitch, tokens, a.D), rows_i = Rows::of<G>(a.i, a.i_pitch, tokens, a.D);
  auto shift = [&](const Rows& rows, int token, int elem) { return kBoxes ? 0 : rows.shift(token, block * W * elem); };
  auto fetch = [&](int round) {
    char* const to = sh.ring[round % kStages][warp];
    if constexpr (kBoxes) {
      if (round < rounds && lane == 0 && !(lost & kCopy)) {
        uint64_t* const bar = &sh.arrived[round % kStages][warp];
        const int w0 = tile_of(round) * kTile + warp * kTau;
        mbar_arrive_expect_tx(bar, kSteps ? kTau * (Shared::kRowX + Shared::kRowG) : Shared::kWindow);
        tma_window(to + Shared::kAtDy, &dy_map, bar, block * W, w0);
        tma_window(to + Shared::kAtG, &g_map, bar, block * W, w0);
        if (!kSteps) tma_window(to, &x_map, bar, block * W, w0);
        if (kFused && !kSteps) tma_window(to + Shared::kAtI, &i_map, bar, block * W, w0);
      }
    } else {
      if (round < rounds) {
        const int start = tile_of(round) * kTile + warp * kTau, values = min(W, a.D - block * W);
        auto copy = [&](auto elem, const Rows& rows, int at) {
          using E = decltype(elem);
          rows.template copy<E, kTau, kRowBytes<E, N, kBoxes>>(to + at, start, part.t0, part.t1, block * W * (int)sizeof(E),
                                                               values * (int)sizeof(E), lane);
        };
        copy(T{}, rows_dy, Shared::kAtDy);
        copy(G{}, rows_g, Shared::kAtG);
        if (!kSteps) copy(T{}, rows_x, 0);
        if (kFused && !kSteps) copy(G{}, rows_i, Shared::kAtI);
      }
      copies_close();
    }
  };
  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages * kWarps; ++k) mbar_init(&sh.arrived[0][k], 1);
    for (int k = 0; k < kWarps; ++k) mbar_init(&sh.state_full[k], 1);
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
                         warp + 1 == kWarps);
  }
  if (warp + 1 == kWarps) sh.chain.start(lane, start);
  Values sum = fill<N>(0.f);   // of a segment's logarithms
  bool any_reset = false;
  for (int round = 0; round < rounds; ++round) {
    const int tile = tile_of(round), w0 = tile * kTile + warp * kTau;
    Values h = fill<N>(0.f);
    if (!kSteps && warp % kGroup == 0 && w0 >= part.t0 && w0 < part.t1)
      h = read_state<N>(a.carries + (size_t)(w0 / kRecCarry) * a.D + ch, mine);
    const Window w = finder.template find<kTau, true>(w0, lane);
    const unsigned reset = w.first | w.dead, reset_e = w.last | w.dead;
    if constexpr (kBoxes) {
      wait_for_copies<kStages>(sh.arrived, warp, round, rounds, &lost, a.dev_status);
    } else {
      copies_wait<kStages - 1>();
      __syncwarp();
    }
    char* const from = sh.ring[round % kStages][warp];
    auto row_x = [&](int j) { return read_row<kBoxes, T, N>(from + j * Shared::kRowX + shift(rows_x, w0 + j, sizeof(T)), lane); };
    auto row_dy = [&](int j) {
      return read_row<kBoxes, T, N>(from + Shared::kAtDy + j * Shared::kRowX + shift(rows_dy, w0 + j, sizeof(T)), lane);
    };
    // s of a token, for the second half, where its r (and i) were: each lane's values take the place of its own (or,
    // of rows that are shifted, of a neighbour's, which has read them)
    auto keep = [&](int j, const Values& root) {
      if (!kBoxes) __syncwarp();
      float* const at = reinterpret_cast<float*>(from + Shared::kAtG + j * Shared::kRowG) + lane;
      at[0] = root.v[0];
      if constexpr (N == 2) at[(Shared::kAtI - Shared::kAtG) / 4] = root.v[1];
    };
    auto kept = [&](int j) {
      const float* const at = reinterpret_cast<const float*>(from + Shared::kAtG + j * Shared::kRowG) + lane;
      Values root;
      root.v[0] = at[0];
      if constexpr (N == 2) root.v[1] = at[(Shared::kAtI - Shared::kAtG) / 4];
      return root;
    };
    // a and b of the window's tokens, and what they do together
    Values da[kTau], db[kTau], L = fill<N>(0.f), H = fill<N>(0.f), E = fill<N>(0.f);
#pragma unroll
    for (int j = 0; j < kTau; ++j) {
      const Values g = read_row<kBoxes, G, N>(from + Shared::kAtG + j * Shared::kRowG + shift(rows_g, w0 + j, sizeof(G)), lane);
      Values l;
      if (kSteps) {
        l = kFused ? times(rate, gate_sigmoid(g)) : g * kLog2e;
        da[j] = ex2(l);
        L = L + l;
        continue;
      }
      const Values x = row_x(j);
      if (kFused) {
        const Values i = read_row<kBoxes, G, N>(from + Shared::kAtI + j * Shared::kRowG + shift(rows_i, w0 + j, sizeof(G)), lane);
        auto sigmoid = [](float x) { return gate_sigmoid(x); };   // (packed, 1% slower here)
        const Values sr = each(sigmoid, g), si = each(sigmoid, i);
        sh.sigmoid[warp][0][j][lane] = sr;
        sh.sigmoid[warp][1][j][lane] = si;
        l = times(rate, sr);
        da[j] = ex2(l);
        const Values root = each(sqrt_approx, one_minus_square(l, da[j]));
        keep(j, root);
        db[j] = times(times(root, si), x);
      } else {
        l = g * kLog2e;
        da[j] = ex2(l);
        db[j] = x;
      }
      L = L + l;
      H = fma(da[j], H, db[j]);
    }
    if (reset && !kSteps) {   // a first token takes its sequence's state in, a dead one nothing
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
        if (reset >> j & 1) {
          const int row = __shfl_sync(~0u, w.row, j);
          db[j] = w.dead >> j & 1 ? fill<N>(0.f) : fma(da[j], state_of(a.initial_state, row), db[j]);
          H = db[j];
        } else {
          H = fma(da[j], H, db[j]);
        }
      }
    }
    if (w.plain) {
#pragma unroll
      for (int j = kTau - 1; j >= 0; --j)   // (of delta; e is a of it)
        E = fma(j + 1 < kTau ? da[j + 1] : E, E, row_dy(j));
      E = da[0] * E;
    } else {
#pragma unroll
      for (int j = kTau - 1; j >= 0; --j) {
        if (w.last >> j & 1) E = state_of(a.d_final_state, __shfl_sync(~0u, w.row, j));
        E = w.dead >> j & 1 ? fill<N>(0.f) : da[j] * (row_dy(j) + E);
      }
    }
    // (a slot of the state is written again after e has come through its reader)
    if (!kSteps && warp % kGroup > 0) {
      wait_or_report(&sh.state_full[warp], round & 1, &lost, a.dev_status);
      h = sh.state[warp][lane];
    }
    if (!kSteps && warp % kGroup + 1 < kGroup) {
      sh.state[warp + 1][lane] = reset ? H : fma(ex2(L), h, H);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.state_full[warp + 1]);
    }
    const int order = kWarps - 1 - warp;
    Values e = sh.chain.hand_over(order, round, rounds, lane, L, E, reset_e != 0, &lost, a.dev_status);
    if (kSteps) {
      sum = sum + L;
      any_reset |= reset_e != 0;
      __syncwarp();
      fetch(round + kStages);
      continue;
    }
    // the state in front of each token, in db's place; then the gradients, right to left
    auto gradients = [&](auto is_plain) {
      constexpr bool plain = decltype(is_plain)::value;
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
        const Values b = db[j];
        if (!plain && (reset >> j & 1)) {
          const int row = __shfl_sync(~0u, w.row, j);
          db[j] = row >= 0 ? state_of(a.initial_state, row) : fill<N>(0.f);
          h = b;
        } else {
          db[j] = h;
          h = fma(da[j], h, b);
        }
      }
      const size_t at = (size_t)w0 * a.D + ch;
      T* const dx = static_cast<T*>(a.dx) + at;
      G* const dg = static_cast<G*>(a.dg) + at;
      G* const di = static_cast<G*>(a.di) + at;
#pragma unroll
      for (int j = kTau - 1; j >= 0; --j) {
        if (!plain && !(w.in >> j & 1)) continue;
        const bool dead = !plain && (w.dead >> j & 1);
        Values ox, og, oi;
        if (!plain && (w.last >> j & 1)) e = state_of(a.d_final_state, __shfl_sync(~0u, w.row, j));
        const Values delta = row_dy(j) + e;
        e = da[j] * delta;
        if (kFused) {
          const Values x = row_x(j);
          const Values sr = sh.sigmoid[warp][0][j][lane], si = sh.sigmoid[warp][1][j][lane];
          // where nothing decays, s = 0; what multiplies 1 / s below is 0 then (bounded, it stays finite)
          const Values root = kept(j), inv = each([](float v) { return rcp(fmaxf(v, 1e-19f)); }, root);
          const Values la = rate_e * sr, ds = delta * root, u = si * x;
          const Values dla = e * each([](float u, float a, float inv, float h) { return fmaf(-u * a, inv, h); }, u, da[j], inv, db[j]);
          ox = ds * si;
          og = each([](float d, float l, float s) { return d * fmaf(-l, s, l); }, dla, la, sr);
          oi = each([](float d, float u, float s) { return d * fmaf(-u, s, u); }, ds, u, si);
          if (dead) ox = og = oi = fill<N>(0.f);
          else dlam = fma(dla, sr, dlam);
        } else {
          ox = delta;
          og = e * db[j];
          if (dead) ox = og = fill<N>(0.f);
        }
        if (dead) e = fill<N>(0.f);
        if (!plain && (w.first >> j & 1)) {
          const int row = __shfl_sync(~0u, w.row, j);
          if (a.d_initial_state) write_state(a.d_initial_state + (size_t)row * a.D + ch, e, mine);
        }
        write_row<kBoxes>(dx + (size_t)j * a.D, ox, mine);
        write_row<kBoxes>(dg + (size_t)j * a.D, og, mine);
        if (kFused) write_row<kBoxes>(di + (size_t)j * a.D, oi, mine);
      }
    };
    if (w.plain) gradients(std::true_type{});
    else gradients(std::false_type{});
    if (kBoxes && kFused) fence_proxy_async_smem();   // (s was written where the next copies go)
    __syncwarp();
    fetch(round + kStages);
  }
  if (!kBoxes) copies_wait<0>();
  if (!kSteps && segment + 1 < segments.count && segment == 0 && warp == 0)   // (nothing is behind it)
    write_step(steps + (size_t)part_index * segments.count * 2 * a.D, a.D, ch, sum, sh.chain.end(rounds, lane), true, mine);
  if (kSteps) {   // (a segment that resets takes nothing from behind it, whatever L says)
    Values(*const sums)[32] = reinterpret_cast<Values(*)[32]>(sh.ring);
    any_reset = __syncthreads_or(any_reset);
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp > 0) return;   // the last one of the chain
    sum = fill<N>(0.f);
    for (int k = 0; k < kWarps; ++k) sum = sum + sums[k][lane];
    write_step(steps + ((size_t)part_index * segments.count + segment) * 2 * a.D, a.D, ch, sum, sh.chain.end(rounds, lane),
               any_reset, mine);
    wait_for_previous();
    return;
  }
  if (kFused && dlam_row) {
    Lanes<N>(*const sums)[32] = sh.sigmoid[0][0];
    __syncthreads();
    sums[warp][lane] = dlam;
    __syncthreads();
    if (warp == 0) {
      Values x = fill<N>(0.f);
      for (int k = 0; k < kWarps; ++k) x = x + sums[k][lane];
      write_state(dlam_row, x, mine);
    }
  }
}

// dlam from the CTAs' sums: 32 channels a CTA, 32 runs of rows side by side, all in order.
__global__ void __launch_bounds__(1024) recurrence_dlam_kernel(RecurrenceArgs a, const float* part, int rows) {
  __shared__ float run[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
  next_may_start();
  wait_for_previous();
  float x = 0.f;
  if (d < a.D)
    for (int n = (int)((long long)rows * w / 32); n < (int)((long long)rows * (w + 1) / 32); ++n)
      x += part[(size_t)n * a.D + d];
  run[w][lane] = x;
  __syncthreads();
  if (w > 0 || d >= a.D) return;
  x = 0.f;
  for (int k = 0; k < 32; ++k) x += run[k][lane];
  a.dlam[d] = x * (-a.c * sigmoid_f(a.lam[d]));
}

RecurrencePlan plan_of(int B, int T, int D, int N, bool packed, int width) {
  return recurrence_plan((long long)B * T, D, N, packed, width, kTile, kFirst);
}

template <typename T, typename G, bool kFused, int N, bool kBoxes, typename... Args>
cudaError_t launch_bwd(const RecurrenceArgs& a, const RecurrencePlan& p, float* steps, const Args&... args) {
  return launch_segments<recurrence_bwd_kernel<T, G, kFused, N, kBoxes, false>, recurrence_bwd_kernel<T, G, kFused, N, kBoxes, true>>(
      a, p, kFirst, kWarps * 32, sizeof(BwdShared<T, G, kFused, N, kBoxes>), steps, args...);
}

template <typename T, typename G, bool kFused, int N>
cudaError_t launch_bwd(const RecurrenceArgs& a, float* steps) {
  const long long tokens = (long long)a.B * a.T;
  auto whole = [&](const void* q, size_t elem) { return reinterpret_cast<uintptr_t>(q) % (N * elem) == 0; };
  const bool boxes = tokens > 0 && box_rows(a.x, a.x_pitch, a.D, sizeof(T)) && box_rows(a.g, a.g_pitch, a.D, sizeof(G)) &&
                     (!kFused || box_rows(a.i, a.i_pitch, a.D, sizeof(G))) && box_rows(a.dy, a.D, a.D, sizeof(T)) &&
                     whole(a.dx, sizeof(T)) && whole(a.dg, sizeof(G)) && whole(a.di, sizeof(G));
  const int W = (boxes ? kLanes<true> : kLanes<false>)*N;
  const RecurrencePlan p = plan_of(a.B, a.T, a.D, a.num_seqs, a.cu_seqlens != nullptr, W);
  float* const part = a.dlam ? reinterpret_cast<float*>(reinterpret_cast<char*>(steps) + up256(steps_bytes(p, a.D))) : nullptr;
  CUtensorMap mx{}, md{}, mg{}, mi{};
  if (boxes && (!rows_map(&mx, a.x, tokens, a.D, a.x_pitch, sizeof(T), W, kTau) ||
                 !rows_map(&md, a.dy, tokens, a.D, a.D, sizeof(T), W, kTau) ||
                 !rows_map(&mg, a.g, tokens, a.D, a.g_pitch, sizeof(G), W, kTau) ||
                 (kFused && !rows_map(&mi, a.i, tokens, a.D, a.i_pitch, sizeof(G), W, kTau))))
    return cudaErrorInvalidValue;
  const cudaError_t err =
      boxes ? launch_bwd<T, G, kFused, N, true>(a, p, steps, part, mx, md, mg, mi)
             : launch_bwd<T, G, kFused, N, false>(a, p, steps, part, mx, md, mg, mi);
  if (err != cudaSuccess || !kFused || !part) return err;
  return launch_behind(recurrence_dlam_kernel, (a.D + 31) / 32, 1024, 0, a.stream, a, (const float*)part,
                       p.parts * p.segments);
}

template <typename T, typename G, int N>
cudaError_t launch_bwd(const RecurrenceArgs& a, float* steps) {
  return a.lam ? launch_bwd<T, G, true, N>(a, steps) : launch_bwd<T, G, false, N>(a, steps);
}

}  // namespace

// The carries and the forward's workspace (where the caller has no carries), segments' steps, the CTAs' rows of
// dlam, for whichever plan the call will have.
size_t recurrence_bwd_workspace_bytes(int B, int T, int D, int num_seqs, bool fused) {
  size_t steps = 0, rows = 0;
  for (int packed = 0; packed < 2; ++packed)
    for (int width : kWidths) {
      const RecurrencePlan p = plan_of(B, T, D, num_seqs, packed, width);
      steps = std::max(steps, steps_bytes(p, D));
      if (fused) rows = std::max(rows, (size_t)p.parts * p.segments);
    }
  return up256(recurrence_carries_bytes((long long)B * T, D)) + up256(recurrence_fwd_workspace_bytes(B, T, D, num_seqs)) +
         up256(steps) + rows * D * sizeof(float);
}

cudaError_t launch_recurrence_bwd(const RecurrenceArgs& args) {
  RecurrenceArgs a = args;
  char* ws = static_cast<char*>(a.workspace);
  float* const carries = reinterpret_cast<float*>(ws);
  ws += up256(recurrence_carries_bytes((long long)a.B * a.T, a.D));
  void* const forward = ws;
  ws += up256(recurrence_fwd_workspace_bytes(a.B, a.T, a.D, a.num_seqs));
  float* const steps = reinterpret_cast<float*>(ws);
  if (!a.carries && (long long)a.B * a.T > 0) {
    const cudaError_t err = launch_recurrence_fwd(carries_again(a, carries, forward));
    if (err != cudaSuccess) return err;
    a.carries = carries;
  }
  if (a.io_dtype == GDN_F32) return launch_bwd<float, float, 1>(a, steps);
  return a.g_dtype == GDN_F32 ? launch_bwd<__nv_bfloat16, float, 1>(a, steps)
                              : launch_bwd<__nv_bfloat16, __nv_bfloat16, 2>(a, steps);
}

}  // namespace gdn
