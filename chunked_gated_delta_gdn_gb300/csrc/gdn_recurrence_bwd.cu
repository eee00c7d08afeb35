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
// The forward's shape from right to left, one reading of the inputs: a CTA of four windows a tile, which
// starts from the state that the forward saved in front of it.  Windows' effects on the state (from the
// left) and on e (from the right) are published at once.  Each lane sums its channels' dlam over its
// CTA's tokens; a second launch adds the CTAs up in order.
#include <algorithm>

#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

constexpr int kWarps = kRecCarry / kTau;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = kRecCarry;
constexpr int kStages = 2;
constexpr int kMaxCluster = 8;

// A window's effect on the state in front of it (A, H) and on e behind it (A, E).
template <int kCh>
struct BothWays {
  float A[kCh], L[kCh], H[kCh], E[kCh];
};

template <typename T, typename G, bool kFused, int kCh>
struct BwdShared {
  static constexpr int kRowX = 32 * kCh * sizeof(T), kRowG = 32 * kCh * sizeof(G);
  static constexpr int kAtDy = kTau * kRowX, kAtG = 2 * kTau * kRowX, kAtI = kAtG + kTau * kRowG;
  static constexpr int kWindow = kAtG + (kFused ? 2 : 1) * kTau * kRowG;
  alignas(128) char ring[kStages][kWarps][kWindow];
  BothWays<kCh> window[2][kWarps][32];
  float tile_L[2][kMaxCluster][kCh][32], tile_E[2][kMaxCluster][kCh][32];
  float dlam[kWarps][kCh][32];
  int window_reset[2][kWarps];       // 1: of the state, 2: of e
  int tile_reset[2][kMaxCluster];
};

template <typename T, typename G, bool kFused, int kCh>
__global__ void __launch_bounds__(kThreads, 3)
    recurrence_bwd_kernel(RecurrenceArgs a, int parts, int x_unit, int g_unit, int i_unit, int dy_unit, bool whole_x,
                          bool whole_g, bool whole_i, float* dlam_part) {
  using Shared = BwdShared<T, G, kFused, kCh>;
  constexpr bool kFast = sizeof(T) == 2;
  extern __shared__ char shared_bytes[];
  Shared& sh = *reinterpret_cast<Shared*>(shared_bytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = cluster_size(), rank = cluster_rank();
  const int part_index = blockIdx.x / S % parts, block = blockIdx.x / S / parts;
  const int ch = block * 32 * kCh + lane * kCh;
  const int mine = max(0, min(kCh, a.D - ch));
  const int left = a.D - block * 32 * kCh;
  WindowFinder finder;
  finder.seq = Sequences{a.cu_seqlens, a.num_seqs, a.T, a.cu_seqlens ? a.T : a.B * a.T};
  finder.slots = nullptr;
  finder.num_slots = 0;
  float* const dlam_row = dlam_part ? dlam_part + ((size_t)part_index * S + rank) * a.D + ch : nullptr;
  if (a.cu_seqlens && !packed_lengths_fit(a.cu_seqlens, a.num_seqs, a.T)) {   // every gradient is zero
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    const int step = parts * S * kWarps, first = (part_index * S + rank) * kWarps + warp;
    for (int c = 0; c < mine; ++c) {
      for (long long t = first; t < a.T; t += step) {
        const size_t at = (size_t)t * a.D + ch + c;
        static_cast<T*>(a.dx)[at] = (T)0.f;
        static_cast<G*>(a.dg)[at] = (G)0.f;
        if (kFused) static_cast<G*>(a.di)[at] = (G)0.f;
      }
      for (long long n = first; n < a.num_seqs && a.d_initial_state; n += step)
        a.d_initial_state[(size_t)n * a.D + ch + c] = 0.f;
      if (dlam_row && warp == 0) dlam_row[c] = 0.f;
    }
    return;
  }
  finder.part = part_of(finder.seq, part_index, parts);
  const Part part = finder.part;
  if (a.d_initial_state) {   // empty sequences
    for (int n = part.n0 + rank * kWarps + warp; n < part.n1; n += S * kWarps) {
      if (finder.seq.end(n) > finder.seq.begin(n)) continue;
      for (int c = 0; c < mine; ++c) {
        const size_t at = (size_t)n * a.D + ch + c;
        a.d_initial_state[at] = a.d_final_state ? a.d_final_state[at] : 0.f;
      }
    }
  }
  float rate[kCh], dlam[kCh];
#pragma unroll
  for (int c = 0; c < kCh; ++c) {
    rate[c] = kFused && c < mine ? gate_rate(a.c, a.lam[ch + c], kFast) : 0.f;
    dlam[c] = 0.f;
  }

  const int tile_end = part.t1 > part.t0 ? (part.t1 - 1) / kTile : 0;
  const int rounds = part.t1 > part.t0 ? (tile_end - part.t0 / kTile + S) / S : 0;
  const long long px = a.x_pitch * (long long)sizeof(T), pg = a.g_pitch * (long long)sizeof(G),
                  pi = a.i_pitch * (long long)sizeof(G), pd = a.D * (long long)sizeof(T);
  auto tile_of = [&](int round) { return tile_end - (round * S + rank); };
  auto fetch = [&](int round) {
    if (round < rounds) {
      const int w0 = tile_of(round) * kTile + warp * kTau, lo = max(0, part.t0 - w0), hi = min(kTau, part.t1 - w0);
      char* const to = sh.ring[round % kStages][warp];
      const size_t first = (size_t)block * 32 * kCh;
      copy_window<Shared::kRowX>(to, static_cast<const char*>(a.x) + w0 * px + first * sizeof(T), px, lo, hi,
                                 left * (int)sizeof(T), x_unit, lane);
      copy_window<Shared::kRowX>(to + Shared::kAtDy, static_cast<const char*>(a.dy) + w0 * pd + first * sizeof(T), pd, lo,
                                 hi, left * (int)sizeof(T), dy_unit, lane);
      copy_window<Shared::kRowG>(to + Shared::kAtG, static_cast<const char*>(a.g) + w0 * pg + first * sizeof(G), pg, lo,
                                 hi, left * (int)sizeof(G), g_unit, lane);
      if (kFused)
        copy_window<Shared::kRowG>(to + Shared::kAtI, static_cast<const char*>(a.i) + w0 * pi + first * sizeof(G), pi, lo,
                                   hi, left * (int)sizeof(G), i_unit, lane);
    }
    copies_close();
  };
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(k);
  if (S > 1) {   // the peers' shared memory is there once they run
    cluster_arrive();
    cluster_wait();
  }

  float carry[kCh];   // e behind the round's tiles
#pragma unroll
  for (int c = 0; c < kCh; ++c) carry[c] = 0.f;
  for (int round = 0; round < rounds; ++round) {
    const int tile = tile_of(round), w0 = tile * kTile + warp * kTau, par = round & 1;
    const bool whole_tile = tile * (long long)kTile >= part.t0;
    float h[kCh];   // the state in front of the tile
#pragma unroll
    for (int c = 0; c < kCh; ++c) h[c] = whole_tile && c < mine ? a.carries[(size_t)tile * a.D + ch + c] : 0.f;
    const Window w = finder.find<true>(w0, lane);
    const unsigned reset = w.first | w.dead, reset_e = w.last | w.dead;
    copies_wait<kStages - 1>();
    __syncwarp();
    const char* const from = sh.ring[round % kStages][warp];
    float da[kTau][kCh], db[kTau][kCh];
    BothWays<kCh> step;
#pragma unroll
    for (int c = 0; c < kCh; ++c) step.L[c] = step.H[c] = step.E[c] = 0.f;
#pragma unroll
    for (int j = 0; j < kTau; ++j) {
      float x[kCh], g[kCh], i[kCh];
      read_row<T, kCh>(from + j * Shared::kRowX, lane, x);
      read_row<G, kCh>(from + Shared::kAtG + j * Shared::kRowG, lane, g);
      if (kFused) read_row<G, kCh>(from + Shared::kAtI + j * Shared::kRowG, lane, i);
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        if (kFused) {
          const FusedGate<kFast> f(g[c], i[c], rate[c]);
          step.L[c] += f.l;
          da[j][c] = f.a;
          db[j][c] = f.s * f.si * x[c];
        } else {
          const float l = kFast ? g[c] * kLog2e : g[c];
          step.L[c] += l;
          da[j][c] = decay_of<kFast>(l);
          db[j][c] = x[c];
        }
      }
    }
    if (reset) {   // a first token takes its sequence's state in, a dead one nothing
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
        if (!(reset >> j & 1)) continue;
        const int row = __shfl_sync(~0u, w.row, j);
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          if (w.dead >> j & 1) db[j][c] = 0.f;
          else if (a.initial_state && c < mine)
            db[j][c] = fmaf(da[j][c], a.initial_state[(size_t)row * a.D + ch + c], db[j][c]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kTau; ++j)
#pragma unroll
      for (int c = 0; c < kCh; ++c) step.H[c] = reset >> j & 1 ? db[j][c] : fmaf(da[j][c], step.H[c], db[j][c]);
#pragma unroll
    for (int j = kTau - 1; j >= 0; --j) {
      float dy[kCh];
      read_row<T, kCh>(from + Shared::kAtDy + j * Shared::kRowX, lane, dy);
      const bool last = w.last >> j & 1, dead = w.dead >> j & 1;
      const int row = last ? __shfl_sync(~0u, w.row, j) : 0;
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        if (last) step.E[c] = a.d_final_state && c < mine ? a.d_final_state[(size_t)row * a.D + ch + c] : 0.f;
        step.E[c] = dead ? 0.f : da[j][c] * (dy[c] + step.E[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < kCh; ++c) step.A[c] = decay_of<kFast>(step.L[c]);
    sh.window[par][warp][lane] = step;
    if (lane == 0) sh.window_reset[par][warp] = (reset ? 1 : 0) | (reset_e ? 2 : 0);
    __syncthreads();
    // the state through the windows in front of this one; e through those behind it, and through all
    float e[kCh], all[kCh], before[kCh], total[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) e[c] = all[c] = before[c] = total[c] = 0.f;
    bool e_reset = false, all_reset = false;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) {
        const bool r = sh.window_reset[par][k] & 1;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          const float A = sh.window[par][k][lane].A[c], H = sh.window[par][k][lane].H[c];
          h[c] = r ? H : fmaf(A, h[c], H);
        }
      }
    }
#pragma unroll
    for (int k = kWarps - 1; k >= 0; --k) {
      if (k == warp) {
        e_reset = all_reset;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          e[c] = all[c];
          before[c] = total[c];
        }
      }
      const bool r = sh.window_reset[par][k] & 2;
      all_reset |= r;
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        const BothWays<kCh>& o = sh.window[par][k][lane];
        all[c] = r ? o.E[c] : fmaf(o.A[c], all[c], o.E[c]);
        total[c] += o.L[c];
      }
    }
    float into[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) into[c] = carry[c];
    if (S > 1) {
      for (int to = warp; to < S; to += kWarps) {
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          store_peer(peer_address(&sh.tile_L[par][rank][c][lane], to), total[c]);
          store_peer(peer_address(&sh.tile_E[par][rank][c][lane], to), all[c]);
        }
        if (lane == 0) store_peer(peer_address(&sh.tile_reset[par][rank], to), (int)all_reset);
      }
      cluster_arrive();
      cluster_wait();
      float sum[kCh], run[kCh];
#pragma unroll
      for (int c = 0; c < kCh; ++c) sum[c] = run[c] = 0.f;
      bool r = false;
      for (int k = 0; k < S; ++k) {
        if (k == rank) {
#pragma unroll
          for (int c = 0; c < kCh; ++c) into[c] = r ? run[c] : fmaf(decay_of<kFast>(sum[c]), carry[c], run[c]);
        }
        const bool here = sh.tile_reset[par][k];
        r |= here;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          const float L = sh.tile_L[par][k][c][lane], E = sh.tile_E[par][k][c][lane];
          run[c] = here ? E : fmaf(decay_of<kFast>(L), run[c], E);
          sum[c] += L;
        }
      }
#pragma unroll
      for (int c = 0; c < kCh; ++c) carry[c] = r ? run[c] : fmaf(decay_of<kFast>(sum[c]), carry[c], run[c]);
    } else {
#pragma unroll
      for (int c = 0; c < kCh; ++c)
        carry[c] = all_reset ? all[c] : fmaf(decay_of<kFast>(total[c]), carry[c], all[c]);
    }
#pragma unroll
    for (int c = 0; c < kCh; ++c) e[c] = e_reset ? e[c] : fmaf(decay_of<kFast>(before[c]), into[c], e[c]);
    // the state in front of each token, in db's place
#pragma unroll
    for (int j = 0; j < kTau; ++j) {
      const bool first = w.first >> j & 1, r = reset >> j & 1;
      const int row = first ? __shfl_sync(~0u, w.row, j) : 0;
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        const float b = db[j][c];
        db[j][c] = !r ? h[c] : first && a.initial_state && c < mine ? a.initial_state[(size_t)row * a.D + ch + c] : 0.f;
        h[c] = r ? b : fmaf(da[j][c], h[c], b);
      }
    }
    // the gradients, right to left
#pragma unroll
    for (int j = kTau - 1; j >= 0; --j) {
      const bool first = w.first >> j & 1, last = w.last >> j & 1, dead = w.dead >> j & 1;
      if (!(w.in >> j & 1)) continue;
      const int row = first || last ? __shfl_sync(~0u, w.row, j) : 0;
      float x[kCh], g[kCh], i[kCh], dy[kCh], ox[kCh], og[kCh], oi[kCh];
      read_row<T, kCh>(from + Shared::kAtDy + j * Shared::kRowX, lane, dy);
      if (kFused) {
        read_row<T, kCh>(from + j * Shared::kRowX, lane, x);
        read_row<G, kCh>(from + Shared::kAtG + j * Shared::kRowG, lane, g);
        read_row<G, kCh>(from + Shared::kAtI + j * Shared::kRowG, lane, i);
      }
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        if (last) e[c] = a.d_final_state && c < mine ? a.d_final_state[(size_t)row * a.D + ch + c] : 0.f;
        const float delta = dead ? 0.f : dy[c] + e[c];
        e[c] = dead ? 0.f : da[j][c] * delta;
        if (kFused) {
          const FusedGate<kFast> f(g[c], i[c], rate[c]);
          const float u = f.si * x[c];
          // where nothing decays, s = 0, what multiplies 1 / s below goes to 0 faster
          const float dla = e[c] * (db[j][c] - (f.s > 0.f ? u * f.a / f.s : 0.f));
          ox[c] = delta * f.s * f.si;
          og[c] = dla * f.l * (kFast ? kLn2 : 1.f) * (1.f - f.sr);
          oi[c] = delta * f.s * u * (1.f - f.si);
          if (dead) ox[c] = og[c] = oi[c] = 0.f;
          else dlam[c] += dla * f.sr;
        } else {
          ox[c] = delta;
          og[c] = dead ? 0.f : e[c] * db[j][c];
        }
        if (first && a.d_initial_state && c < mine) a.d_initial_state[(size_t)row * a.D + ch + c] = e[c];
      }
      const size_t at = (size_t)(w0 + j) * a.D + ch;
      write_row<T, kCh>(static_cast<T*>(a.dx) + at, ox, mine, whole_x && mine == kCh);
      write_row<G, kCh>(static_cast<G*>(a.dg) + at, og, mine, whole_g && mine == kCh);
      if (kFused) write_row<G, kCh>(static_cast<G*>(a.di) + at, oi, mine, whole_i && mine == kCh);
    }
    __syncwarp();
    fetch(round + kStages);
  }
  copies_wait<0>();
  if (kFused && dlam_row) {
#pragma unroll
    for (int c = 0; c < kCh; ++c) sh.dlam[warp][c][lane] = dlam[c];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        float x = 0.f;
        for (int k = 0; k < kWarps; ++k) x += sh.dlam[k][c][lane];
        if (c < mine) dlam_row[c] = x;
      }
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
  return recurrence_plan((long long)B * T, D, N, packed, width, kTile, kMaxCluster, 3);
}

template <typename T, typename G, bool kFused, int kCh>
cudaError_t launch_bwd(const RecurrenceArgs& a, float* part) {
  const RecurrencePlan p = plan_of(a.B, a.T, a.D, a.num_seqs, a.cu_seqlens != nullptr, 32 * kCh);
  auto* const kernel = recurrence_bwd_kernel<T, G, kFused, kCh>;
  const size_t shared = sizeof(BwdShared<T, G, kFused, kCh>);
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)p.S, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.blocks * p.parts * p.S);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = a.stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto whole = [&](const void* q, size_t elem) {
    return a.D % kCh == 0 && reinterpret_cast<uintptr_t>(q) % (kCh * elem) == 0;
  };
  err = cudaLaunchKernelEx(&cfg, kernel, a, p.parts, copy_unit(a.x, a.x_pitch, a.D, sizeof(T)),
                           copy_unit(a.g, a.g_pitch, a.D, sizeof(G)), copy_unit(a.i, a.i_pitch, a.D, sizeof(G)),
                           copy_unit(a.dy, a.D, a.D, sizeof(T)), whole(a.dx, sizeof(T)), whole(a.dg, sizeof(G)),
                           whole(a.di, sizeof(G)), part);
  if (err != cudaSuccess || !kFused || !part) return err;
  return launch_behind(recurrence_dlam_kernel, (a.D + 31) / 32, 1024, 0, a.stream, a, (const float*)part,
                       p.parts * p.S);
}

template <typename T, typename G, int kCh>
cudaError_t launch_bwd(const RecurrenceArgs& a, float* part) {
  return a.lam ? launch_bwd<T, G, true, kCh>(a, part) : launch_bwd<T, G, false, kCh>(a, part);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// The carries (where the caller has none), then the CTAs' rows of dlam.
size_t recurrence_bwd_workspace_bytes(int B, int T, int D, int num_seqs, bool fused) {
  size_t rows = 0;
  if (fused)
    for (int packed = 0; packed < 2; ++packed)
      for (int width = 32; width <= 64; width *= 2) {
        const RecurrencePlan p = plan_of(B, T, D, num_seqs, packed, width);
        rows = std::max(rows, (size_t)p.parts * p.S);
      }
  return up256(recurrence_carries_bytes((long long)B * T, D)) + rows * D * sizeof(float);
}

cudaError_t launch_recurrence_bwd(const RecurrenceArgs& args) {
  RecurrenceArgs a = args;
  char* const ws = static_cast<char*>(a.workspace);
  float* const part = a.dlam ? reinterpret_cast<float*>(ws + up256(recurrence_carries_bytes((long long)a.B * a.T, a.D)))
                             : nullptr;
  if (!a.carries && (long long)a.B * a.T > 0) {
    RecurrenceArgs f = a;
    f.carries = a.carries = reinterpret_cast<float*>(ws);
    f.y = nullptr;
    f.dev_status = nullptr;
    const cudaError_t err = launch_recurrence_fwd(f);
    if (err != cudaSuccess) return err;
  }
  if (a.io_dtype == GDN_F32) return launch_bwd<float, float, 1>(a, part);
  return a.g_dtype == GDN_F32 ? launch_bwd<__nv_bfloat16, float, 1>(a, part)
                              : launch_bwd<__nv_bfloat16, __nv_bfloat16, 2>(a, part);
}

}  // namespace gdn
