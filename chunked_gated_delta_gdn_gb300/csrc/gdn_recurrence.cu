// gdn_recurrence.cu -- the gated linear recurrence: forward and single-token decode.
//
//     h_t = a_t h_{t-1} + b_t   per channel, with a_t = exp(g_t), b_t = x_t, or
//     a_t = exp(-c softplus(lam) sigmoid(r_t)),  b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t.
//
// Forward: one reading of the inputs.  A cluster of S CTAs walks a part's tokens S tiles at a time, a
// CTA a tile of kWarps windows.  Each warp turns its window's inputs, which were copied ahead into
// shared memory, into a and b in registers and into the window's (A, L, H); windows and tiles are joined
// through shared memory of the CTA and of the cluster; with the state that enters its window each warp
// then walks its tokens.
#include <algorithm>

#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = kWarps * kTau;
constexpr int kStages = 2;
constexpr int kMaxCluster = 8;

// One window's or tile's effect on a state, for a lane's channels.
template <int kCh>
struct Step {
  float A[kCh], L[kCh], H[kCh];
};

template <typename T, typename G, bool kFused, int kCh>
struct FwdShared {
  static constexpr int kTensors = kFused ? 3 : 2;
  static constexpr int kRowX = 32 * kCh * sizeof(T), kRowG = 32 * kCh * sizeof(G);
  static constexpr int kWindow = kTau * (kRowX + (kTensors - 1) * kRowG);
  alignas(128) char ring[kStages][kWarps][kWindow];
  // the windows' steps: of every other round in `odd` where a CTA is alone; in a cluster its barrier
  // stands between a round's reads and the next one's writes, and the tiles' steps are there
  Step<kCh> even[kWarps][32];
  union {
    Step<kCh> odd[kWarps][32];
    struct {
      float L[2][kMaxCluster][kCh][32], H[2][kMaxCluster][kCh][32];
    } tile;
  };
  int warp_reset[2][kWarps];
  int tile_reset[2][kMaxCluster];
};

template <typename T, typename G, bool kFused, int kCh>
__global__ void __launch_bounds__(kThreads, 2)
    recurrence_fwd_kernel(RecurrenceArgs a, int parts, int x_unit, int g_unit, int i_unit, bool whole) {
  using Shared = FwdShared<T, G, kFused, kCh>;
  constexpr bool kFast = sizeof(T) == 2;
  extern __shared__ char shared_bytes[];
  Shared& sh = *reinterpret_cast<Shared*>(shared_bytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int S = cluster_size(), rank = cluster_rank();
  const int part_index = blockIdx.x / S % parts, block = blockIdx.x / S / parts;
  const int ch = block * 32 * kCh + lane * kCh;   // this lane's first channel
  const int mine = max(0, min(kCh, a.D - ch));
  const int left = a.D - block * 32 * kCh;
  WindowFinder finder;
  finder.seq = Sequences{a.cu_seqlens, a.num_seqs, a.T, a.cu_seqlens ? a.T : a.B * a.T};
  finder.slots = a.state_indices;
  finder.num_slots = a.num_slots;
  if (a.cu_seqlens && !packed_lengths_fit(a.cu_seqlens, a.num_seqs, a.T)) {
    // no sequence: every row is zero
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    finder.seq.N = 0;
    finder.part = Part{0, 0, (int)((long long)a.T * part_index / parts), (int)((long long)a.T * (part_index + 1) / parts)};
    for (int t = finder.part.t0 + rank * kWarps + warp; t < finder.part.t1 && a.y; t += S * kWarps)
      for (int c = 0; c < mine; ++c) static_cast<T*>(a.y)[(size_t)t * a.D + ch + c] = (T)0.f;
    return;
  }
  finder.part = part_of(finder.seq, part_index, parts);
  const Part part = finder.part;
  // empty sequences' states, and bad slots
  for (int n = part.n0 + rank * kWarps + warp; n < part.n1; n += S * kWarps) {
    int row = n;
    if (a.state_indices) {
      row = a.state_indices[n];
      if (row < 0 || row >= a.num_slots) {
        if (row != -1 && block == 0 && lane == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
        continue;
      }
    }
    if (finder.seq.end(n) > finder.seq.begin(n) || !a.final_state) continue;
    for (int c = 0; c < mine; ++c) {
      const size_t at = (size_t)row * a.D + ch + c;
      a.final_state[at] = a.initial_state ? a.initial_state[at] : 0.f;
    }
  }
  float rate[kCh];
#pragma unroll
  for (int c = 0; c < kCh; ++c) rate[c] = kFused && c < mine ? gate_rate(a.c, a.lam[ch + c], kFast) : 0.f;

  const int tile0 = part.t0 / kTile;
  const int rounds = part.t1 > part.t0 ? ((part.t1 + kTile - 1) / kTile - tile0 + S - 1) / S : 0;
  const long long px = a.x_pitch * (long long)sizeof(T), pg = a.g_pitch * (long long)sizeof(G),
                  pi = a.i_pitch * (long long)sizeof(G);
  auto window_start = [&](int round) { return (tile0 + round * S + rank) * kTile + warp * kTau; };
  auto fetch = [&](int round) {
    if (round < rounds) {
      const int w0 = window_start(round), lo = max(0, part.t0 - w0), hi = min(kTau, part.t1 - w0);
      char* const to = sh.ring[round % kStages][warp];
      const size_t first = (size_t)block * 32 * kCh;
      copy_window<Shared::kRowX>(to, static_cast<const char*>(a.x) + w0 * px + first * sizeof(T), px, lo, hi,
                                 left * (int)sizeof(T), x_unit, lane);
      copy_window<Shared::kRowG>(to + kTau * Shared::kRowX, static_cast<const char*>(a.g) + w0 * pg + first * sizeof(G),
                                 pg, lo, hi, left * (int)sizeof(G), g_unit, lane);
      if (kFused)
        copy_window<Shared::kRowG>(to + kTau * (Shared::kRowX + Shared::kRowG),
                                   static_cast<const char*>(a.i) + w0 * pi + first * sizeof(G), pi, lo, hi,
                                   left * (int)sizeof(G), i_unit, lane);
    }
    copies_close();
  };
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(k);

  if (S > 1) {   // the peers' shared memory is there once they run
    cluster_arrive();
    cluster_wait();
  }
  float carry[kCh];   // the state in front of the round's tiles
#pragma unroll
  for (int c = 0; c < kCh; ++c) carry[c] = 0.f;
  for (int round = 0; round < rounds; ++round) {
    const int w0 = window_start(round), par = round & 1;
    const Window w = finder.find<false>(w0, lane);
    const unsigned reset = w.first | w.dead;
    copies_wait<kStages - 1>();
    __syncwarp();
    // a and b of the window's tokens
    float da[kTau][kCh], db[kTau][kCh];
    Step<kCh> step;
#pragma unroll
    for (int c = 0; c < kCh; ++c) step.L[c] = 0.f;
    const char* const from = sh.ring[round % kStages][warp];
#pragma unroll
    for (int j = 0; j < kTau; ++j) {
      float x[kCh], g[kCh], i[kCh];
      read_row<T, kCh>(from + j * Shared::kRowX, lane, x);
      read_row<G, kCh>(from + kTau * Shared::kRowX + j * Shared::kRowG, lane, g);
      if (kFused) read_row<G, kCh>(from + kTau * (Shared::kRowX + Shared::kRowG) + j * Shared::kRowG, lane, i);
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
    __syncwarp();
    fetch(round + kStages);
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
    for (int c = 0; c < kCh; ++c) {
      step.A[c] = decay_of<kFast>(step.L[c]);
      step.H[c] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kTau; ++j)
#pragma unroll
      for (int c = 0; c < kCh; ++c) step.H[c] = reset >> j & 1 ? db[j][c] : fmaf(da[j][c], step.H[c], db[j][c]);
    Step<kCh>(*const windows)[32] = S == 1 && par ? sh.odd : sh.even;
    windows[warp][lane] = step;
    if (lane == 0) sh.warp_reset[par][warp] = reset != 0;
    __syncthreads();
    // the windows of the tile up to this one, and all of them
    float h[kCh], all[kCh], before[kCh], total[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) h[c] = all[c] = before[c] = total[c] = 0.f;
    bool h_reset = false, all_reset = false;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k == warp) {
        h_reset = all_reset;
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          h[c] = all[c];
          before[c] = total[c];
        }
      }
      const Step<kCh> o = windows[k][lane];
      const bool r = sh.warp_reset[par][k];
      all_reset |= r;
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        all[c] = r ? o.H[c] : fmaf(o.A[c], all[c], o.H[c]);
        total[c] += o.L[c];
      }
    }
    if (S > 1) {
      if (warp < S) {
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
          store_peer(peer_address(&sh.tile.L[par][rank][c][lane], warp), total[c]);
          store_peer(peer_address(&sh.tile.H[par][rank][c][lane], warp), all[c]);
        }
        if (lane == 0) store_peer(peer_address(&sh.tile_reset[par][rank], warp), (int)all_reset);
      }
      cluster_arrive();
      cluster_wait();
      float into[kCh], sum[kCh], run[kCh];
#pragma unroll
      for (int c = 0; c < kCh; ++c) into[c] = sum[c] = run[c] = 0.f;
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
          const float L = sh.tile.L[par][k][c][lane], H = sh.tile.H[par][k][c][lane];
          run[c] = here ? H : fmaf(decay_of<kFast>(L), run[c], H);
          sum[c] += L;
        }
      }
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        h[c] = h_reset ? h[c] : fmaf(decay_of<kFast>(before[c]), into[c], h[c]);
        carry[c] = r ? run[c] : fmaf(decay_of<kFast>(sum[c]), carry[c], run[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        h[c] = h_reset ? h[c] : fmaf(decay_of<kFast>(before[c]), carry[c], h[c]);
        carry[c] = all_reset ? all[c] : fmaf(decay_of<kFast>(total[c]), carry[c], all[c]);
      }
    }
    // the window's tokens from the state in front of it
    if (a.carries && w0 % kRecCarry == 0 && (w.in & 1)) {
#pragma unroll
      for (int c = 0; c < kCh; ++c)
        if (c < mine) a.carries[(size_t)(w0 / kRecCarry) * a.D + ch + c] = h[c];
    }
    T* const y = static_cast<T*>(a.y) + (size_t)w0 * a.D + ch;
    if (w.plain) {
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
#pragma unroll
        for (int c = 0; c < kCh; ++c) h[c] = fmaf(da[j][c], h[c], db[j][c]);
        if (a.y) write_row<T, kCh>(y + (size_t)j * a.D, h, mine, whole && mine == kCh);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kTau; ++j) {
#pragma unroll
        for (int c = 0; c < kCh; ++c) h[c] = reset >> j & 1 ? db[j][c] : fmaf(da[j][c], h[c], db[j][c]);
        if (a.y && (w.in >> j & 1)) write_row<T, kCh>(y + (size_t)j * a.D, h, mine, whole && mine == kCh);
        if (a.final_state && (w.last >> j & 1)) {
          const int row = __shfl_sync(~0u, w.row, j);
#pragma unroll
          for (int c = 0; c < kCh; ++c)
            if (c < mine) a.final_state[(size_t)row * a.D + ch + c] = h[c];
        }
      }
    }
  }
  copies_wait<0>();
}

template <typename T, typename G, bool kFused, int kCh>
cudaError_t launch_fwd(const RecurrenceArgs& a) {
  const RecurrencePlan p = recurrence_plan((long long)a.B * a.T, a.D, a.num_seqs, a.cu_seqlens != nullptr, 32 * kCh,
                                           kTile, kMaxCluster, 2);
  auto* const kernel = recurrence_fwd_kernel<T, G, kFused, kCh>;
  const size_t shared = sizeof(FwdShared<T, G, kFused, kCh>);
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
  const bool whole = a.D % kCh == 0 && reinterpret_cast<uintptr_t>(a.y) % (kCh * sizeof(T)) == 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, p.parts, copy_unit(a.x, a.x_pitch, a.D, sizeof(T)),
                            copy_unit(a.g, a.g_pitch, a.D, sizeof(G)), copy_unit(a.i, a.i_pitch, a.D, sizeof(G)), whole);
}

template <typename T, typename G, int kCh>
cudaError_t launch_fwd(const RecurrenceArgs& a) {
  return a.lam ? launch_fwd<T, G, true, kCh>(a) : launch_fwd<T, G, false, kCh>(a);
}

constexpr int kDecodeThreads = 128;

__global__ void recurrence_decode_kernel(RecurrenceArgs a) {
  const int n = blockIdx.y, d = blockIdx.x * kDecodeThreads + threadIdx.x;
  if (d >= a.D) return;
  const int slot = a.batch_indices ? a.batch_indices[n] : n;
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1 && d == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
    store_elem(a.y, (size_t)n * a.D + d, 0.f, a.io_dtype);
    return;
  }
  float la = load_elem(a.g, (size_t)n * a.g_pitch + d, a.g_dtype);
  float b = load_elem(a.x, (size_t)n * a.x_pitch + d, a.io_dtype);
  if (a.lam) {
    const FusedGate<false> f(la, load_elem(a.i, (size_t)n * a.i_pitch + d, a.g_dtype), gate_rate(a.c, a.lam[d], false));
    la = f.l;
    b *= f.s * f.si;
  }
  float* const state = a.state + (size_t)slot * a.D + d;
  const float h = decayed(la, *state, b);
  *state = h;
  store_elem(a.y, (size_t)n * a.D + d, h, a.io_dtype);
}

}  // namespace

size_t recurrence_carries_bytes(long long tokens, int D) {
  return (size_t)((tokens + kRecCarry - 1) / kRecCarry) * D * sizeof(float);
}

cudaError_t launch_recurrence_fwd(const RecurrenceArgs& a) {
  if (a.io_dtype == GDN_F32) return launch_fwd<float, float, 1>(a);
  return a.g_dtype == GDN_F32 ? launch_fwd<__nv_bfloat16, float, 1>(a) : launch_fwd<__nv_bfloat16, __nv_bfloat16, 2>(a);
}

cudaError_t launch_recurrence_decode(const RecurrenceArgs& a) {
  recurrence_decode_kernel<<<dim3((a.D + kDecodeThreads - 1) / kDecodeThreads, a.n), kDecodeThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
