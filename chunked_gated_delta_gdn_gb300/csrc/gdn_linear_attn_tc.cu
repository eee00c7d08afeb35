// gdn_linear_attn_tc.cu -- the chunked pass of linear attention with a decay for each head on
// the tcgen05 tensor cores: bf16 I/O, any accepted head dims (padded to 64 or 128 by the TMA
// loads' zero fill).
//
// One CTA per (sequence, head, segment), chunks of 64 tokens in order.  Per chunk, with X the
// K x V state entering it and w_d = gamma^d (forward in time; the reverse pass mirrors the
// exponents, see gdn_linear_attn.h):
//
//   D    = [Q; K] K^T                      M=128 N=64  (rows 0-63 are Q K^T)
//   P_ij = s_in s_out w_{i-j} D_ij, j <= i bf16, shared memory
//   O1^T = X^T Q^T                         M=128 (value features) N=64 (tokens)
//   O2^T = V^T P^T                         M=128 N=64
//   o_i  = s_out w_{i+1} O1_i + O2_i
//   U^T  = V^T K~, K~_j = s_in w_{L-1-j} k_j     M=128 N=K
//   X   <- w_L X + U
//
// The running state lives in fp32 registers of the state warps (value feature = TMEM lane, key
// feature = column), so a chunk's only serial work on it is one multiply-add per element; the
// tensor cores see it as the bf16 A operand of O1, read from TMEM.  V is the exact input; K~ is
// not representable in bf16, so it is split into a sum of bf16 terms: two (error 2^-18, far
// below the bf16 outputs) where only outputs leave, three (24 bits, all of fp32) where the state
// does.  P and the X operand are rounded to bf16 once, like the output itself.
//
// Roles: warps 0-7 state (K~ of chunk c + 1, then the update of chunk c), warps 8-11 output,
// warps 12-13 P, warp 14 issues the MMAs, warp 15 the loads.  They meet through mbarriers; every
// wait is bounded: a timeout sets GDN_DEV_TIMEOUT, every role leaves, TMEM is freed.
#include <cuda.h>

#include <atomic>
#include <cstring>

#include "gdn_internal.h"
#include "gdn_linear_attn.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kStateWarps = 8, kOutWarps = 4, kPWarps = 2;
constexpr int kMmaWarp = 14, kLoadWarp = 15;
constexpr uint64_t kWaitNs = 2000000000ull;

// Shared memory (bytes from a 1024-byte-aligned base).
constexpr uint32_t kStage = 49152;                 // [k half][Q 64 rows | K 64 rows][128 B], V
constexpr uint32_t kStageV = 32768;                // [v half][64 tokens][128 B]
constexpr uint32_t OFF_KT = 2 * kStage;            // 2 buffers x 3 terms of K~, tiles as K's
constexpr uint32_t kKtTerm = 16384, kKtBuf = 3 * kKtTerm;
constexpr uint32_t OFF_P = OFF_KT + 2 * kKtBuf;    // [64 i][64 j] bf16
constexpr uint32_t OFF_O = OFF_P + 8192;       // output tile, [v half][64 tokens][128 B]
constexpr uint32_t OFF_W = OFF_O + 16384;          // float[72]: w_0 .. w_64
constexpr uint32_t OFF_WP = OFF_W + 288;           // factors of P, see fill_p_table
constexpr uint32_t kWpStride = 136;                // floats of one copy
constexpr uint32_t OFF_G = OFF_WP + 4 * 4 * kWpStride;   // float2[2]: decay of a full / the partial chunk
constexpr uint32_t OFF_BAR = OFF_G + 32;
constexpr uint32_t SMEM_USED = OFF_BAR + 256;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;   // slack for aligning the base
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

// TMEM columns.
constexpr uint32_t COL_U = 0, COL_D = 128, COL_X = 192, COL_O1 = 256 /* 2 x 64 */,
                   COL_O2 = 384 /* 2 x 64 */, TMEM_COLS = 512;

enum {
  B_FULL = 0,     // [2] stage landed
  B_EMPTY = 2,    // [2] stage free (MMA commit)
  B_KT = 4,       // [2] K~ written (state warps)
  B_U = 6,        // U of a chunk complete (commit)
  B_UFREE = 7,    // U read (state warps)
  B_X = 8,        // X operand written (state warps)
  B_XFREE = 9,    // O1 complete (commit): X operand read
  B_D = 10,       // D complete (commit)
  B_P = 11,       // P written, D read (P warps)
  B_O = 12,       // [2] O1, O2 complete (commit)
  B_OFREE = 14,   // [2] O1, O2 read (output warps)
  B_COUNT = 16
};
constexpr uint32_t OFF_FLAG = OFF_BAR + 8 * B_COUNT, OFF_TSLOT = OFF_FLAG + 8;

struct Unit {
  int h, bos, eos;       // the sequence
  int nch, c0, c1;       // its chunks, and the range (in order of processing) of this CTA
  const float* init;
  float* fin;
};

// A bounded wait that reads the clock only now and then (the failing polls of fifteen warps
// share the issue slots with the work they wait for).
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 0 && globaltimer_ns() - t0 > kWaitNs) return false;
  }
}
// Every lane of the warp waits; the answer is the same for all of them.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}
// Two fp32 multiply-adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2v(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// The upper halves of two fp32 values: both truncated to bf16, packed.
__device__ __forceinline__ uint32_t top2(float2 x) {
  return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
// What that truncation leaves (exact).
__device__ __forceinline__ float2 rest2(float2 x) {
  const float2 t = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                               __uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
  return fma2(t, make_float2(-1.f, -1.f), x);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

struct ChunkAt {
  int t0, L;
};
__device__ __forceinline__ ChunkAt chunk_at(const LinAttnPass& p, const Unit& u, int c) {
  const int ch = p.reverse ? u.nch - 1 - c : c;
  ChunkAt r;
  r.t0 = u.bos + ch * kChunk;
  r.L = min(kChunk, u.eos - r.t0);
  return r;
}

// ------------------------------------------------------------------ loads (one thread)
__device__ void load_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint64_t* bars,
                          const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv) {
  const int hq = u.h / (p.H / p.Hq), hk = u.h / (p.H / p.Hk), hv = u.h / (p.H / p.Hv);
  const int kh = (p.K + 63) >> 6, vh = (p.V + 63) >> 6;
  for (int c = u.c0; c < u.c1; ++c) {
    const int i = c - u.c0, s = i & 1;
    if (i >= 2 && !wait_bar(&bars[B_EMPTY + s], (uint32_t)((i - 2) >> 1) & 1u)) return;
    const int t0 = chunk_at(p, u, c).t0;
    uint8_t* st = sm + s * kStage;
    mbar_arrive_expect_tx(&bars[B_FULL + s], (uint32_t)(2 * kh + vh) * 8192u);
    for (int x = 0; x < kh; ++x) {
      tma_load_3d(st + x * 16384 + 8192, tk, &bars[B_FULL + s], 64 * x, hk, t0);
      tma_load_3d(st + x * 16384, tq, &bars[B_FULL + s], 64 * x, hq, t0);
    }
    for (int x = 0; x < vh; ++x)
      tma_load_3d(st + kStageV + x * 8192, tv, &bars[B_FULL + s], 64 * x, hv, t0);
  }
}

// ------------------------------------------------------------------ MMAs (one thread)
// `steps` MMAs of 16 K elements each; the descriptors advance by whole tiles' rows (units of 16
// bytes), and by `skip` more after every fourth (the second 64-element half of a K-major tile).
// The loops stay rolled: this code runs once a chunk between fifteen other warps' and is fetched
// anew each time, so what it costs is its length.
__device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t id, int steps,
                                      uint32_t step_a, uint32_t step_b, uint32_t skip_a, uint32_t skip_b) {
#pragma unroll 1
  for (int h = 0; h < steps; h += 4) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) mma_bf16(d, a + ks * step_a, b + ks * step_b, id, h + ks > 0);
    a += skip_a;
    b += skip_b;
  }
}

__device__ bool mma_role(const LinAttnPass& p, const Unit& u, uint32_t sb, uint32_t tbase,
                         uint64_t* bars, int terms) {
  const int kh = p.K > 64 ? 2 : 1, n = u.c1 - u.c0;
  constexpr uint32_t kS16 = kStage >> 4;
  const uint64_t dQ = sdesc_sw128(sb, 16, 1024), dK = sdesc_sw128(sb + 8192, 16, 1024),
                 dV = sdesc_sw128(sb + kStageV, 8192, 1024), dT = sdesc_sw128(sb + OFF_KT, 8192, 1024),
                 dP = sdesc_sw128(sb + OFF_P, 16, 1024);
  const uint32_t idU = kh == 2 ? idesc_bf16(128, 128, true, true) : idesc_bf16(128, 64, true, true);
  constexpr uint32_t idO1 = idesc_bf16(128, 64, false, false), idO2 = idesc_bf16(128, 64, true, false);
  if (!wait_bar(&bars[B_FULL], 0u)) return false;
  tc_fence_after();
  issue(tbase + COL_D, dQ, dK, idO1, 4 * kh, 2, 2, 1024, 1024);
  mma_commit(&bars[B_D]);
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int s = i & 1;
    const uint32_t par = (uint32_t)i & 1u, par2 = (uint32_t)(i >> 1) & 1u;
    const uint64_t q = dQ + s * kS16, v = dV + s * kS16;
    // U^T = V^T K~
    if (!wait_bar(&bars[B_KT + s], par2)) return false;
    if (i > 0 && !wait_bar(&bars[B_UFREE], par ^ 1u)) return false;
    tc_fence_after();
    issue(tbase + COL_U, v, dT + s * (kKtBuf >> 4), idU, 4 * terms, 128, 128, 0, kKtTerm >> 4);
    mma_commit(&bars[B_U]);
    // O1^T = X^T Q^T
    if (!wait_bar(&bars[B_X], par)) return false;
    if (i >= 2 && !wait_bar(&bars[B_OFREE + s], par2 ^ 1u)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int h = 0; h < kh; ++h)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_bf16_ta(tbase + COL_O1 + 64 * s, tbase + COL_X + 32 * h + 8 * ks, q + 1024 * h + 2 * ks, idO1,
                    h + ks > 0);
    if (i + 1 < n) mma_commit(&bars[B_XFREE]);
    // O2^T = V^T P^T
    if (!wait_bar(&bars[B_P], par)) return false;
    tc_fence_after();
    issue(tbase + COL_O2 + 64 * s, v, dP, idO2, 4, 128, 2, 0, 0);
    if (i + 2 < n) mma_commit(&bars[B_EMPTY + s]);
    mma_commit(&bars[B_O + s]);
    if (i + 1 < n) {
      const int s1 = s ^ 1;
      if (!wait_bar(&bars[B_FULL + s1], (uint32_t)((i + 1) >> 1) & 1u)) return false;
      tc_fence_after();
      issue(tbase + COL_D, dQ + s1 * kS16, dK + s1 * kS16, idO1, 4 * kh, 2, 2, 1024, 1024);
      mma_commit(&bars[B_D]);
    }
  }
  return true;
}

// ------------------------------------------------------------------ P (warps 12, 13)
// The factor of P_ij depends on j - i alone: f[x] for x = j - i + 63 in 0 .. 126, zero where the
// mask is.  Row i reads f[63 - i ..], four at a time: four copies shifted by one float each keep
// those reads 16-byte aligned whatever i is, and their stride of 8 banks keeps them apart.
__device__ __forceinline__ void fill_p_table(const LinAttnPass& p, float ld, float* wp, int tid) {
  for (int e = tid; e < 4 * (int)kWpStride; e += kThreads) {
    const int copy = e / (int)kWpStride, x = e - copy * (int)kWpStride + copy;   // copy[y] = f[y + copy]
    const int dist = p.reverse ? x - 63 : 63 - x;
    wp[e] = (dist >= 0 && dist < kChunk) ? p.s_in * p.s_out * decay_pow(ld, (float)dist) : 0.f;
  }
}

__device__ bool p_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase,
                       uint64_t* bars) {
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 1, row = 32 * wq + lane;
  const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
  const int shift = (63 - row) & 3;
  const float4* f4 = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm + OFF_WP) +
                                                     shift * kWpStride + (63 - row - shift));
#pragma unroll 1
  for (int c = u.c0; c < u.c1; ++c) {
    const int i = c - u.c0;
    const int L = chunk_at(p, u, c).L;
    // (D of a chunk is issued after O2 of the one before, so P has been read when it is complete)
    if (!wait_warp(&bars[B_D], (uint32_t)i & 1u)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      float x[32];
      tmem_ld32(tbase + lane_off + COL_D + 32 * half, x);
      if (L < kChunk) {   // rows and columns past the end may hold anything
#pragma unroll
        for (int jj = 0; jj < 32; ++jj)
          if (row >= L || 32 * half + jj >= L) x[jj] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 a = f4[8 * half + 2 * g], b = f4[8 * half + 2 * g + 1];
        uint4 q;
        float2 t = mul2v(make_float2(a.x, a.y), make_float2(x[8 * g], x[8 * g + 1]));
        q.x = pack2(t.x, t.y);
        t = mul2v(make_float2(a.z, a.w), make_float2(x[8 * g + 2], x[8 * g + 3]));
        q.y = pack2(t.x, t.y);
        t = mul2v(make_float2(b.x, b.y), make_float2(x[8 * g + 4], x[8 * g + 5]));
        q.z = pack2(t.x, t.y);
        t = mul2v(make_float2(b.z, b.w), make_float2(x[8 * g + 6], x[8 * g + 7]));
        q.w = pack2(t.x, t.y);
        *reinterpret_cast<uint4*>(sm + OFF_P + sw128_offset(row, 32 * half + 8 * g)) = q;
      }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    warp_arrive(&bars[B_P], lane);
  }
  return true;
}

// ------------------------------------------------------------------ state (warps 0-7)
// K~ of one chunk: each 16-byte piece of a K row scaled by its token's weight and split into
// bf16 tiles by truncation: three 8-bit pieces hold all 24 bits; with two, the second is rounded.
// Rows past the chunk's end become zero, and so do V's (they belong to another sequence, or to
// none, and a NaN there must not meet the zero).
template <int kTerms>
__device__ __forceinline__ void make_kt(const LinAttnPass& p, uint8_t* sm, int s, int L, int kh, int tid) {
  const float* w = reinterpret_cast<const float*>(sm + OFF_W);
  uint8_t* st = sm + s * kStage;
  uint8_t* kt = sm + OFF_KT + s * kKtBuf;
#pragma unroll 2
  for (int e = tid; e < 512 * kh; e += 256) {
    const int half = e >> 9, t = (e >> 3) & 63;
    const uint32_t at = (uint32_t)(t * 128 + (e & 7) * 16);
    uint32_t o[3][4] = {};
    if (t < L) {
      const uint4 k4 = *reinterpret_cast<const uint4*>(st + half * 16384 + 8192 + at);
      const float f = p.s_in * w[p.reverse ? t + 1 : L - 1 - t];
      const uint32_t in[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 x = mul2v(make_float2(f, f), make_float2(lo_f(in[j]), hi_f(in[j])));
        o[0][j] = top2(x);
        x = rest2(x);
        if (kTerms == 3) {
          o[1][j] = top2(x);
          o[2][j] = top2(rest2(x));
        } else {
          o[1][j] = pack2(x.x, x.y);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < kTerms; ++m)
      *reinterpret_cast<uint4*>(kt + m * kKtTerm + half * 8192 + at) =
          make_uint4(o[m][0], o[m][1], o[m][2], o[m][3]);
  }
  if (L < kChunk) {
    for (int e = tid; e < 1024; e += 256) {
      const int t = (e >> 3) & 63;
      if (t >= L)
        *reinterpret_cast<uint4*>(st + kStageV + (e >> 9) * 8192 + t * 128 + (e & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

template <int kTerms>
__device__ bool state_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase,
                           uint64_t* bars) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int dv = 32 * (warp & 3) + lane, dk0 = 64 * (warp >> 2);   // this thread's 64 elements
  const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
  const int kh = (p.K + 63) >> 6, n = u.c1 - u.c0;
  const bool mine = dk0 < 64 * kh;
  const float2* g = reinterpret_cast<const float2*>(sm + OFF_G);
  float2 X[32];
  auto at = [&](int j) -> float {
    const int k = dk0 + j;
    return (u.init && dv < p.V && k < p.K)
               ? u.init[p.initial_t ? (size_t)dv * p.K + k : (size_t)k * p.V + dv] : 0.f;
  };
#pragma unroll
  for (int j = 0; j < 32; ++j) X[j] = make_float2(at(2 * j), at(2 * j + 1));
  // the X operand of the next O1
  auto put_x = [&]() {
    if (mine) {
      float r[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = __uint_as_float(pack2(X[j].x, X[j].y));
      tmem_st32(tbase + lane_off + COL_X + (dk0 >> 1), r);
    }
    tc_fence_before();
    warp_arrive(&bars[B_X], lane);
  };
  put_x();
#pragma unroll 1
  for (int i = -1; i < n; ++i) {
    if (i + 1 < n) {   // K~ of the next chunk, while the MMAs of this one run
      const int s = (i + 1) & 1;
      if (!wait_warp(&bars[B_FULL + s], (uint32_t)((i + 1) >> 1) & 1u)) return false;
      make_kt<kTerms>(p, sm, s, chunk_at(p, u, u.c0 + i + 1).L, kh, tid);
      fence_proxy_async_smem();
      warp_arrive(&bars[B_KT + s], lane);
    }
    if (i < 0) continue;
    const float2 gl = g[chunk_at(p, u, u.c0 + i).L < kChunk];
    if (!wait_warp(&bars[B_U], (uint32_t)i & 1u)) return false;
    tc_fence_after();
    if (mine) {   // X <- X (hi + lo) + U
      const float2 hi = make_float2(gl.x, gl.x), lo = make_float2(gl.y, gl.y);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[32];
        tmem_ld32(tbase + lane_off + COL_U + dk0 + 32 * half, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float2& a = X[16 * half + j];
          a = fma2(a, hi, fma2(a, lo, make_float2(x[2 * j], x[2 * j + 1])));
        }
      }
    }
    tc_fence_before();
    warp_arrive(&bars[B_UFREE], lane);
    if (i + 1 < n) {
      if (!wait_warp(&bars[B_XFREE], (uint32_t)i & 1u)) return false;
      tc_fence_after();
      put_x();
    }
  }
  if (u.fin) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (dv < p.V && dk0 + j < p.K)
        u.fin[(size_t)(dk0 + j) * p.V + dv] = (j & 1) ? X[j >> 1].y : X[j >> 1].x;
  }
  return true;
}

// ------------------------------------------------------------------ output (warps 8-11)
__device__ __noinline__ void store_rows(const LinAttnPass& p, const float* w, const ChunkAt& ch,
                                        uint32_t o1, uint32_t o2, int h, int dv) {
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    float x[32], y[32];
    tmem_ld32(o1 + 32 * half, x);
    tmem_ld32(o2 + 32 * half, y);
#pragma unroll
    for (int jj = 0; jj < 32; ++jj) {
      const int t = 32 * half + jj;
      if (t < ch.L && dv < p.V)
        store_elem(p.o, ((size_t)(ch.t0 + t) * p.H + h) * p.V + dv,
                   fmaf(p.s_out * w[p.reverse ? ch.L - 1 - t : t + 1], x[jj], y[jj]),
                   p.o_f32 ? GDN_F32 : GDN_BF16);
    }
  }
}

__device__ bool out_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase,
                         uint64_t* bars, const CUtensorMap* to) {
  const int tid = threadIdx.x - 32 * kStateWarps, lane = tid & 31, wq = tid >> 5;
  const uint32_t lane_off = (uint32_t)(32 * wq) << 16, sbase = smem_u32(sm);
  const float* w = reinterpret_cast<const float*>(sm + OFF_W);
  const bool leader = tid == 0;
  bool ok = true;
#pragma unroll 1
  for (int c = u.c0; c < u.c1; ++c) {
    const int i = c - u.c0, s = i & 1;
    const ChunkAt ch = chunk_at(p, u, c);
    const uint32_t o1 = tbase + lane_off + COL_O1 + 64 * s, o2 = tbase + lane_off + COL_O2 + 64 * s;
    if (leader) tma_store_wait_read();   // the previous tile has left the staging
    ok = wait_warp(&bars[B_O + s], (uint32_t)(i >> 1) & 1u);
    if (group_sync_or(1, 32 * kOutWarps, !ok)) {
      ok = false;
      break;
    }
    tc_fence_after();
    if (ch.L < kChunk || p.o_f32) {
      store_rows(p, w, ch, o1, o2, u.h, 32 * wq + lane);
      tc_fence_before();
      warp_arrive(&bars[B_OFREE + s], lane);
      continue;
    }
    // 16x256b loads give each thread value features (t/4, t/4 + 8) x tokens (2 (t%4), + 1): the
    // fragment that stmatrix .trans writes as 16-byte rows (8 features of one token) of the
    // 128-byte-swizzled tile.  Lane l addresses feature block l / 8, token l % 8.
    const int mblk = lane >> 3, rr = lane & 7, d0 = 32 * wq + 8 * mblk;
    const uint32_t st_base = sbase + OFF_O + (d0 >> 6) * 8192 + rr * 128 + ((((d0 & 63) >> 3) ^ rr) << 4);
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {   // tokens 32 pass .. + 31
      uint32_t a0[16], a1[16], b0[16], b1[16];
      tmem_ld16x256b_x4(o1 + 32 * pass, a0);
      tmem_ld16x256b_x4(o1 + (16u << 16) + 32 * pass, a1);
      tmem_ld16x256b_x4(o2 + 32 * pass, b0);
      tmem_ld16x256b_x4(o2 + (16u << 16) + 32 * pass, b1);
      tmem_wait_ld();
      if (pass == 1) {
        tc_fence_before();
        warp_arrive(&bars[B_OFREE + s], lane);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 32 * pass + 8 * j + 2 * (lane & 3);
        const float2 wt = make_float2(p.s_out * w[p.reverse ? 63 - t : t + 1],
                                      p.s_out * w[p.reverse ? 62 - t : t + 2]);
        uint32_t f[4];
#pragma unroll
        for (int mm = 0; mm < 4; ++mm) {
          const uint32_t* x = (mm >> 1) ? a1 : a0;
          const uint32_t* y = (mm >> 1) ? b1 : b0;
          const int e = 4 * j + 2 * (mm & 1);
          const float2 o = fma2(wt, make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])));
          f[mm] = pack2(o.x, o.y);
        }
        stmatrix_x4_trans(st_base + (4 * pass + j) * 1024, f);
      }
    }
    fence_proxy_async_smem();
    group_sync(1, 32 * kOutWarps);
    if (leader) {
      tma_store_3d(to, sm + OFF_O, 0, u.h, ch.t0);
      if (p.V > 64) tma_store_3d(to, sm + OFF_O + 8192, 64, u.h, ch.t0);
      tma_store_commit();
    }
  }
  if (leader) tma_store_wait_all();
  return ok;
}

__global__ void __launch_bounds__(kThreads, 1)
    linear_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                          const LinAttnPass p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  volatile int* flag = reinterpret_cast<volatile int*>(sm + OFF_FLAG);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_TSLOT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = blockIdx.x / p.H;
  Unit u;
  u.h = blockIdx.x % p.H;
  const LaChain c = la_chain(p, n, u.h, tid == 0 && u.h == 0);
  la_zero_rows(p, u.h, c.tail, p.cu_seqlens ? p.T : p.B * p.T, tid, kThreads);
  if (c.skip) return;
  if (c.padding) {
    la_zero_rows(p, u.h, c.bos, c.eos, tid, kThreads);
    return;
  }
  u.bos = c.bos;
  u.eos = c.eos;
  u.nch = (c.eos - c.bos + kChunk - 1) / kChunk;
  u.c0 = 0;
  u.c1 = u.nch;
  u.init = c.init;
  u.fin = c.fin;
  if (u.nch == 0) {   // empty sequence: the state passes through
    if (u.fin)
      for (int e = tid; e < p.K * p.V; e += kThreads) {
        const int kk = e / p.V, vv = e - kk * p.V;
        u.fin[e] = u.init ? u.init[p.initial_t ? vv * p.K + kk : e] : 0.f;
      }
    return;
  }
  const float ld = clamp_log_decay(p.log_decay[u.h]);
  if (tid <= kChunk) reinterpret_cast<float*>(sm + OFF_W)[tid] = decay_pow(ld, (float)tid);
  fill_p_table(p, ld, reinterpret_cast<float*>(sm + OFF_WP), tid);
  if (tid >= 128 && tid < 192 && lane == 0) {
    const int L = warp == 4 ? kChunk : c.eos - c.bos - (u.nch - 1) * kChunk;
    reinterpret_cast<float2*>(sm + OFF_G)[warp - 4] = decay_pow2(ld, L);
  }
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const int count = (i == B_KT || i == B_KT + 1 || i == B_UFREE || i == B_X) ? kStateWarps
                        : i == B_P ? kPWarps
                        : (i == B_OFREE || i == B_OFREE + 1) ? kOutWarps : 1;
      mbar_init(&bars[i], count);
    }
    *flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int terms = p.final_state ? 3 : 2;

  bool ok = true;
  if (warp < kStateWarps) {
    ok = terms == 3 ? state_role<3>(p, u, sm, tbase, bars) : state_role<2>(p, u, sm, tbase, bars);
  } else if (warp < kStateWarps + kOutWarps) {
    ok = out_role(p, u, sm, tbase, bars, &tmO);
  } else if (warp < kMmaWarp) {
    ok = p_role(p, u, sm, tbase, bars);
  } else if (warp == kMmaWarp) {
    if (lane == 0) ok = mma_role(p, u, smem_u32(sm), tbase, bars, terms);
    __syncwarp();
  } else {
    if (lane == 0) load_role(p, u, sm, bars, &tmQ, &tmK, &tmV);
    __syncwarp();
  }
  if (!ok) *flag = 1;
  __syncthreads();
  if (*flag) {   // a wait ran out: give what is still in flight time to land
    if (tid == 0) report(p.dev_status, GDN_DEV_TIMEOUT);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kWaitNs / 8) {
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tbase, TMEM_COLS);
}

}  // namespace

cudaError_t launch_linear_attn_tc(const LinAttnPass& p) {
  const long long blocks = (long long)p.num_seqs * p.H;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int T_total = p.cu_seqlens ? p.T : p.B * p.T;
  CUtensorMap mq, mk, mv, mo;
  memset(&mq, 0, sizeof(mq));
  memset(&mk, 0, sizeof(mk));
  memset(&mv, 0, sizeof(mv));
  memset(&mo, 0, sizeof(mo));
  if (T_total > 0) {   // fp32 rows are stored without a map
    if (!encode_rows_map_bf16(&mq, p.q, p.Hq, T_total, p.K) ||
        !encode_rows_map_bf16(&mk, p.k, p.Hk, T_total, p.K) ||
        !encode_rows_map_bf16(&mv, p.v, p.Hv, T_total, p.V) ||
        (!p.o_f32 && !encode_rows_map_bf16(&mo, p.o, p.H, T_total, p.V)))
      return cudaErrorInvalidValue;
  }
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    err = cudaFuncSetAttribute(linear_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)SMEM_BYTES);
    if (err != cudaSuccess) return err;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  linear_attn_tc_kernel<<<(unsigned)blocks, kThreads, SMEM_BYTES, p.stream>>>(mq, mk, mv, mo, p);
  return cudaGetLastError();
}

}  // namespace gdn
