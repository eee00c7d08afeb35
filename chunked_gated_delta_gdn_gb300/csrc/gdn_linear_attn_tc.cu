// gdn_linear_attn_tc.cu -- the chunked pass of linear attention with a decay for each head on
// the tcgen05 tensor cores: bf16 I/O, any accepted head dims (padded to 64 or 128 by the TMA
// loads' zero fill).
//
// One CTA per (sequence, head, segment), chunks of 64 tokens in order.  Per chunk, with X the K x V
// state entering it and w_d = gamma^d (forward in time; the reverse pass mirrors the exponents, see
// gdn_linear_attn.h):
//
//   D    = [Q; K] K^T                      M=128 N=64  (rows 0-63 are Q K^T)
//   P_ij = s_in w_{i-j} / R_i D_ij, j <= i bf16, shared memory; R_i = max(w_{i+1}, 2^-60)
//   O^T  = X^T Q^T + V^T P^T               M=128 (value features) N=64 (tokens)
//   o_i  = s_out R_i O_i
//   U^T  = V~^T K, V~_j = s_in w_{L-1-j} v_j     M=128 N=K
//   X   <- w_L X + U
//
// The read-out of the state and the in-chunk sum share one accumulator by taking the row's decay
// R_i out of both (two accumulators, combined at the end, left no columns for a second output
// buffer, and the MMAs waited for the output warps: 1330 ns a chunk).  Where w_{i+1} is below
// 2^-60 the state's share of the row is below that too, and stands with 2^-60 in its place.
//
// The running state lives in fp32 registers of the state warps (value feature = TMEM lane, key
// feature = column), so a chunk's only serial work on it is one multiply-add per element; the
// tensor cores see it as the bf16 A operand of O1, read from TMEM.  K is the exact input; V~ is
// not representable in bf16, so it is a sum of bf16 terms, formed by packed bf16 multiply-adds
// alone.  With the weight f = f1 + f2 + f3 in bf16 pieces (exact), h = f1 v rounded and
// r = f1 v - h (exact: a product of two 8-bit values has 16 bits):
//   two terms    h, r + f2 v           error 2^-17, far below the bf16 outputs: where only those leave
//   four terms   h, r, a = f2 v rounded, (f2 v - a) + f3 v     error 2^-25, as fp32: where the
//                                                              state leaves too
// (three instructions for two values where scaling and splitting in fp32 took eight, and the
// state warps, which do this, are what a chunk waits for).  The terms go to TMEM as the A operand
// of U, which leaves the shared memory to four stages of Q, K, V in flight (scaled K tiles in
// shared memory left room for two, and a chunk took 4050 cycles: a stage's life is a memory
// latency of 2300 plus its way through the roles).  P and the X operand are rounded to bf16 once,
// like the output itself (P of a sequence of one chunk has a second term, see write_p_rest).
//
// Where chains are too few to fill the GPU, or their last wave would leave most of it idle, they
// (or those of that wave) are cut into segments of whole chunks: a first launch makes every
// segment's own contribution to the state (K, V and U only), and in the second each segment starts
// from X = sum of the contributions before it, each decayed over the tokens in between, and the
// given state.  Several passes (the backward's three) run as one launch.
//
// Measured at K = V = 128 with 152 SMs busy: 1.55 us a chunk where the state leaves, 1.34 where
// only outputs do, 1.0 and 0.65 for a segment's own contribution.  64 KB a chunk and SM are 6.3 and 7.3 TB/s
// (grouped heads find a part of theirs in L2); what bounds it is a chunk's way through the roles,
// and of that the instructions fetched anew for each chunk.  Every piece of a role's loop is
// therefore written for few instructions rather than few steps.
//
// Roles: warps 0-7 state (V~ of a chunk while U of the one before runs, then the update), warps
// 8-11 output, warps 12-13 P, warp 14 issues the MMAs, warp 15 the loads.  (Two issuing warps,
// one for U and O1 and one for D and O2, measured slower: 1.9 us a chunk instead of 1.5.)  They
// meet through mbarriers; every wait is bounded: a timeout sets GDN_DEV_TIMEOUT, every role
// leaves, TMEM is freed.
#include <cuda.h>

#include <atomic>
#include <cstring>

#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_linear_attn.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kStateWarps = 8, kOutWarps = 4, kPWarps = 2;
constexpr int kMmaWarp = 14;   // (warp 15 loads)
constexpr uint64_t kWaitNs = 2000000000ull;

// Shared memory (bytes from a 1024-byte-aligned base).
constexpr int kStages = 4;
constexpr uint32_t kStage = 49152;                 // [k half][Q 64 rows | K 64 rows][128 B], V
constexpr uint32_t kStageV = 32768;                // [v half][64 tokens][128 B]
constexpr uint32_t OFF_P = kStages * kStage;       // [64 i][64 j] bf16
constexpr uint32_t OFF_P_REST = kStage;   // (a sequence of one chunk leaves the second stage empty)
constexpr uint32_t OFF_O = OFF_P + 8192;           // output tile, [v half][64 tokens][128 B]; before its
                                                   // first use the lengths of packed sequences
constexpr uint32_t OFF_W = OFF_O + 16384;          // float[72]: w_0 .. w_64
constexpr uint32_t OFF_F = OFF_W + 288;            // Weights4[2][16]: the weights of V~ in a full and
                                                   // in the partial chunk
constexpr uint32_t OFF_R = OFF_F + 2 * 16 * 24;   // float[2][64]: s_out R of the rows of a full and
                                                  // of the partial chunk
constexpr uint32_t OFF_WP = OFF_R + 512;           // factors of P, see fill_p_table
constexpr uint32_t kWpStride = 136;                // floats of one copy
constexpr uint32_t OFF_G = OFF_WP + 4 * 4 * kWpStride;   // float2[2]: decay of a full / the partial chunk
constexpr uint32_t OFF_SG = OFF_G + 32;            // float2[16]: decay over a whole earlier segment
constexpr uint32_t OFF_BAR = OFF_SG + 8 * kLaMaxSegments;
constexpr uint32_t SMEM_USED = OFF_BAR + 256;
constexpr uint32_t SMEM_BYTES = SMEM_USED + 1024;   // slack for aligning the base
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

// TMEM columns.  O and V~ share the upper half: two terms of V~ have two buffers (128 columns) and
// so has O; of four terms the first two have two buffers, the others one, and O has one.
constexpr uint32_t COL_U = 0, COL_D = 128, COL_X = 192, COL_O = 256, TMEM_COLS = 512;

enum {
  B_FULL = 0,     // [4] stage landed
  B_EMPTY = 4,    // [4] stage free (an output warp, once O is complete)
  B_V = 8,        // V~ written and U of the chunk before read (state warps)
  B_U = 9,        // U complete (commit): V~ read
  B_X = 10,       // X operand written (state warps)
  B_XFREE = 11,   // X^T Q^T complete (commit): the X operand read
  B_D = 12,       // D complete (commit)
  B_P = 13,       // P written, D read (P warps)
  B_O = 14,       // [2] O complete (commit): the chunk's stage has been read
  B_OFREE = 16,   // [2] O read (output warps)
  B_P2 = 18,      // (local contributions: the odd chunks' weights)
  B_COUNT = 19
};
constexpr uint32_t OFF_FLAG = OFF_BAR + 8 * B_COUNT, OFF_TSLOT = OFF_FLAG + 8;

__device__ __forceinline__ uint32_t o_col(int i, int terms) {
  return COL_O + (terms == 2 ? 64u * (i & 1) : 0u);
}
// The columns of the first two terms of V~ of chunk i, and of the other two.
__device__ __forceinline__ uint32_t vt_col(int i, int terms) {
  return COL_O + (terms == 2 ? 128u : 64u) + 64u * (i & 1);
}
constexpr uint32_t COL_VT_LATE = COL_O + 192;

struct Unit {
  int h, bos, eos;       // the sequence
  int nch, c0, c1;       // its chunks, and the range (in order of processing) of this CTA
  const float* init;
  float* fin;            // exit state, when the range ends the sequence
  const float* local;    // this chain's scratch: the entry state, then the contributions of the
                         // segments in order, 128 x 128 floats each
  int before;            // segments before this one
  float* store;          // where this segment's contribution goes (and nothing else is made), or NULL
  float* copy;           // where the entry state is copied to first, or NULL
};

// A bounded wait, short: the roles' loops are fetched anew every chunk (five roles' code does not
// fit the innermost instruction caches), so an instruction costs some five cycles wherever it
// stands.  4 million tries are 40 ms at the very least.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
  uint32_t tries = 0;
  while (!mbar_try_wait(bar, parity))
    if (++tries > (1u << 22)) return false;
  return true;
}
// The same for a whole warp, asleep between the tries (the tries of fourteen warps would take
// issue slots from the work they wait for: 1730 instead of 1560 ns a chunk with the state kept);
// the answer is the same for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  uint32_t tries = 0;
  while (!mbar_try_wait(bar, parity)) {
    __nanosleep(20);
    if (++tries > (1u << 22)) break;
  }
  return __all_sync(0xffffffffu, tries <= (1u << 22));
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
// Packed bf16 arithmetic, each result rounded once.
__device__ __forceinline__ uint32_t bf_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf_mul(uint32_t a, uint32_t b) {   // (-0: keeps a product's sign)
  return bf_fma(a, b, 0x80008000u);
}
__device__ __forceinline__ uint32_t bf_neg(uint32_t a) { return a ^ 0x80008000u; }
// fp32 as a sum of three bf16 values (exact), as bits.
__device__ __forceinline__ void split3(float x, uint32_t (&o)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    o[i] = __bfloat16_as_ushort(h);
    x -= __bfloat162float(h);
  }
}
// The three pieces of the weights of four consecutive tokens, two to a register.
struct Weights4 {
  uint32_t f[3][2];
};
__device__ __forceinline__ Weights4 pack_weights(const float (&x)[4]) {
  Weights4 w;
  uint32_t o[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) split3(x[i], o[i]);
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    w.f[m][0] = o[0][m] | (o[1][m] << 16);
    w.f[m][1] = o[2][m] | (o[3][m] << 16);
  }
  return w;
}
// R of a row whose decay is gamma^e.
__device__ __forceinline__ float row_factor(const float* w, int e) { return fmaxf(w[e], 0x1p-60f); }

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
#pragma unroll 1
  for (int c = u.c0; c < u.c1; ++c) {
    const int i = c - u.c0, s = i & (kStages - 1);
    if (i >= kStages && !wait_bar(&bars[B_EMPTY + s], (uint32_t)(i / kStages - 1) & 1u)) return;
    const int t0 = chunk_at(p, u, c).t0;
    uint8_t* st = sm + s * kStage;
    mbar_arrive_expect_tx(&bars[B_FULL + s], (uint32_t)((u.store ? 1 : 2) * kh + vh) * 8192u);
#pragma unroll 1
    for (int x = 0; x < kh; ++x) {
      tma_load_3d(st + x * 16384 + 8192, tk, &bars[B_FULL + s], 64 * x, hk, t0);
      if (!u.store) tma_load_3d(st + x * 16384, tq, &bars[B_FULL + s], 64 * x, hq, t0);
    }
#pragma unroll 1
    for (int x = 0; x < vh; ++x)
      tma_load_3d(st + kStageV + x * 8192, tv, &bars[B_FULL + s], 64 * x, hv, t0);
  }
}

// ------------------------------------------------------------------ MMAs (one elected thread)
// Descriptors by their low words (address and leading offset); the high word is the same for all.
constexpr uint32_t kDescHi = (uint32_t)((((uint64_t)(1024 >> 4)) << 32 | (1ull << 46) | (2ull << 61)) >> 32);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n"
      " mov.b64 db, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescHi)
      : "memory");
}

__device__ bool mma_role(const LinAttnPass& p, const Unit& u, uint32_t sb, uint32_t tbase,
                         uint64_t* bars, int terms) {
  const int kh = p.K > 64 ? 2 : 1, n = u.c1 - u.c0;
  constexpr uint32_t kS16 = kStage >> 4;
  const uint32_t dQ = desc_lo(sb, 16), dK = desc_lo(sb + 8192, 16), dKm = desc_lo(sb + 8192, 16384),
                 dV = desc_lo(sb + kStageV, 8192), dP = desc_lo(sb + OFF_P, 16);
  const uint32_t idU = kh == 2 ? idesc_bf16(128, 128, false, true) : idesc_bf16(128, 64, false, true);
  constexpr uint32_t idS = idesc_bf16(128, 64, false, false), idO2 = idesc_bf16(128, 64, true, false);
  // chunk -1 has only the next one's D
#pragma unroll 1
  for (int i = -1; i < n; ++i) {
    const uint32_t so = (uint32_t)(i & (kStages - 1)) * kS16, par = (uint32_t)i & 1u;
    if (i >= 0) {   // U^T = V~^T K
      if (!wait_bar(&bars[B_V], par)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int t = 0; t < terms; ++t) {
        const uint32_t a = tbase + (t < 2 ? vt_col(i, terms) + 32 * t : COL_VT_LATE + 32 * (t - 2));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(tbase + COL_U, a + 8 * ks, dKm + so + 128 * ks, idU, (uint32_t)(t | ks));
      }
      mma_commit(&bars[B_U]);
      // O^T = X^T Q^T + V^T P^T
      const uint32_t o = tbase + o_col(i, terms);
      if (!wait_bar(&bars[B_X], par)) return false;
      const int before = terms == 2 ? i - 2 : i - 1;   // the chunk whose output had these columns
      if (before >= 0 && !wait_bar(&bars[B_OFREE + (before & 1)], (uint32_t)(before >> 1) & 1u)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < kh; ++h)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(o, tbase + COL_X + 32 * h + 8 * ks, dQ + so + 1024 * h + 2 * ks, idS, (uint32_t)(h | ks));
      mma_commit(&bars[B_XFREE]);
      if (!wait_bar(&bars[B_P], par)) return false;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma_ss(o, dV + so + 128 * ks, dP + 2 * ks, idO2, 1);
      if (u.nch == 1) {
        const uint32_t dR = desc_lo(sb + OFF_P_REST, 16);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_ss(o, dV + 128 * ks, dR + 2 * ks, idO2, 1);
      }
      mma_commit(&bars[B_O + par]);
    }
    if (i + 1 < n) {   // D = [Q; K] K^T of the next chunk
      const uint32_t s1 = (uint32_t)(i + 1) & (kStages - 1);
      if (!wait_bar(&bars[B_FULL + s1], (uint32_t)((i + 1) / kStages) & 1u)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < kh; ++h)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t off = s1 * kS16 + 1024 * h + 2 * ks;
          mma_ss(tbase + COL_D, dQ + off, dK + off, idS, (uint32_t)(h | ks));
        }
      mma_commit(&bars[B_D]);
    }
  }
  return true;
}

// ------------------------------------------------------------------ a segment's own contribution
// sum_i gamma^(64 (n - 1 - i)) V~_i^T K_i over its n chunks (the last one to be processed is full):
// the decay goes into the weights of V~, which the P warps make for each chunk, so that nothing runs
// in series but the MMAs.  Where the state leaves (four terms) the sum stays in TMEM for two chunks
// and is then added to fp32 registers while the next two fill a second accumulator: the MMAs'
// accumulation does not round to nearest, and over a whole segment of 32 chunks the state's error
// grew to 2e-6 (eight at a time 1.2e-6 to 1.7e-6, four 1.0e-6, two 7e-7; 34, 37, 38, 39 us for
// 8192 tokens of 32 heads).  Where only bf16 outputs do, it stays there to the segment's end.  V~
// and the weights have two buffers each, and everything that says so two barriers, for even and
// odd chunks (no wait falls two phases behind).
__host__ __device__ constexpr int local_run(int terms) { return terms == 4 ? 2 : 1 << 24; }
__device__ __forceinline__ uint32_t local_sum(int i, int run) { return COL_U + 128u * ((i / run) & 1); }
__device__ __forceinline__ uint64_t* local_v(uint64_t* bars, int i) { return &bars[(i & 1) ? B_X : B_V]; }
__device__ __forceinline__ uint64_t* local_w(uint64_t* bars, int i) { return &bars[(i & 1) ? B_P2 : B_P]; }
__device__ __forceinline__ uint32_t local_col(int i) { return COL_O + 128u * (i & 1); }

__device__ bool local_weights_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint64_t* bars) {
  const int lane = threadIdx.x & 31, e = 8 * ((threadIdx.x >> 5) - kStateWarps - kOutWarps) + lane;
  const double lg = (double)clamp_log_decay(p.log_decay[u.h]) * 1.4426950408889634;
  const float hi = (float)lg, lo = (float)(lg - (double)hi);
  const float* w = reinterpret_cast<const float*>(sm + OFF_W);
  const int n = u.c1 - u.c0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    if (i >= 2 && !wait_warp(local_v(bars, i), (uint32_t)((i - 2) >> 1) & 1u)) return false;
    const int L = chunk_at(p, u, u.c0 + i).L, after = kChunk * (n - 1 - i);
    if (lane < 8) {
      // gamma^after = 2^(a + b), a rounded and b the rest
      const float a = hi * (float)after, b = fmaf(hi, (float)after, -a) + lo * (float)after;
      const float g = exp2f(a), f = p.s_in * fmaf(g, b * 0.69314718f, g);
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = f * w[p.reverse ? 4 * e + j + 1 : max(L - 1 - 4 * e - j, 0)];
      reinterpret_cast<Weights4*>(sm + OFF_F)[16 * (i & 1) + e] = pack_weights(x);
    }
    warp_arrive(local_w(bars, i), lane);
  }
  return true;
}

__device__ bool local_mma_role(const LinAttnPass& p, const Unit& u, uint32_t sb, uint32_t tbase, uint64_t* bars,
                               int terms) {
  const int n = u.c1 - u.c0, run = local_run(terms);
  const uint32_t dKm = desc_lo(sb + 8192, 16384), id = idesc_bf16(128, p.K > 64 ? 128 : 64, false, true);
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int s = i & (kStages - 1);
    if (!wait_bar(local_v(bars, i), (uint32_t)(i >> 1) & 1u)) return false;
    if (!wait_bar(&bars[B_FULL + s], (uint32_t)(i / kStages) & 1u)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int t = 0; t < terms; ++t)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ts(tbase + local_sum(i, run), tbase + local_col(i) + 32 * t + 8 * ks, dKm + s * (kStage >> 4) + 128 * ks,
               id, (uint32_t)((i % run) | t | ks));
    if (i + kStages < n) mma_commit(&bars[B_EMPTY + s]);
    mma_commit(&bars[B_O + (i & 1)]);
  }
  return true;
}

// ------------------------------------------------------------------ P (warps 12, 13)
// The factor s_in w_{i-j} of P_ij depends on j - i alone: f[x] for x = j - i + 63 in 0 .. 126, zero
// where the mask is.  Row i reads f[63 - i ..], four at a time: four copies shifted by one float each keep
// those reads 16-byte aligned whatever i is, and their stride of 8 banks keeps them apart.
__device__ __forceinline__ void fill_p_table(const LinAttnPass& p, float ld, float* wp, int tid) {
  for (int e = tid; e < 4 * (int)kWpStride; e += kThreads) {
    const int copy = e / (int)kWpStride, x = e - copy * (int)kWpStride + copy;   // copy[y] = f[y + copy]
    const int dist = p.reverse ? x - 63 : 63 - x;
    wp[e] = (dist >= 0 && dist < kChunk) ? p.s_in * decay_pow(ld, (float)dist) : 0.f;
  }
}

// Row `row` of P from column L on: zero, whatever the rows past the chunk's end held.
__device__ __noinline__ void clear_columns(uint8_t* tile, int row, int L) {
#pragma unroll 1
  for (int j = L; j < kChunk; ++j)
    *reinterpret_cast<uint16_t*>(tile + sw128_offset(row, j)) = (uint16_t)0;
}

// What the rounding of P left, as a second tile: for a sequence of one chunk, whose outputs have as
// few entries of P as factors as they have tokens before them (one token: one), so that its error
// would not average out.  (A second term for every chunk took 9 to 17% more time.)
__device__ __noinline__ void write_p_rest(uint8_t* sm, uint32_t d, int row, const float4* f4, float inv) {
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    float x[32];
    tmem_ld32(d + 32 * half, x);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const float4 f = f4[8 * half + g];
      const float t[4] = {f.x * (inv * x[4 * g]), f.y * (inv * x[4 * g + 1]), f.z * (inv * x[4 * g + 2]),
                          f.w * (inv * x[4 * g + 3])};
      uint2 q;
      float rest[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) rest[k] = t[k] - __bfloat162float(__float2bfloat16_rn(t[k]));
      q.x = pack2(rest[0], rest[1]);
      q.y = pack2(rest[2], rest[3]);
      *reinterpret_cast<uint2*>(sm + OFF_P_REST + sw128_offset(row, 32 * half + 4 * g)) = q;
    }
  }
}

__device__ bool p_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase,
                       uint64_t* bars) {
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 1, row = 32 * wq + lane;
  const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
  const float* w = reinterpret_cast<const float*>(sm + OFF_W);
  const int shift = (63 - row) & 3;
  const float4* f4 = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm + OFF_WP) +
                                                     shift * kWpStride + (63 - row - shift));
#pragma unroll 1
  for (int c = u.c0; c < u.c1; ++c) {
    const int i = c - u.c0;
    const int L = chunk_at(p, u, c).L;
    if (!wait_warp(&bars[B_D], (uint32_t)i & 1u)) return false;
    // (D of a chunk is issued after V^T P^T of the one before: P has been read when it is complete)
    tc_fence_after();
    const float inv = 1.f / row_factor(w, p.reverse ? max(L - 1 - row, 0) : row + 1);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      float x[32];
      tmem_ld32(tbase + lane_off + COL_D + 32 * half, x);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 a = f4[8 * half + 2 * g], b = f4[8 * half + 2 * g + 1];
        uint4 q;
        float2 t = mul2v(make_float2(a.x, a.y), make_float2(inv * x[8 * g], inv * x[8 * g + 1]));
        q.x = pack2(t.x, t.y);
        t = mul2v(make_float2(a.z, a.w), make_float2(inv * x[8 * g + 2], inv * x[8 * g + 3]));
        q.y = pack2(t.x, t.y);
        t = mul2v(make_float2(b.x, b.y), make_float2(inv * x[8 * g + 4], inv * x[8 * g + 5]));
        q.z = pack2(t.x, t.y);
        t = mul2v(make_float2(b.z, b.w), make_float2(inv * x[8 * g + 6], inv * x[8 * g + 7]));
        q.w = pack2(t.x, t.y);
        *reinterpret_cast<uint4*>(sm + OFF_P + sw128_offset(row, 32 * half + 8 * g)) = q;
      }
    }
    if (L < kChunk) clear_columns(sm + OFF_P, row, L);
    if (u.nch == 1) {
      write_p_rest(sm, tbase + lane_off + COL_D, row, f4, inv);
      clear_columns(sm + OFF_P_REST, row, L);
    }
    tc_fence_before();
    fence_proxy_async_smem();
    warp_arrive(&bars[B_P], lane);
  }
  return true;
}

// ------------------------------------------------------------------ state (warps 0-7)
// Rows L .. 63 of a stage's K and V become zero: they belong to another sequence, or to none, and
// a NaN there must not meet the zero weights.  Each state warp clears the 16 V columns that it
// reads itself and every eighth row of K.
__device__ __noinline__ void clear_rows(uint8_t* st, int L, int vt0, int warp, int lane) {
  uint8_t* v = st + kStageV + (vt0 >> 6) * 8192;
  for (int e = lane; e < 128; e += 32) {
    const int t = e >> 1;
    if (t >= L)
      *reinterpret_cast<uint4*>(v + t * 128 + (((((vt0 & 63) >> 3) + (e & 1)) ^ (t & 7)) << 4)) =
          make_uint4(0u, 0u, 0u, 0u);
  }
  for (int e = lane; e < 128; e += 32) {
    const int t = 8 * (e >> 4) + warp;
    if (t >= L)
      *reinterpret_cast<uint4*>(st + 8192 + ((e >> 3) & 1) * 16384 + t * 128 + (e & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// This warp's 16 value features of V~^T as TMEM fragments.  Fragment register 4 g + r of thread t
// holds features t/4 (r < 2) or t/4 + 8 and TMEM column 8 g + 2 (t%4) + (r & 1), that is tokens
// 16 g + 4 (t%4) + 2 (r & 1) and the next; ldmatrix .trans delivers exactly that when its row
// addresses name the tokens 0, 1, 4, 5, 8, 9, 12, 13 (r even) or 2, 3, 6, .. (odd).
template <int kTerms>
__device__ __forceinline__ void make_vt(const uint8_t* sm, uint32_t v_tile, int d0,
                                        int table, int lane, uint32_t dst, uint32_t (&late)[2][16]) {
  const Weights4* fw = reinterpret_cast<const Weights4*>(sm + OFF_F) + 16 * table + (lane & 3);
  const int r = lane >> 3, j = lane & 7;              // matrix (register) this lane addresses, row
  const int tok0 = 4 * (j >> 1) + 2 * (r & 1) + (j & 1), d = d0 + 8 * (r >> 1);
  const uint32_t tile = v_tile + (d >> 6) * 8192 + (uint32_t)tok0 * 128u + ((((d & 63) >> 3) ^ (tok0 & 7)) << 4);
#pragma unroll(kTerms == 2 ? 2 : 4)
  for (int g = 0; g < 4; ++g) {
    uint32_t x[4], o[2][4];
    ldmatrix_x4_trans(tile + g * 2048, x);
    const Weights4 f = fw[4 * g];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t f1 = f.f[0][m & 1], f2 = f.f[1][m & 1], f3 = f.f[2][m & 1];
      const uint32_t h = bf_mul(x[m], f1), rest = bf_fma(x[m], f1, bf_neg(h));
      o[0][m] = h;
      if (kTerms == 2) {
        o[1][m] = bf_fma(x[m], f2, rest);
      } else {
        const uint32_t a = bf_mul(x[m], f2);
        o[1][m] = rest;
        late[0][4 * g + m] = a;
        late[1][4 * g + m] = bf_fma(x[m], f3, bf_fma(x[m], f2, bf_neg(a)));
      }
    }
    tmem_st16x256b_x1(dst + 8 * g, o[0]);
    tmem_st16x256b_x1(dst + 32 + 8 * g, o[1]);
  }
}

// V~ of a segment's chunks, for its own contribution, which is left in X.
template <int kTerms>
__device__ bool local_state_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase, uint64_t* bars,
                                 float2 (&X)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vt0 = 32 * (warp & 3) + 16 * (warp >> 2);
  const uint32_t vt_off = (uint32_t)vt0 << 16, sb = smem_u32(sm);
  const int n = u.c1 - u.c0, dk0 = 64 * (warp >> 2);
  constexpr int kRun = local_run(kTerms);
  auto add_run = [&](int i) {   // the run that ended with chunk i
    if (dk0 >= p.K) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x[32];
      tmem_ld32(tbase + ((uint32_t)(32 * (warp & 3)) << 16) + local_sum(i, kRun) + dk0 + 32 * half, x);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float2& a = X[16 * half + j];
        a = make_float2(a.x + x[2 * j], a.y + x[2 * j + 1]);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < 32; ++j) X[j] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int s = i & (kStages - 1), L = chunk_at(p, u, u.c0 + i).L;
    if (!wait_warp(&bars[B_FULL + s], (uint32_t)(i / kStages) & 1u)) return false;
    if (L < kChunk) clear_rows(sm + s * kStage, L, vt0, warp, lane);
    if (i >= 2 && !wait_warp(&bars[B_O + (i & 1)], (uint32_t)((i - 2) >> 1) & 1u)) return false;
    if (!wait_warp(local_w(bars, i), (uint32_t)(i >> 1) & 1u)) return false;
    tc_fence_after();
    if (vt0 < p.V) {
      uint32_t late[2][16];
      const uint32_t dst = tbase + vt_off + local_col(i);
      make_vt<kTerms>(sm, sb + s * kStage + kStageV, vt0, i & 1, lane, dst, late);
      if (kTerms == 4) {
        tmem_st16x256b_x4(dst + 64, late[0]);
        tmem_st16x256b_x4(dst + 96, late[1]);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    warp_arrive(local_v(bars, i), lane);
    // (chunk i - 2 is complete; the MMAs come back to its accumulator after another run's V~)
    if (kTerms == 4 && i >= 2 && (i - 2) % kRun == kRun - 1) add_run(i - 2);
  }
  if (!wait_warp(&bars[B_O + ((n - 1) & 1)], (uint32_t)((n - 1) >> 1) & 1u)) return false;
  tc_fence_after();
  if (kTerms == 4 && n >= 2 && (n - 2) % kRun == kRun - 1) add_run(n - 2);
  add_run(n - 1);
  return true;
}

template <int kTerms>
__device__ bool state_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase,
                           uint64_t* bars) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int dv = 32 * (warp & 3) + lane, dk0 = 64 * (warp >> 2);   // this thread's 64 state elements
  const int vt0 = 32 * (warp & 3) + 16 * (warp >> 2);              // this warp's 16 rows of V~^T
  const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16, vt_off = (uint32_t)vt0 << 16;
  const uint32_t sb = smem_u32(sm);
  const int n = u.c1 - u.c0;
  const bool mine = dk0 < p.K, mine_v = vt0 < p.V;   // (features past the head dim: nothing to do)
  const float2* g = reinterpret_cast<const float2*>(sm + OFF_G);
  float2 X[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) X[j] = make_float2(0.f, 0.f);
  if (u.init && dv < p.V) {
    const size_t step = p.initial_t ? 1 : p.V;
    const float* src = u.init + (p.initial_t ? (size_t)dv * p.K + dk0 : (size_t)dk0 * p.V + dv);
#pragma unroll
    for (int j = 0; j < 32; ++j) {   // (K is even)
      if (dk0 + 2 * j < p.K) X[j] = make_float2(src[0], src[step]);
      src += 2 * step;
    }
  }
  constexpr int kStep = 32 * kStateWarps;       // a slot holds the threads' elements side by side
  auto slot = [&](const float* base, int r) {   // this thread's, 4 every kStep, in slot r
    return reinterpret_cast<float4*>(const_cast<float*>(base) + (size_t)r * 16384) + tid;
  };
  auto put_slot = [&](float4* dst) {
#pragma unroll
    for (int j = 0; j < 16; ++j) dst[j * kStep] = make_float4(X[2 * j].x, X[2 * j].y, X[2 * j + 1].x, X[2 * j + 1].y);
  };
  if (u.copy) put_slot(slot(u.copy, 0));
  if (u.store) {
    if (!local_state_role<kTerms>(p, u, sm, tbase, bars, X)) return false;
    put_slot(slot(u.store, 0));
    return true;
  }
  if (u.local) {   // X <- X (hi + lo) + slot r
    const float2* sg = reinterpret_cast<const float2*>(sm + OFF_SG);
#pragma unroll 1
    for (int r = 0; r <= u.before; ++r) {
      const float4* src = slot(u.local, r);
      const float2 gr = r > 0 ? sg[r - 1] : make_float2(0.f, 0.f);
      const float2 hi = make_float2(gr.x, gr.x), lo = make_float2(gr.y, gr.y);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 x = __ldcg(src + j * kStep);
        X[2 * j] = fma2(X[2 * j], hi, fma2(X[2 * j], lo, make_float2(x.x, x.y)));
        X[2 * j + 1] = fma2(X[2 * j + 1], hi, fma2(X[2 * j + 1], lo, make_float2(x.z, x.w)));
      }
    }
  }
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
  // X <- X (hi + lo) + U of chunk i
  auto update = [&](int i) {
    if (mine) {
      const float2 gl = g[chunk_at(p, u, u.c0 + i).L < kChunk];
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
  };
  // V~ of chunk i is made while U of chunk i - 1 runs; the terms that have no second buffer wait
  // for its end in registers.
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int s = i & (kStages - 1), L = chunk_at(p, u, u.c0 + i).L;
    uint32_t late[2][16];
    if (!wait_warp(&bars[B_FULL + s], (uint32_t)(i / kStages) & 1u)) return false;
    if (L < kChunk) clear_rows(sm + s * kStage, L, vt0, warp, lane);
    if (mine_v)
      make_vt<kTerms>(sm, sb + s * kStage + kStageV, vt0, L < kChunk, lane,
                      tbase + vt_off + vt_col(i, kTerms), late);
    if (i > 0) {
      if (!wait_warp(&bars[B_U], (uint32_t)(i - 1) & 1u)) return false;
      tc_fence_after();
    }
    if (kTerms == 4 && mine_v) {
      tmem_st16x256b_x4(tbase + vt_off + COL_VT_LATE, late[0]);
      tmem_st16x256b_x4(tbase + vt_off + COL_VT_LATE + 32, late[1]);
    }
    if (i > 0) update(i - 1);
    tmem_wait_st();
    tc_fence_before();
    warp_arrive(&bars[B_V], lane);
    if (i > 0) {
      if (!wait_warp(&bars[B_XFREE], (uint32_t)(i - 1) & 1u)) return false;
      tc_fence_after();
      put_x();
    }
  }
  if (u.fin) {
    if (!wait_warp(&bars[B_U], (uint32_t)(n - 1) & 1u)) return false;
    tc_fence_after();
    update(n - 1);
    float* dst = u.fin + (size_t)dk0 * p.V + dv;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (dv < p.V && dk0 + 2 * j < p.K) {
        dst[0] = X[j].x;
        dst[p.V] = X[j].y;
      }
      dst += 2 * p.V;
    }
  }
  return true;
}

// ------------------------------------------------------------------ output (warps 8-11)
// The first L rows of the staged tile (a partial chunk; the tile's TMA store would write all 64).
__device__ __noinline__ void store_rows(const LinAttnPass& p, const uint8_t* tile, const ChunkAt& ch, int h,
                                        int tid) {
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + ((size_t)ch.t0 * p.H + h) * p.V;
  const int per = p.V / 8;   // 16-byte pieces a row
#pragma unroll 1
  for (int e = tid; e < ch.L * per; e += 32 * kOutWarps) {
    const int t = e / per, d = e - t * per;
    *reinterpret_cast<uint4*>(dst + (size_t)t * p.H * p.V + 8 * d) =
        *reinterpret_cast<const uint4*>(tile + (d >> 3) * 8192 + t * 128 + (((d & 7) ^ (t & 7)) << 4));
  }
}

// A partial chunk's rows in fp32, from the accumulator.
__device__ __noinline__ void store_rows_f32(const LinAttnPass& p, const ChunkAt& ch, const float* factor,
                                            uint32_t o, int h, int dv) {
  float* dst = reinterpret_cast<float*>(p.o) + ((size_t)ch.t0 * p.H + h) * p.V + dv;
#pragma unroll 1
  for (int t0 = 0; t0 < ch.L; t0 += 32) {
    float x[32];
    tmem_ld32(o + t0, x);
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (t0 + t < ch.L && dv < p.V) dst[(size_t)(t0 + t) * p.H * p.V] = factor[t0 + t] * x[t];
  }
}

__device__ bool out_role(const LinAttnPass& p, const Unit& u, uint8_t* sm, uint32_t tbase,
                         uint64_t* bars, int terms, const CUtensorMap* to) {
  const int tid = threadIdx.x - 32 * kStateWarps, lane = tid & 31, wq = tid >> 5;
  const uint32_t lane_off = (uint32_t)(32 * wq) << 16, sbase = smem_u32(sm);
  const bool leader = tid == 0;
  bool ok = true;
#pragma unroll 1
  for (int c = u.c0; c < u.c1; ++c) {
    const int i = c - u.c0;
    const ChunkAt ch = chunk_at(p, u, c);
    const uint32_t par = (uint32_t)i & 1u, o = tbase + lane_off + o_col(i, terms);
    if (leader) tma_store_wait_read();   // the previous tile has left the staging
    ok = wait_warp(&bars[B_O + par], (uint32_t)(i >> 1) & 1u);
    if (group_sync_or(1, 32 * kOutWarps, !ok)) {
      ok = false;
      break;
    }
    tc_fence_after();
    if (leader) mbar_arrive(&bars[B_EMPTY + (i & (kStages - 1))]);   // (a chunk's last MMAs)
    if (p.o_f32 && ch.L < kChunk) {
      store_rows_f32(p, ch, reinterpret_cast<const float*>(sm + OFF_R) + kChunk, o, u.h, 32 * wq + lane);
      tc_fence_before();
      warp_arrive(&bars[B_OFREE + par], lane);
      continue;
    }
    if (p.o_f32) {
      // fp32 rows: this lane's value feature of each token, 128 bytes a warp and store
      const int dv = 32 * wq + lane;
      float* dst = reinterpret_cast<float*>(p.o) + ((size_t)ch.t0 * p.H + u.h) * p.V + dv;
      const size_t step = (size_t)p.H * p.V;
      const float4* r4 = reinterpret_cast<const float4*>(sm + OFF_R);
#pragma unroll 1
      for (int t0 = 0; t0 < kChunk; t0 += 32) {
        float x[32];
        tmem_ld32(o + t0, x);
        if (t0 > 0) {
          tc_fence_before();
          warp_arrive(&bars[B_OFREE + par], lane);
        }
        if (dv < p.V) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 r = r4[(t0 >> 2) + j];
            dst[0] = r.x * x[4 * j];
            dst[step] = r.y * x[4 * j + 1];
            dst[2 * step] = r.z * x[4 * j + 2];
            dst[3 * step] = r.w * x[4 * j + 3];
            dst += 4 * step;
          }
        }
        __syncwarp();
      }
      continue;
    }
    // the factors s_out R of this lane's tokens 2 (lane % 4) and the next
    const float2* rf = reinterpret_cast<const float2*>(sm + OFF_R) + (ch.L < kChunk ? 32 : 0) + (lane & 3);
    // 16x256b loads give each thread value features (t/4, t/4 + 8) x tokens (2 (t%4), + 1): the
    // fragment that stmatrix .trans writes as 16-byte rows (8 features of one token) of the
    // 128-byte-swizzled tile.  Lane l addresses feature block l / 8, token l % 8.
    const int mblk = lane >> 3, rr = lane & 7, d0 = 32 * wq + 8 * mblk;
    const uint32_t st_base = sbase + OFF_O + (d0 >> 6) * 8192 + rr * 128 + ((((d0 & 63) >> 3) ^ rr) << 4);
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {   // tokens 32 pass .. + 31
      uint32_t a0[16], a1[16];
      tmem_ld16x256b_x4(o + 32 * pass, a0);
      tmem_ld16x256b_x4(o + (16u << 16) + 32 * pass, a1);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 wt = rf[16 * pass + 4 * j];
        uint32_t f[4];
#pragma unroll
        for (int mm = 0; mm < 4; ++mm) {
          const uint32_t* x = (mm >> 1) ? a1 : a0;
          const int e = 4 * j + 2 * (mm & 1);
          const float2 y = mul2v(wt, make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
          f[mm] = pack2(y.x, y.y);
        }
        stmatrix_x4_trans(st_base + (4 * pass + j) * 1024, f);
      }
    }
    tc_fence_before();
    warp_arrive(&bars[B_OFREE + par], lane);
    if (ch.L < kChunk) {
      group_sync(1, 32 * kOutWarps);
      store_rows(p, sm + OFF_O, ch, u.h, tid);
      group_sync(1, 32 * kOutWarps);   // (the tile is free again)
      continue;
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

// The sequence that stands at `place` by length, longest first (equals by number): CTAs start in
// order, and a long chain that starts among the last keeps the others waiting.  `len` must be shared
// memory that no load lands in: nothing orders these ordinary accesses before the asynchronous writes
// of the first chunk.
constexpr int kMaxSorted = 128;
static_assert(OFF_O >= kStages * kStage && 4 * (kMaxSorted + 1) <= 16384, "lengths in the output tile");
__device__ __forceinline__ int sequence_by_length(const int32_t* cu, int n, int place, int* len) {
  const int t = threadIdx.x;
  if (t < n) len[t] = cu[t + 1] - cu[t];
  __syncthreads();
  if (t < n) {
    const int mine = len[t];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += len[j] > mine || (len[j] == mine && j < t);
    if (rank == place) len[kMaxSorted] = t;
  }
  __syncthreads();
  return len[kMaxSorted];
}

struct LaLaunch {
  CUtensorMap map[kLaMaxPasses][4];   // q, k, v, o
  LinAttnPass pass[kLaMaxPasses];
  int longest_first;
  int whole;           // this launch's CTAs for chains that are not cut, before the others
  int first_cut, cut;  // the chains that are cut, and in how many
  int segs;
  int local_only;      // the first launch of a segmented run
  float* local;        // [chain that is cut][segs][128][128]
};

__global__ void __launch_bounds__(kThreads, 1) linear_attn_tc_kernel(const __grid_constant__ LaLaunch a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  volatile int* flag = reinterpret_cast<volatile int*>(sm + OFF_FLAG);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_TSLOT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (a.local_only) next_may_start();   // (the second launch's CTAs, as SMs come free)
  Unit u;
  // chains by heads (those that share a row of q or k run side by side), sequences, passes
  int e = blockIdx.x, seg = 0, segs = 1, chain_cut = 0;
  bool local_only = false;
  if (e >= a.whole) {
    e -= a.whole;
    seg = e / a.cut;
    chain_cut = e - seg * a.cut;
    e = a.first_cut + chain_cut;
    segs = a.segs;
    local_only = a.local_only;
  }
  u.h = e % a.pass[0].H;
  e /= a.pass[0].H;
  int n = e % a.pass[0].num_seqs;
  e /= a.pass[0].num_seqs;
  if (a.longest_first)
    n = sequence_by_length(a.pass[0].cu_seqlens, a.pass[0].num_seqs, n, reinterpret_cast<int*>(sm + OFF_O));
  const int pi = e;
  const LinAttnPass p = a.pass[pi];
  const LaChain c = la_chain(p, n, u.h, tid == 0 && u.h == 0 && seg == 0);
  if (seg == 0 && !local_only) {
    la_zero_rows(p, u.h, c.tail, p.cu_seqlens ? p.T : p.B * p.T, tid, kThreads);
    if (c.padding) la_zero_rows(p, u.h, c.bos, c.eos, tid, kThreads);
  }
  if (c.skip || c.padding) {
    wait_for_previous();
    return;
  }
  u.bos = c.bos;
  u.eos = c.eos;
  u.nch = (c.eos - c.bos + kChunk - 1) / kChunk;
  const int per = max((u.nch + segs - 1) / segs, kLaMinSegmentChunks);
  u.c0 = min(seg * per, u.nch);
  u.c1 = min(u.c0 + per, u.nch);
  const bool whole = seg == 0 && u.c1 == u.nch;   // (no other CTA works on this chain)
  if (local_only && u.c1 == u.nch) return;       // (its contribution is nobody's entry state)
  // The entry state comes from the scratch where another CTA of the second launch may be writing
  // the exit state to the same place.
  float* local = whole ? nullptr : a.local + (size_t)chain_cut * segs * 16384;
  u.init = whole || (local_only && seg == 0) ? c.init : nullptr;
  u.fin = local_only || u.c1 < u.nch ? nullptr : c.fin;
  u.before = seg;
  u.local = local;
  u.store = local_only ? local + (size_t)(seg + 1) * 16384 : nullptr;
  u.copy = local_only && seg == 0 ? local : nullptr;
  if (u.c0 == u.c1) {
    wait_for_previous();
    if (whole && u.fin)   // empty sequence: the state passes through
      for (int x = tid; x < p.K * p.V; x += kThreads) {
        const int kk = x / p.V, vv = x - kk * p.V;
        u.fin[x] = u.init ? u.init[p.initial_t ? vv * p.K + kk : x] : 0.f;
      }
    return;
  }
  const float ld = clamp_log_decay(p.log_decay[u.h]);
  if (tid <= kChunk) reinterpret_cast<float*>(sm + OFF_W)[tid] = decay_pow(ld, (float)tid);
  if (tid < 2 * kChunk) {
    const int t = tid & (kChunk - 1), L = tid < kChunk ? kChunk : c.eos - c.bos - (u.nch - 1) * kChunk;
    reinterpret_cast<float*>(sm + OFF_R)[tid] =
        p.s_out * fmaxf(decay_pow(ld, p.reverse ? (float)max(L - 1 - t, 0) : (float)(t + 1)), 0x1p-60f);
  }
  if (tid >= 64 && tid < 96) {   // (rows past the partial chunk's end are clear, whatever their weight)
    const int t = 4 * (tid & 15), L = tid < 80 ? kChunk : c.eos - c.bos - (u.nch - 1) * kChunk;
    float x[4];
    for (int i = 0; i < 4; ++i)
      x[i] = p.s_in * decay_pow(ld, p.reverse ? (float)(t + i + 1) : (float)max(L - 1 - t - i, 0));
    reinterpret_cast<Weights4*>(sm + OFF_F)[tid - 64] = pack_weights(x);
  }
  fill_p_table(p, ld, reinterpret_cast<float*>(sm + OFF_WP), tid);
  if (tid >= 128 && tid < 192 && lane == 0) {
    const int L = warp == 4 ? kChunk : c.eos - c.bos - (u.nch - 1) * kChunk;
    reinterpret_cast<float2*>(sm + OFF_G)[warp - 4] = decay_pow2(ld, L);
  }
  if (!local_only && tid >= 256 && tid < 256 + u.before) {
    // (backwards the first segment holds the partial chunk)
    const int r = tid - 256, last = c.eos - c.bos - (u.nch - 1) * kChunk;
    reinterpret_cast<float2*>(sm + OFF_SG)[r] =
        decay_pow2(ld, per * kChunk - (p.reverse && r == 0 ? kChunk - last : 0));
  }
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const int count = (i == B_V || i == B_X) ? kStateWarps
                        : i == B_P || i == B_P2 ? kPWarps : (i == B_OFREE || i == B_OFREE + 1) ? kOutWarps : 1;
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
  wait_for_previous();
  // a segment's contribution may end in a final state; the passes from it to there add nothing
  const int terms = u.fin || (u.store && p.final_state) ? 4 : 2;

  bool ok = true;
  if (warp < kStateWarps) {
    ok = terms == 4 ? state_role<4>(p, u, sm, tbase, bars) : state_role<2>(p, u, sm, tbase, bars);
  } else if (warp < kStateWarps + kOutWarps) {
    if (!u.store) ok = out_role(p, u, sm, tbase, bars, terms, &a.map[pi][3]);
  } else if (warp < kMmaWarp) {
    ok = u.store ? local_weights_role(p, u, sm, bars) : p_role(p, u, sm, tbase, bars);
  } else if (warp == kMmaWarp) {
    if (elect_one())
      ok = u.store ? local_mma_role(p, u, smem_u32(sm), tbase, bars, terms)
                   : mma_role(p, u, smem_u32(sm), tbase, bars, terms);
    __syncwarp();
  } else {
    if (lane == 0) load_role(p, u, sm, bars, &a.map[pi][0], &a.map[pi][1], &a.map[pi][2]);
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

cudaError_t launch_linear_attn_tc(const LinAttnPass* passes, int num_passes, LaPlan plan, float* local) {
  const LinAttnPass& p0 = passes[0];
  const long long chains = (long long)num_passes * p0.num_seqs * p0.H;
  if (chains <= 0) return cudaSuccess;
  const long long cut = chains - plan.whole;
  const int segs = plan.segs;
  if (num_passes > kLaMaxPasses || segs < 1 || segs > kLaMaxSegments || cut < 0 || (segs == 1 && cut > 0) ||
      plan.whole + cut * segs > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  const int T_total = p0.cu_seqlens ? p0.T : p0.B * p0.T;
  LaLaunch a;
  memset(&a, 0, sizeof(a));
  a.whole = (int)plan.whole;
  a.first_cut = (int)plan.whole;
  a.cut = (int)cut;
  a.segs = segs;
  a.local = local;
  // (with up to a hundred sequences finding one's place takes a CTA less than a microsecond)
  a.longest_first = p0.cu_seqlens && p0.num_seqs > 1 && p0.num_seqs <= kMaxSorted;
  for (int i = 0; i < num_passes; ++i) {
    const LinAttnPass& p = a.pass[i] = passes[i];
    if (T_total > 0 &&   // (fp32 rows are stored without a map)
        (!encode_rows_map_bf16(&a.map[i][0], p.q, p.Hq, T_total, p.K) ||
         !encode_rows_map_bf16(&a.map[i][1], p.k, p.Hk, T_total, p.K) ||
         !encode_rows_map_bf16(&a.map[i][2], p.v, p.Hv, T_total, p.V) ||
         (!p.o_f32 && !encode_rows_map_bf16(&a.map[i][3], p.o, p.H, T_total, p.V))))
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
  if (cut > 0) {
    a.local_only = 1;
    linear_attn_tc_kernel<<<(unsigned)(plan.whole + cut * (segs - 1)), kThreads, SMEM_BYTES, p0.stream>>>(a);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    a.local_only = 0;
    a.whole = 0;
    return launch_behind(linear_attn_tc_kernel, (unsigned)(cut * segs), kThreads, SMEM_BYTES, p0.stream, a);
  }
  linear_attn_tc_kernel<<<(unsigned)plan.whole, kThreads, SMEM_BYTES, p0.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
