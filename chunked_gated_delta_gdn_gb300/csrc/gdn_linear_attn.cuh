// gdn_linear_attn.cuh -- device helpers shared by the linear attention kernels.
#pragma once

#include "gdn_common.cuh"
#include "gdn_linear_attn.h"

namespace gdn {
namespace {

// log_decay as the kernels use it: -inf (and anything below -1e4) becomes -1e4, whose powers
// are 1 for exponent 0 and 0 for every other one, without the NaN of -inf * 0.
__device__ __forceinline__ float clamp_log_decay(float x) { return x < -1e4f ? -1e4f : x; }

// gamma^n in fp32, for the weights inside a chunk.
__device__ __forceinline__ float decay_pow(float ld, float n) {
  return exp2f(ld * (float)1.4426950408889634 * n);
}

// gamma^n as an unevaluated fp32 sum hi + lo.  A state is multiplied by its chunk's decay once a
// chunk, so an error of that factor would add up over the sequence (about 1e-7 a chunk and
// head, always of the same sign); the pair keeps it below 2^-48 and leaves the rounding of the
// products, which averages out.
__device__ __forceinline__ float2 decay_pow2(float ld, int n) {
  const double g = exp((double)ld * (double)n);
  const float hi = (float)g;
  return make_float2(hi, isinf(hi) ? 0.f : (float)(g - (double)hi));
}
__device__ __forceinline__ float mul2(float x, float2 g) { return fmaf(x, g.x, x * g.y); }
// x g + y, rounded once but for y's own size.
__device__ __forceinline__ float mul2_add(float x, float2 g, float y) { return fmaf(x, g.x, fmaf(x, g.y, y)); }

// gamma as hi + lo without 64 bits (those take a decode step 4 us of 170): 1 + (gamma - 1), the
// difference to 24 bits, is off by 2^-24 |gamma - 1|, so by some 2^-24 over the whole memory of
// 1 / |gamma - 1| tokens.  Below exp(-0.7) a memory is a few tokens and 24 bits of gamma serve.
__device__ __forceinline__ float2 decay_pair(float ld) {
  if (fabsf(ld) >= 0.7f) return make_float2(expf(ld), 0.f);
  const float d = expm1f(ld), hi = 1.f + d;
  return make_float2(hi, d - (hi - 1.f));
}

// What one (sequence, head) chain works on.
struct LaChain {
  int bos, eos;
  const float* init;    // entry state or NULL
  float* fin;           // exit state or NULL
  bool skip;            // rejected sequence: nothing is written
  bool padding;         // zero rows, no state access
  int tail;             // rows [tail, T_total) belong to no sequence and are zeroed by this chain
};

__device__ __forceinline__ LaChain la_chain(const LinAttnPass& p, int n, int h, bool reporter) {
  LaChain c;
  const int T_total = p.cu_seqlens ? p.T : p.B * p.T;
  c.skip = c.padding = false;
  c.tail = T_total;
  if (p.cu_seqlens) {
    c.bos = p.cu_seqlens[n];
    c.eos = p.cu_seqlens[n + 1];
    if (n == p.num_seqs - 1) c.tail = max(0, min(c.eos, T_total));
  } else {
    c.bos = n * p.T;
    c.eos = c.bos + p.T;
  }
  c.init = nullptr;
  c.fin = nullptr;
  if (c.bos < 0 || c.eos < c.bos || c.eos > T_total || (n == 0 && c.bos != 0)) {
    if (reporter) report(p.dev_status, GDN_DEV_BAD_CU_SEQLENS);
    c.skip = true;
    c.bos = c.eos = 0;
    c.tail = T_total;
    return c;
  }
  int slot = n;
  if (p.state_indices) {
    slot = p.state_indices[n];
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1 && reporter) report(p.dev_status, GDN_DEV_BAD_SLOT);
      c.padding = true;
      return c;
    }
  }
  const size_t off = ((size_t)slot * p.H + h) * (size_t)p.K * p.V;
  if (p.initial) c.init = p.initial + off;
  if (p.final_state) c.fin = p.final_state + off;
  return c;
}

// Zero the output rows [t0, t1) of head h.
__device__ __forceinline__ void la_zero_rows(const LinAttnPass& p, int h, int t0, int t1, int tid,
                                             int nthreads) {
  const size_t n = (size_t)max(0, t1 - t0) * p.V;
  const int dt = p.o_f32 ? GDN_F32 : p.io_dtype;
  for (size_t e = tid; e < n; e += nthreads) {
    const size_t t = e / p.V, d = e - t * p.V;
    store_elem(p.o, (((size_t)t0 + t) * p.H + h) * p.V + d, 0.f, dt);
  }
}

}  // namespace
}  // namespace gdn
