// gdn_linear_attn.cu -- linear attention with a decay for each head on the CUDA cores: the
// chunked pass for any accepted head dims and type, the single-token decode step, and the sum
// over the value heads that share a query/key head.
//
// A chunk of L <= 64 tokens, with X the K x V state entering it and w_d = gamma^d:
//   P_ij  = s_in w_{i-j} (q_i . k_j)   for j <= i, else 0           (reverse: w_{j-i}, j >= i)
//   o_i   = s_out (w_{i+1} X^T q_i + sum_j P_ij v_j)                (reverse: w_{L-1-i})
//   X    <- w_L X + sum_j s_in w_{L-1-j} k_j v_j^T                  (reverse: w_{j+1})
#include <algorithm>
#include <atomic>

#include "gdn_launch.cuh"
#include "gdn_linear_attn.cuh"

namespace gdn {
namespace {

constexpr int kLaThreads = 256;

// 4 consecutive elements as floats.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&lo);
  u.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p) = u;
}

__device__ __forceinline__ void fma4(float4& a, float s, const float4& x) {
  a.x = fmaf(s, x.x, a.x); a.y = fmaf(s, x.y, a.y);
  a.z = fmaf(s, x.z, a.z); a.w = fmaf(s, x.w, a.w);
}
// Packed fp32: two multiply-adds an instruction.
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
struct F4 {
  float2 a, b;
};
__device__ __forceinline__ F4 f4(const float* p) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  return F4{make_float2(x.x, x.y), make_float2(x.z, x.w)};
}
__device__ __forceinline__ void put4(float* p, const F4& x) {
  *reinterpret_cast<float4*>(p) = make_float4(x.a.x, x.a.y, x.b.x, x.b.y);
}
__device__ __forceinline__ void fma4(F4& acc, float s, const F4& x) {
  const float2 ss = make_float2(s, s);
  acc.a = f2_fma(ss, x.a, acc.a);
  acc.b = f2_fma(ss, x.b, acc.b);
}
__device__ __forceinline__ void scale4(F4& x, float s) {
  x.a.x *= s; x.a.y *= s; x.b.x *= s; x.b.y *= s;
}
// The dot product of four pairs, its even and odd terms apart.
__device__ __forceinline__ float2 dot4x2(const float4& a, const float4& b, float2 acc) {
  acc = f2_fma(make_float2(a.x, a.y), make_float2(b.x, b.y), acc);
  return f2_fma(make_float2(a.z, a.w), make_float2(b.z, b.w), acc);
}

// 16 bytes to shared memory asynchronously, or zeros (the source is not touched then).
__device__ __forceinline__ void copy16(float* dst, const float* src, bool in) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if (in) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else *reinterpret_cast<float4*>(dst) = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Shared floats of the chunked pass: q, k rows padded by 4 (the rows that 16 threads read at
// one column fall into different banks), v, the state, P padded by 4, the decay tables.
__host__ __device__ inline int la_smem_floats(int K, int V) {
  return 2 * kChunk * (K + 4) + kChunk * V + K * V + kChunk * (kChunk + 4) + 80 + 2 * (kLaMaxSegments + 2);
}

// One CTA per (sequence, head, segment), 256 threads as 16 x 16; the state stays in shared memory.
// Every product is register-blocked (P 4 x 4 a thread, o 4 x 8, X 8 x 8) in packed fp32, two
// multiply-adds an instruction: the two warps a scheduler that shared memory leaves at K = V = 128
// do not hide the latencies of twice as many (34 us a chunk, now 23; 512 threads with half the
// block each 39).  Smaller head dims run two CTAs an SM.  What the mask takes away of P and P V is
// left out by blocks.  Bound by the fp32 units (2.7 M multiply-adds a chunk at K = V = 128, about
// 21k cycles of them).  Chains that do not fill the GPU are cut into segments as on the tensor
// cores: a launch (`local_only`) for each segment's own contribution, and one from the entry
// states.  A chain's scratch holds a copy of its entry state (the exit state may go to the same
// place), then the contributions in order, [K][V] each.
struct LaPasses {
  LinAttnPass pass[kLaMaxPasses];
  int segs, local_only;
  float* scratch;        // [pass][n][h][segs][K][V]
};

__global__ void __launch_bounds__(kLaThreads, 2) linear_attn_kernel(const __grid_constant__ LaPasses a) {
  extern __shared__ __align__(16) float sm[];
  const int segs = a.segs, local_only = a.local_only;
  int unit = blockIdx.x;   // heads vary fastest, then sequences, segments, passes
  const int h = unit % a.pass[0].H;
  unit /= a.pass[0].H;
  const int n = unit % a.pass[0].num_seqs;
  unit /= a.pass[0].num_seqs;
  const int parts = local_only ? segs - 1 : segs, seg = unit % parts, pi = unit / parts;
  const LinAttnPass p = a.pass[pi];
  const int K = p.K, V = p.V, KS = K + 4;
  float* sQ = sm;
  float* sK = sQ + kChunk * KS;
  float* sV = sK + kChunk * KS;
  float* sX = sV + kChunk * V;
  float* sP = sX + K * V;                 // [64][68]
  float* sW = sP + kChunk * (kChunk + 4);   // gamma^0 .. gamma^64
  constexpr int PS = kChunk + 4;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (local_only) next_may_start();
  const LaChain c = la_chain(p, n, h, tid == 0 && h == 0 && seg == 0);
  const int T_total = p.cu_seqlens ? p.T : p.B * p.T;
  if (seg == 0 && !local_only) {
    la_zero_rows(p, h, c.tail, T_total, tid, kLaThreads);
    if (c.padding) la_zero_rows(p, h, c.bos, c.eos, tid, kLaThreads);
  }
  if (c.skip || c.padding) {
    wait_for_previous();
    return;
  }
  const int nch = (c.eos - c.bos + kChunk - 1) / kChunk;
  const int per = max(1, (nch + segs - 1) / segs);
  const int c0 = min(seg * per, nch), c1 = min(c0 + per, nch);
  const bool last = c1 == nch, whole = seg == 0 && last;
  if (local_only ? last : (c0 == c1 && !whole)) {
    wait_for_previous();
    return;
  }
  const float ld = clamp_log_decay(p.log_decay[h]);
  // decay over a full chunk, the partial chunk and each segment before this one (by one thread each:
  // they are made in 64 bits)
  float2* sG = reinterpret_cast<float2*>(sW + 80);
  if (tid <= kChunk) sW[tid] = decay_pow(ld, (float)tid);
  if (tid < seg + 2) {
    const int rest = nch * kChunk - (c.eos - c.bos);   // tokens that the partial chunk lacks
    const int tokens = tid == 0 ? kChunk : tid == 1 ? kChunk - rest
                       : per * kChunk - (p.reverse && tid == 2 ? rest : 0);   // (backwards it is first)
    sG[tid] = decay_pow2(ld, tokens);
  }
  __syncthreads();
  float* slots =   // (segs > 1 only)
      a.scratch + ((size_t)(pi * p.num_seqs + n) * p.H + h) * segs * (size_t)(K * V);
  wait_for_previous();
  {   // the entry state
    const float* init = whole || (local_only && seg == 0) ? c.init : nullptr;
    for (int e = tid; e < K * V; e += kLaThreads) {
      const int kk = e / V, vv = e - kk * V;
      float x = init ? init[p.initial_t ? vv * K + kk : e] : 0.f;
      if (local_only) {
        if (seg == 0) slots[e] = x;
        x = 0.f;
      } else if (!whole) {
        x = __ldcg(slots + e);
      }
      sX[e] = x;
    }
    if (!local_only && !whole)
      for (int r = 0; r < seg; ++r) {
        const float2 g = sG[r + 2];
        const float* src = slots + (size_t)(r + 1) * K * V;
        for (int e = tid; e < K * V; e += kLaThreads) sX[e] = mul2(sX[e], g) + __ldcg(src + e);
      }
  }
  const int K4 = K / 4, V4 = V / 4;
  const float* gq = reinterpret_cast<const float*>(p.q);
  const float* gk = reinterpret_cast<const float*>(p.k);
  const float* gv = reinterpret_cast<const float*>(p.v);
  const int hq = h / (p.H / p.Hq), hk = h / (p.H / p.Hk), hv = h / (p.H / p.Hv);
  for (int cc = c0; cc < c1; ++cc) {
    const int ch = p.reverse ? nch - 1 - cc : cc;
    const int t0 = c.bos + ch * kChunk, L = min(kChunk, c.eos - t0);
    __syncthreads();
    // q, k, v of the chunk, all copies in flight at once; rows past its end zero
    for (int t = tid / K4; t < kChunk; t += kLaThreads / K4) {
      const int d = 4 * (tid % K4);
      if (tid / K4 >= kLaThreads / K4) break;   // (threads beyond the last whole row)
      if (!local_only) copy16(sQ + t * KS + d, gq + ((size_t)(t0 + t) * p.Hq + hq) * K + d, t < L);
      copy16(sK + t * KS + d, gk + ((size_t)(t0 + t) * p.Hk + hk) * K + d, t < L);
    }
    for (int t = tid / V4; t < kChunk; t += kLaThreads / V4) {
      const int d = 4 * (tid % V4);
      if (tid / V4 >= kLaThreads / V4) break;
      copy16(sV + t * V + d, gv + ((size_t)(t0 + t) * p.Hv + hv) * V + d, t < L);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!local_only) {
      {   // P: rows ty + 16 i, columns tx + 16 j; blocks beyond the diagonal are masked
        float2 acc[4][4] = {};
        for (int d = 0; d < K; d += 4) {
          float4 a[4], b[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            a[m] = *reinterpret_cast<const float4*>(sQ + (ty + 16 * m) * KS + d);
            b[m] = *reinterpret_cast<const float4*>(sK + (tx + 16 * m) * KS + d);
          }
          if (p.reverse) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = i; j < 4; ++j) acc[i][j] = dot4x2(a[i], b[j], acc[i][j]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j <= i; ++j) acc[i][j] = dot4x2(a[i], b[j], acc[i][j]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = ty + 16 * i, s = tx + 16 * j, dist = p.reverse ? s - r : r - s;
            sP[r * PS + s] = dist >= 0 ? p.s_in * sW[dist] * (acc[i][j].x + acc[i][j].y) : 0.f;
          }
      }
      __syncthreads();
      // o: rows 4 ty .. + 3, columns 4 tx + 64 m .. + 3
      {
        const bool two = 4 * tx + 64 < V, one = 4 * tx < V;
        F4 acc[2][4] = {};
        auto rows = [&](const float* left, int stride, const float* right, int d0, int d1) {
#pragma unroll 2
          for (int d = d0; d < d1; d += 4) {
            float4 a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(left + (4 * ty + i) * stride + d);
#pragma unroll
            for (int dd = 0; dd < 4; ++dd) {
              const float* x = right + (d + dd) * V + 4 * tx;
              const F4 x0 = one ? f4(x) : F4{}, x1 = two ? f4(x + 64) : F4{};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = dd == 0 ? a[i].x : dd == 1 ? a[i].y : dd == 2 ? a[i].z : a[i].w;
                fma4(acc[0][i], e, x0);
                if (two) fma4(acc[1][i], e, x1);
              }
            }
          }
        };
        rows(sQ, KS, sX, 0, K);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * ty + i;
          const float w = sW[p.reverse ? max(0, L - 1 - r) : r + 1];
          scale4(acc[0][i], w);
          scale4(acc[1][i], w);
        }
        // (P is zero on the far side of the diagonal, and from L on)
        rows(sP, PS, sV, p.reverse ? 4 * ty : 0, p.reverse ? L : min(L, 4 * ty + 4));
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i, col = 4 * tx + 64 * m;
            if (r >= L || col >= V) continue;
            scale4(acc[m][i], p.s_out);
            put4(reinterpret_cast<float*>(p.o) + ((size_t)(t0 + r) * p.H + h) * V + col, acc[m][i]);
          }
      }
      if (last && cc + 1 == c1 && !c.fin) break;   // nobody wants the state any more
      __syncthreads();   // the state has been read
    }
    // X: rows 4 ty + 64 a .. + 3, columns 4 tx + 64 m .. + 3; the chunk's products are summed first, so
    // that the state is rounded once a chunk (over a memory of 4096 tokens an error of 3 2^-24 instead of 11)
    const float2 gl = sG[L == kChunk ? 0 : 1];
    const bool two = 4 * tx + 64 < V, one = 4 * tx < V;
#pragma unroll
    for (int ma = 0; ma < 2; ++ma) {
      const int row = 4 * ty + 64 * ma;
      if (row >= K) break;
      F4 acc[2][4] = {};
#pragma unroll 4
      for (int j = 0; j < L; ++j) {
        float4 kk = *reinterpret_cast<const float4*>(sK + j * KS + row);
        const float w = p.s_in * sW[p.reverse ? j + 1 : L - 1 - j];
        kk.x *= w; kk.y *= w; kk.z *= w; kk.w *= w;
        const float* x = sV + j * V + 4 * tx;
        const F4 x0 = one ? f4(x) : F4{}, x1 = two ? f4(x + 64) : F4{};
        fma4(acc[0][0], kk.x, x0);
        fma4(acc[0][1], kk.y, x0);
        fma4(acc[0][2], kk.z, x0);
        fma4(acc[0][3], kk.w, x0);
        if (two) {
          fma4(acc[1][0], kk.x, x1);
          fma4(acc[1][1], kk.y, x1);
          fma4(acc[1][2], kk.z, x1);
          fma4(acc[1][3], kk.w, x1);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (m ? two : one) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float* at = sX + (row + i) * V + 4 * tx + 64 * m;
            const F4 x = f4(at), u = acc[m][i];
            put4(at, F4{make_float2(mul2_add(x.a.x, gl, u.a.x), mul2_add(x.a.y, gl, u.a.y)),
                        make_float2(mul2_add(x.b.x, gl, u.b.x), mul2_add(x.b.y, gl, u.b.y))});
          }
        }
    }
  }
  __syncthreads();
  float* out = local_only ? slots + (size_t)(seg + 1) * K * V : last ? c.fin : nullptr;
  if (out)
    for (int e = tid; e < K * V; e += kLaThreads) out[e] = sX[e];
}

// Sum of the value heads that share a query/key head.  A thread keeps its 4 channels and walks over
// rows, four at a time (their loads in flight together).  Bound by bytes: 98 us for
// 671 MB (6.8 TB/s).
constexpr int kFoldRows = 4;
template <typename T>
__global__ void __launch_bounds__(kLaThreads)
    linear_attn_fold_kernel(const float* part0, const float* part1, T* out0, T* out1, long long rows, int group,
                            int D) {
  const float* part = blockIdx.y ? part1 : part0;
  T* out = blockIdx.y ? out1 : out0;
  const int D4 = D / 4, per = kLaThreads / D4, d = 4 * (threadIdx.x % D4), row = threadIdx.x / D4;
  if (row >= per) return;
  const long long step = (long long)gridDim.x * per;
  for (long long r = (long long)blockIdx.x * per + row; r < rows; r += kFoldRows * step) {
    float4 s[kFoldRows];
#pragma unroll
    for (int i = 0; i < kFoldRows; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < group; ++j) {
#pragma unroll
      for (int i = 0; i < kFoldRows; ++i)
        if (r + i * step < rows) {
          const float4 x = __ldcs(reinterpret_cast<const float4*>(part + ((r + i * step) * group + j) * D + d));
          s[i].x += x.x; s[i].y += x.y; s[i].z += x.z; s[i].w += x.w;
        }
    }
#pragma unroll
    for (int i = 0; i < kFoldRows; ++i)
      if (r + i * step < rows) store4(out + (r + i * step) * D + d, s[i]);
  }
}

// One CTA per (request, head): S <- gamma S + k v^T, o = scale S^T q, the state read and written
// once.  Bound by those bytes: 166 us for 230 requests' 967 MB (5.8 TB/s).  Thread t owns the
// float4 column group t % (V / 4) of every (threads / (V / 4))-th row.
template <typename T>
__global__ void __launch_bounds__(kLaThreads) linear_attn_decode_kernel(const LinAttnDecodeArgs a) {
  __shared__ float sq[GDN_MAX_HEAD_DIM], sk[GDN_MAX_HEAD_DIM];
  __shared__ float4 red[kLaThreads];
  const int K = a.K, V = a.V, V4 = V / 4;
  const int h = blockIdx.x % a.Hv, i = blockIdx.x / a.Hv, tid = threadIdx.x;
  const int slot = a.batch_indices ? a.batch_indices[i] : i;
  T* o = reinterpret_cast<T*>(a.o) + ((size_t)i * a.Hv + h) * V;
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1 && tid == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
    for (int d = tid; d < V; d += kLaThreads) store_elem(o, d, 0.f, a.io_dtype);
    return;
  }
  const int hq = h / (a.Hv / a.Hqk);
  const size_t qk = ((size_t)i * a.Hqk + hq) * K;
  if (tid < K) {
    sq[tid] = load_elem(a.q, qk + tid, a.io_dtype) * a.scale;
    sk[tid] = load_elem(a.k, qk + tid, a.io_dtype);
  }
  // The decay as hi + lo, and one rounding of the new state: a decay rounded to 24 bits is off in the
  // same direction at every token, 1e-4 of the state after 4096 of them, and a decayed state rounded
  // before k v^T is added does not decay at all where gamma is within 2^-25 of 1.
  const float2 g = decay_pair(a.log_decay[h]);
  __syncthreads();
  const int G = kLaThreads / V4, c = tid % V4, r0 = tid / V4;
  float* S = a.state + ((size_t)slot * a.Hv + h) * (size_t)K * V;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r0 < G) {
    const float4 v = load4(reinterpret_cast<const T*>(a.v) + ((size_t)i * a.Hv + h) * V + 4 * c);
    for (int r = r0; r < K; r += G) {
      float4* s = reinterpret_cast<float4*>(S + (size_t)r * V) + c;
      float4 x = *s;
      const float k = sk[r], q = sq[r];
      x.x = mul2_add(x.x, g, k * v.x); x.y = mul2_add(x.y, g, k * v.y);
      x.z = mul2_add(x.z, g, k * v.z); x.w = mul2_add(x.w, g, k * v.w);
      *s = x;
      fma4(acc, q, x);
    }
  }
  red[tid] = acc;
  __syncthreads();
  if (tid < V4) {
    for (int r = 1; r < G; ++r) {
      const float4 x = red[r * V4 + tid];
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    store4(o + 4 * tid, acc);
  }
}

}  // namespace

int linear_attn_segments(long long chains, long long most_tokens, int places, int min_chunks) {
  if (chains <= 0 || places <= 0) return 1;
  const long long chunks = (most_tokens + kChunk - 1) / kChunk;
  return (int)std::max(1LL, std::min({(long long)kLaMaxSegments, places / chains, chunks / min_chunks}));
}

int linear_attn_generic_per_sm(int K, int V) {
  return la_smem_floats(K, V) * sizeof(float) + 1024 <= 113 * 1024 ? 2 : 1;
}

LaPlan linear_attn_plan(long long chains, long long most_tokens, bool uniform, int places) {
  const int few = linear_attn_segments(chains, most_tokens, places, kLaMinSegmentChunks);
  LaPlan best{few > 1 ? 0 : chains, few};
  if (!uniform || few > 1 || chains <= places || chains > 4LL * places) return best;
  // More chains than places: the last, partly empty wave of whole ones costs as much as a full one
  // (192 chains on 152 SMs: 350 us; cut, see below, 290).  Costs in chunks: a CTA's start 8, a
  // chunk of a segment's own contribution 0.5.  Beside `rem` whole chains of a wave the others'
  // contributions are made.
  const double chunks = (double)((most_tokens + kChunk - 1) / kChunk), start = 8.0;
  const auto waves = [&](long long n) { return (double)((n + places - 1) / places); };
  double least = 0.95 * waves(chains) * (chunks + start);
  for (int s = 2; s <= kLaMaxSegments && chunks >= s * (double)kLaMinSegmentChunks; ++s) {
    const double part = chunks / s + start, own = 0.5 * chunks / s + start;
    for (int full = 1; full <= s; ++full) {   // (of the second launch's waves)
      const long long cut = std::min(chains, (long long)full * places / s), whole = chains - cut;
      const long long rem = whole % places;
      const long long beside = rem > 0 ? (places - rem) * (long long)((chunks + start) / own) : 0;
      const double first = waves(whole) * (chunks + start) + waves(std::max(0LL, cut * (s - 1) - beside)) * own;
      const double total = first + waves(cut * s) * part;
      if (total < least) {
        least = total;
        best = LaPlan{whole, s};
      }
    }
  }
  return best;
}

cudaError_t launch_linear_attn_generic(const LinAttnPass* passes, int num_passes, int segs, float* scratch) {
  const LinAttnPass& p0 = passes[0];
  const long long chains = (long long)num_passes * p0.num_seqs * p0.H;
  if (chains <= 0) return cudaSuccess;
  if (num_passes > kLaMaxPasses || segs < 1 || segs > kLaMaxSegments || chains * segs > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    err = cudaFuncSetAttribute(linear_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               la_smem_floats(GDN_MAX_HEAD_DIM, GDN_MAX_HEAD_DIM) * (int)sizeof(float));
    if (err != cudaSuccess) return err;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  LaPasses a{};
  size_t smem = 0;
  for (int i = 0; i < num_passes; ++i) {
    a.pass[i] = passes[i];
    smem = std::max(smem, la_smem_floats(passes[i].K, passes[i].V) * sizeof(float));
  }
  a.segs = segs;
  a.scratch = scratch;
  if (segs > 1) {
    a.local_only = 1;
    linear_attn_kernel<<<(unsigned)(chains * (segs - 1)), kLaThreads, smem, p0.stream>>>(a);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    a.local_only = 0;
    return launch_behind(linear_attn_kernel, (unsigned)(chains * segs), kLaThreads, smem, p0.stream, a);
  }
  linear_attn_kernel<<<(unsigned)chains, kLaThreads, smem, p0.stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_linear_attn_fold(const float* const (&part)[2], void* const (&out)[2], long long T_total,
                                    int Hqk, int group, int D, int io_dtype, cudaStream_t stream) {
  const long long rows = T_total * Hqk, per = kLaThreads / (D / 4);
  if (rows == 0) return cudaSuccess;
  const dim3 grid((unsigned)std::min((rows + per - 1) / per, std::max(1LL, 8LL * current_sm_count())), 2);
  if (io_dtype == GDN_F32)
    linear_attn_fold_kernel<<<grid, kLaThreads, 0, stream>>>(part[0], part[1], reinterpret_cast<float*>(out[0]),
                                                      reinterpret_cast<float*>(out[1]), rows, group, D);
  else
    linear_attn_fold_kernel<<<grid, kLaThreads, 0, stream>>>(part[0], part[1],
                                                      reinterpret_cast<__nv_bfloat16*>(out[0]),
                                                      reinterpret_cast<__nv_bfloat16*>(out[1]), rows, group, D);
  return cudaGetLastError();
}

cudaError_t launch_linear_attn_decode(const LinAttnDecodeArgs& a) {
  const long long blocks = (long long)a.n * a.Hv;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (a.io_dtype == GDN_F32)
    linear_attn_decode_kernel<float><<<(unsigned)blocks, kLaThreads, 0, a.stream>>>(a);
  else
    linear_attn_decode_kernel<__nv_bfloat16><<<(unsigned)blocks, kLaThreads, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdn
