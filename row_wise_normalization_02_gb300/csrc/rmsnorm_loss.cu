// Log-probability of each row's target token, the clipped policy loss and the
// preference loss over it, and the gradient of the logits (sm_103a).
//
//   z = logits / temperature,  lse = log sum_j exp(z_j),  logp = z_t - lse
//   d logp / d logits_j = ([j = t] - exp(z_j - lse)) / temperature
//
// A row of logits is one of the largest things a model touches (V to 10^5 and
// more), and everything else here is a handful of numbers per row: the kernels
// are bound by reading the logits once, and by writing their gradient.
//
// Row kernel: one pass with a running maximum and sum.  A thread keeps its
// maximum m and s = sum 2^((x - m) c), c = log2(e) / temperature: the difference
// first, so that nothing overflows or loses digits however large the logits are
// (a mask may hold the type's lowest value).  A batch of vectors is loaded, its
// maximum taken (bf16 from the packed words), s rescaled if the maximum grew,
// then the batch added.  Threads, warps and the cluster's CTAs merge their (m, s)
// in a fixed order.  lse = m / temperature + log s is put together in 64 bits by
// one thread, so logp carries the error of s alone (about 1e-7), not a rounding
// of lse, and differences of log-probabilities are taken before the result is
// rounded to fp32.
//
// Few rows: a row is split over a cluster of up to eight CTAs that exchange
// (m, s) through distributed shared memory; no workspace, one launch.
#include <math_constants.h>

#include "rmsnorm_device.cuh"
#include "rmsnorm_internal.h"

#ifndef RMSN_PAIR
#error "compile once per dtype with -DRMSN_PAIR=0 (f32), 1 (bf16)"
#endif

namespace rmsn {
namespace {

#define kNegInf (-CUDART_INF_F)
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maximum of U 16-byte vectors.  A NaN is passed over here and shows in the sum.
template <int U>
__device__ __forceinline__ float max_of(const uint4 (&v)[U], float*) {
  float m = kNegInf;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    float f[4];
    unpack(v[k], f);
    m = fmaxf(fmaxf(m, f[0]), fmaxf(f[1], fmaxf(f[2], f[3])));
  }
  return m;
}
template <int U>
__device__ __forceinline__ float max_of(const uint4 (&v)[U], bf16*) {
  const uint32_t ninf2 = 0xFF80FF80u;
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&ninf2);
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v[k]);
    m = __hmax2(m, __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
  }
  return fmaxf(__low2float(m), __high2float(m));
}
template <typename TX>
__device__ __forceinline__ uint4 neg_inf_vec() {
  constexpr uint32_t w = sizeof(TX) == 4 ? 0xFF800000u : 0xFF80FF80u;
  return make_uint4(w, w, w, w);
}

// A running maximum m with s = sum 2^((x - origin(m)) c); the origin of -inf is
// 0, so that rows and parts of nothing but -inf sum to zero.
struct Run {
  float m, s;
};
__device__ __forceinline__ float origin(float m) { return m == kNegInf ? 0.f : m; }
__device__ __forceinline__ void raise(Run& r, float m, float c) {
  if (m > r.m) {
    r.s *= ex2((r.m - m) * c);
    r.m = m;
  }
}
__device__ __forceinline__ Run warp_merge(Run r, float c) {
  float m = r.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  raise(r, m, c);
  r.s = group_sum<32>(r.s);
  return Run{m, r.s};
}

// Warp 0 gets the CTA's.  part: shared, one per warp.
__device__ __forceinline__ Run cta_merge(Run r, float c, float2* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  r = warp_merge(r, c);
  if (lane == 0) part[warp] = make_float2(r.m, r.s);
  __syncthreads();
  if (warp == 0) {
    const float2 q = lane < (int)(blockDim.x >> 5) ? part[lane] : make_float2(kNegInf, 0.f);
    r = warp_merge(Run{q.x, q.y}, c);
  }
  return r;
}
template <typename TX, int U>
__device__ __forceinline__ void add_batch(Run& r, const uint4 (&b)[U], float c) {
  constexpr int E = Elem<TX>::kPerVec;
  raise(r, max_of(b, static_cast<TX*>(nullptr)), c);
  const float o = origin(r.m);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < U; ++k) {
    float q[E];
    unpack(b[k], q);
#pragma unroll
    for (int i = 0; i < E; ++i) s[i & 3] += ex2((q[i] - o) * c);
  }
  r.s += (s[0] + s[1]) + (s[2] + s[3]);
}
__device__ __forceinline__ void add_one(Run& r, float q, float c) {
  raise(r, q, c);
  r.s += ex2((q - origin(r.m)) * c);
}

// A row as elements up to the first 16-byte boundary, vectors, and the rest.
struct Frame {
  int head, nvec, tail0;   // tail0: first element behind the vectors
};
template <typename TX>
__device__ __forceinline__ Frame frame_of(const TX* row, int V) {
  constexpr int E = Elem<TX>::kPerVec;
  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(TX));
  Frame f;
  f.head = off ? min(E - off, V) : 0;
  f.nvec = (V - f.head) / E;
  f.tail0 = f.head + f.nvec * E;
  return f;
}

// ---------------------------------------------------------------- per-row losses

struct PolicyTerm {
  float loss, slope;   // of the row, times its weight
};
__device__ __forceinline__ PolicyTerm policy_term(const LossParams& p, int64_t row, double logp) {
  const float w = p.weights ? p.weights[row] : 1.f;
  if (w == 0.f) return PolicyTerm{0.f, 0.f};
  const float A = p.advantages[row];
  const float r = expf((float)(logp - (double)p.old_logp[row]));
  const bool up = A >= 0.f && r > p.ratio_hi, down = A < 0.f && r < p.ratio_lo;
  float loss = -A * (up ? p.ratio_hi : down ? p.ratio_lo : r);
  float slope = up || down ? 0.f : -A * r;
  if (p.ref_logp) {
    const float d = (float)((double)p.ref_logp[row] - logp), e = expm1f(d);
    loss = fmaf(p.kl, e - d, loss);
    slope = fmaf(-p.kl, e, slope);
  }
  return PolicyTerm{w * loss, w * slope};
}

// log(s) in 64 bits from fp32 functions: the exponent is exact and the mantissa,
// in [0.75, 1.5), has a logarithm small enough that its rounding is below 2^-25.
__device__ __forceinline__ double log_sum(float s) {
  if (!(s > 0.f) || !(s < CUDART_INF_F)) return (double)logf(s);
  const uint32_t b = __float_as_uint(s);
  const int e = (int)(b - 0x3F400000u) >> 23;   // 0x3F400000: 0.75
  return (double)e * kLn2 + (double)logf(__uint_as_float(b - ((uint32_t)e << 23)));
}

// ---------------------------------------------------------------- row kernel

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

template <typename TX, int MODE, int CL>
__global__ void __launch_bounds__(kLossThreads, 4) loss_row_kernel(LossParams p) {
  constexpr int E = Elem<TX>::kPerVec, U = kLossBatch;
  __shared__ float2 part[32];
  __shared__ float2 peers[8];
  __shared__ float4 verdict;   // coefficient of 2^((x - m) c), origin(m), the target's addend
  pdl_begin();
  const int64_t row = blockIdx.x / CL;
  const int rank = CL > 1 ? (int)cta_rank() : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int64_t t = p.targets[row];
  const TX* x = static_cast<const TX*>(p.logits) + row * p.ld;
  TX* dx = MODE == kLossPolicyGrad ? static_cast<TX*>(p.dlogits) + row * p.ld_out : nullptr;
  const Frame f = frame_of(x, p.V);
  const int v0 = CL > 1 ? (int)((int64_t)f.nvec * rank / CL) : 0;
  const int v1 = CL > 1 ? (int)((int64_t)f.nvec * (rank + 1) / CL) : f.nvec;
  const bool first = rank == 0, last = rank == CL - 1;
  const TX* xv = x + f.head;
  const bool same = MODE == kLossPolicyGrad &&
                    ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
  // this CTA's elements, for rows whose gradient starts elsewhere modulo 16
  const int e0 = first ? 0 : f.head + v0 * E, e1 = last ? p.V : f.head + v1 * E;

  if (t < 0) {   // the row takes no part
    if (first && tid == 0) {
      p.logp[row] = 0.f;
      p.lse[row] = 0.f;
      if (MODE != kLossLogprob) p.dlogp[row] = 0.f;
      if (MODE == kLossPolicy || MODE == kLossPolicyGrad) p.token_loss[row] = 0.f;
    }
    if (MODE == kLossPolicyGrad) {
      if (same) {
        for (int v = v0 + tid; v < v1; v += nt)
          st_stream(dx + f.head + (size_t)v * E, make_uint4(0, 0, 0, 0));
        if (first)
          for (int j = tid; j < f.head; j += nt) st_scalar(dx + j, 0.f);
        if (last)
          for (int j = f.tail0 + tid; j < p.V; j += nt) st_scalar(dx + j, 0.f);
      } else {
        for (int j = e0 + tid; j < e1; j += nt) st_scalar(dx + j, 0.f);
      }
    }
    return;
  }
  if (CL > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  float xt = CUDART_NAN_F;   // a target past the row gives NaN
  if (tid == 0 && t < p.V) xt = ld_scalar(x + t);

  Run r{kNegInf, 0.f};
  const float c = p.c1;
  for (int v = v0 + tid; v < v1; v += U * nt) {
    uint4 b[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      b[k] = v + k * nt < v1 ? ld_rw(xv + (size_t)(v + k * nt) * E)
                             : neg_inf_vec<TX>();
    add_batch<TX>(r, b, c);
  }
  if (first)
    for (int j = tid; j < f.head; j += nt) add_one(r, ld_scalar(x + j), c);
  if (last)
    for (int j = f.tail0 + tid; j < p.V; j += nt) add_one(r, ld_scalar(x + j), c);
  r = cta_merge(r, c, part);
  if (CL > 1) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");   // every CTA has started
    if (tid < CL) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(peers + rank)),
                   "r"(tid));
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(r.m), "f"(r.s)
                   : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (warp == 0) {
      const float2 q = lane < CL ? peers[lane] : make_float2(kNegInf, 0.f);
      r = warp_merge(Run{q.x, q.y}, c);
    }
  }
  if (MODE != kLossPolicyGrad && !first) return;
  if (tid == 0) {
    const double lse = (double)r.m * p.inv_t + log_sum(r.s);
    const double logp = (double)xt * p.inv_t - lse;
    if (first) {
      p.logp[row] = (float)logp;
      p.lse[row] = (float)lse;
    }
    if (MODE == kLossPolicy || MODE == kLossPolicyGrad) {
      const PolicyTerm q = policy_term(p, row, logp);
      if (first) {
        p.token_loss[row] = q.loss;
        p.dlogp[row] = q.slope;
      }
      if (MODE == kLossPolicyGrad) {
        const float g = q.slope * p.inv_tf;
        verdict = make_float4(g == 0.f ? 0.f : -g / r.s, origin(r.m), g, 0.f);
      }
    }
    if (MODE == kLossPreference) {
      const bool inside = row >= p.cu[0] && row < p.cu[2 * p.pairs];
      p.dlogp[row] = inside ? (float)(logp - (p.ref_logp ? (double)p.ref_logp[row] : 0.0)) : 0.f;
    }
  }
  if (MODE == kLossPolicyGrad) {
    __syncthreads();
    const float coef = verdict.x, o = verdict.y, g = verdict.z;
    // (no fused add of the target's g: every path rounds alike)
    auto value = [&](float q) { return __fmul_rn(coef, ex2((q - o) * c)); };
    auto grad = [&](int j) {
      float d = 0.f;
      if (g != 0.f) d = value(ld_scalar(x + j)) + (j == t ? g : 0.f);
      st_scalar(dx + j, d);
    };
    if (!same) {
      for (int j = e0 + tid; j < e1; j += nt) grad(j);
      return;
    }
    const int64_t tv = t - f.head;   // the target's place among the vectors' elements
    for (int v = v0 + tid; v < v1; v += U * nt) {
      uint4 b[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (v + k * nt < v1) b[k] = ld_rw(xv + (size_t)(v + k * nt) * E);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int w = v + k * nt;
        if (w >= v1) break;
        float q[E];
        unpack(b[k], q);
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] = value(q[i]);
        if (g == 0.f) {
#pragma unroll
          for (int i = 0; i < E; ++i) q[i] = 0.f;
        } else if (tv >= 0 && tv / E == w) {
#pragma unroll
          for (int i = 0; i < E; ++i) q[i] += (int)(tv % E) == i ? g : 0.f;
        }
        st_stream(dx + f.head + (size_t)w * E, pack(q));
      }
    }
    if (first)
      for (int j = tid; j < f.head; j += nt) grad(j);
    if (last)
      for (int j = f.tail0 + tid; j < p.V; j += nt) grad(j);
  }
}

// ---------------------------------------------------------------- backward

// dlogits_j = g ([j = t] - exp(z_j - lse)), g = dlogp scale / temperature.  A CTA
// takes kLossBwdVecs vectors of a row; rows that take no part and rows whose g
// is zero are zeroed without being read.  An fp32 lse has lost the digits that
// exp(z - lse) needs where it is large (2^-24 |lse| relative): behind kLseFine, which
// the logits of a working model do not reach, a CTA takes its row's maximum and
// sum again and uses those.
constexpr float kLseFine = 2048.f;
template <typename TX>
__global__ void __launch_bounds__(kLossThreads, 4) loss_bwd_kernel(LossParams p) {
  constexpr int E = Elem<TX>::kPerVec, U = kLossBatch;
  __shared__ float2 part[32];
  __shared__ float2 again;
  pdl_begin();
  const int tid = threadIdx.x;
  const int chunks = (p.V + kLossBwdVecs * E - 1) / (kLossBwdVecs * E);
  const int64_t items = p.M * chunks;
  const float scale = (p.scale ? *p.scale : 1.f) * p.inv_tf;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / chunks;
    const int chunk = (int)(it - row * chunks);
    const int64_t t = p.targets[row];
    const float g = t < 0 ? 0.f : t < p.V ? p.dlogp_in[row] * scale : CUDART_NAN_F;
    const float lse = p.lse[row];
    const TX* x = static_cast<const TX*>(p.logits) + row * p.ld;
    TX* dx = static_cast<TX*>(p.dlogits) + row * p.ld_out;
    // exp(z - lse) times -g as coef 2^((x fac - o) c)
    float coef = -g, fac = p.inv_tf, o = lse, c = kLog2e;
    int c0 = chunk, c1 = chunk + 1;
    if (g != 0.f && fabsf(lse) > kLseFine) {
      if (chunk != 0) continue;   // the row's first CTA takes all of it: dlogits may be logits
      c1 = chunks;
      Run r{kNegInf, 0.f};
      for (int j = tid; j < p.V; j += kLossThreads) add_one(r, ld_scalar(x + j), p.c1);
      r = cta_merge(r, p.c1, part);
      if (tid == 0) again = make_float2(origin(r.m), r.s);
      __syncthreads();
      coef = -g / again.y;
      fac = 1.f;
      o = again.x;
      c = p.c1;
      __syncthreads();   // before another item writes `part` or `again`
    }
    // (no fused add of the target's g: every path rounds alike)
    auto value = [&](float q) { return __fmul_rn(coef, ex2(fmaf(q, fac, -o) * c)); };
    auto element = [&](int j) {
      float d = 0.f;
      if (g != 0.f) d = value(ld_scalar(x + j)) + (j == t ? g : 0.f);
      st_scalar(dx + j, d);
    };
    if (((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) != 0) {
      const int e1 = min((int64_t)p.V, (int64_t)c1 * kLossBwdVecs * E);
      for (int j = c0 * kLossBwdVecs * E + tid; j < e1; j += kLossThreads) element(j);
      continue;
    }
    // chunks of the row's vectors; the last one is short by the head at most,
    // so the row's `chunks` chunks cover them all
    const Frame f = frame_of(x, p.V);
    const int64_t tv = t - f.head;
    for (int w0 = c0 * kLossBwdVecs + tid; w0 < c1 * kLossBwdVecs; w0 += kLossBwdVecs) {
      uint4 b[U];
      if (g != 0.f) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (w0 + k * kLossThreads < f.nvec)
            b[k] = ld_rw(x + f.head + (size_t)(w0 + k * kLossThreads) * E);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int w = w0 + k * kLossThreads;
        if (w >= f.nvec) break;
        uint4 out = make_uint4(0, 0, 0, 0);
        if (g != 0.f) {
          float q[E];
          unpack(b[k], q);
#pragma unroll
          for (int i = 0; i < E; ++i) q[i] = value(q[i]);
          if (tv >= 0 && tv / E == w) {
#pragma unroll
            for (int i = 0; i < E; ++i) q[i] += (int)(tv % E) == i ? g : 0.f;
          }
          out = pack(q);
        }
        st_stream(dx + f.head + (size_t)w * E, out);
      }
    }
    if (chunk == 0) {
      for (int j = tid; j < f.head; j += kLossThreads) element(j);
      for (int j = f.tail0 + tid; j < p.V; j += kLossThreads) element(j);
    }
  }
}

#if RMSN_PAIR == 0
// ---------------------------------------------------------------- sums over rows

constexpr int kSumThreads = 1024;

// Sum over the CTA in a fixed order, 64 bits; every thread gets it.
__device__ __forceinline__ double cta_sum64(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();   // earlier readers of red are done
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += red[w];
  return s;
}

__global__ void __launch_bounds__(kSumThreads) loss_sum_kernel(LossParams p) {
  __shared__ double red[32];
  pdl_begin();
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < p.M; i += kSumThreads) s += (double)p.token_loss[i];
  s = cta_sum64(s, red);
  if (threadIdx.x == 0) *p.loss = (float)s;
}

// Rows [a, b) of sequence s, kept inside the batch whatever the offsets say.
__device__ __forceinline__ void rows_of(const LossParams& p, int64_t s, int64_t* a, int64_t* b) {
  *a = min(max(p.cu[s], (int64_t)0), p.M);
  *b = min(max(p.cu[s + 1], *a), p.M);
}

// Pair b: margin h = beta (sum over the chosen rows - sum over the rejected rows)
// of logp - ref, which the row kernel left in dlogp; then dlogp itself.
__global__ void __launch_bounds__(kLossThreads) loss_pairs_kernel(LossParams p) {
  __shared__ double red[32];
  pdl_begin();
  const int64_t b = blockIdx.x;
  int64_t a[2], e[2];
  double sum = 0.0;
  for (int side = 0; side < 2; ++side) {
    rows_of(p, b + side * p.pairs, &a[side], &e[side]);
    double s = 0.0;
    for (int64_t i = a[side] + threadIdx.x; i < e[side]; i += kLossThreads)
      s += (double)p.dlogp[i];
    sum += side ? -s : s;
  }
  const double h = (double)p.beta * cta_sum64(sum, red);
  const float hf = (float)h;
  const float slope = (p.smoothing / (1.f + expf(-hf)) - (1.f - p.smoothing) / (1.f + expf(hf))) *
                      (p.beta / (float)p.pairs);
  if (threadIdx.x == 0) p.margins[b] = hf;
  for (int side = 0; side < 2; ++side)
    for (int64_t i = a[side] + threadIdx.x; i < e[side]; i += kLossThreads)
      p.dlogp[i] = p.targets[i] < 0 ? 0.f : side ? -slope : slope;
}

// log(1 + exp(x))
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}
__global__ void __launch_bounds__(kLossThreads) loss_pairs_mean_kernel(LossParams p) {
  __shared__ double red[32];
  pdl_begin();
  double s = 0.0;
  for (int64_t b = threadIdx.x; b < p.pairs; b += kLossThreads) {
    const float h = p.margins[b];
    // a NaN margin passes fmaxf by: add it
    s += (double)((1.f - p.smoothing) * softplus(-h) + p.smoothing * softplus(h)) +
         (h == h ? 0.0 : (double)h);
  }
  s = cta_sum64(s, red);
  if (threadIdx.x == 0) *p.loss = (float)(s / (double)p.pairs);
}
#endif

template <typename TX, int MODE>
LossKernel pick_row(int cluster) {
  switch (cluster) {
    case 1: return loss_row_kernel<TX, MODE, 1>;
    case 2: return loss_row_kernel<TX, MODE, 2>;
    case 4: return loss_row_kernel<TX, MODE, 4>;
    case 8: return loss_row_kernel<TX, MODE, 8>;
    default: return nullptr;
  }
}
template <typename TX>
LossKernel pick_mode(int mode, int cluster) {
  switch (mode) {
    case kLossLogprob: return pick_row<TX, kLossLogprob>(cluster);
    case kLossPolicy: return pick_row<TX, kLossPolicy>(cluster);
    case kLossPolicyGrad: return pick_row<TX, kLossPolicyGrad>(cluster);
    case kLossPreference: return pick_row<TX, kLossPreference>(cluster);
    default: return nullptr;
  }
}

}  // namespace

#if RMSN_PAIR == 0
LossKernel get_loss_row_f32(int mode, int cluster) { return pick_mode<float>(mode, cluster); }
LossKernel get_loss_bwd_f32() { return loss_bwd_kernel<float>; }
LossKernel get_loss_sum() { return loss_sum_kernel; }
LossKernel get_loss_pairs() { return loss_pairs_kernel; }
LossKernel get_loss_pairs_mean() { return loss_pairs_mean_kernel; }
#else
LossKernel get_loss_row_bf16(int mode, int cluster) { return pick_mode<bf16>(mode, cluster); }
LossKernel get_loss_bwd_bf16() { return loss_bwd_kernel<bf16>; }
#endif

}  // namespace rmsn
