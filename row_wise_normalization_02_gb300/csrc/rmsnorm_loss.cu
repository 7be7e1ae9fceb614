// Log-probability of each row's target token, the clipped policy loss and the
// preference loss over it, and the gradient of the logits (sm_103a).
//
//   z = logits / temperature,  logp = z_t - log sum_j exp(z_j)
//   d logp / d logits_j = ([j = t] - p_j) / temperature,   p_j = exp(z_j) / sum_k exp(z_k)
//
// A row of logits is one of the largest things a model touches (V to 10^5 and
// more), and everything else here is a handful of numbers per row: the kernels
// are bound by reading the logits once, and by writing their gradient.
//
// Row kernel: one pass with a running maximum and sum.  A thread keeps its
// maximum m and s = sum 2^((x - m) c), c = log2(e) / temperature in two parts: the
// difference first, so that nothing overflows or loses digits however large the logits are
// (a mask may hold the type's lowest value).  A batch of vectors is loaded, its
// maximum taken (bf16 from the packed words), s rescaled if the maximum grew,
// then the batch added.  Threads, warps and the cluster's CTAs merge their (m, s)
// in a fixed order.  logp = (x_t - m) / temperature - log s is put together in two
// fp32 parts by one thread, so it carries the error of s alone (about 1e-7), not a
// rounding of the log-sum-exp, and differences of log-probabilities are taken
// before the result is rounded to fp32.
//
// Few rows: a row is split over a cluster of up to eight CTAs that exchange
// (m, s) through distributed shared memory; no workspace, one launch.
#include <math_constants.h>

#include "rmsnorm_device.cuh"
#include "rmsnorm_internal.h"
#include "rmsnorm_operators.h"
#include "rmsnorm_ring.cuh"   // kDrainLimit

#ifndef RMSN_PAIR
#error "compile once per dtype with -DRMSN_PAIR=0 (f32), 1 (bf16)"
#endif

namespace rmsn {
namespace {

#define kNegInf (-CUDART_INF_F)
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t bits2(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 float2_of(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}

// x - o of a vector's elements in pairs; bf16 ones straight from the packed halves
// by the mixed-precision fma (x 1 - o), which saves unpacking them.
[[maybe_unused]] __device__ __forceinline__ void differences(const uint4& v, float o,
                                                             float2 (&d)[2]) {
  const float2 n = make_float2(-o, -o);
  d[0] = add2(make_float2(__uint_as_float(v.x), __uint_as_float(v.y)), n);
  d[1] = add2(make_float2(__uint_as_float(v.z), __uint_as_float(v.w)), n);
}
[[maybe_unused]] __device__ __forceinline__ void differences(const uint4& v, float o,
                                                             float2 (&d)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 l, h, one;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "mov.b16 one, 0x3F80;\n\t"
        "fma.rn.f32.bf16 %0, l, one, %3;\n\t"
        "fma.rn.f32.bf16 %1, h, one, %3;\n\t}"
        : "=f"(d[i].x), "=f"(d[i].y)
        : "r"(w[i]), "f"(-o));
}

// log2(e) / temperature in two parts, hi rounded down and lo > 0 (so that -inf
// stays -inf): one part alone is off by up to 2^-24, which every row's sum would
// carry the same way and a sequence's sum of log-probabilities would add up.
struct Scale {
  float hi, lo;
};
// exp of a scaled difference of logits (the exponent rounded once)
__device__ __forceinline__ float term(float d, const Scale& c) {
  return ex2(fmaf(d, c.hi, __fmul_rn(d, c.lo)));
}
// ex2.approx reads low by 5.0e-8 on average over every octave (2^20 arguments
// each on a GB300; largest error 1.4e-7), and is exact at 0.  A row's many terms
// share that, each rescaling of a sum adds its own, and the log-probabilities of a
// whole sequence would add it up.  So raise and log_sum put back what rows show of it,
// 3.8e-8 (4096 rows each of 1000 to 65536 normal logits, bf16 and fp32, at four
// temperatures: logp off by 4e-8 to 1.3e-7 on average without, by 6e-9 with, at most
// 2e-8; with 5.0e-8 by 2 to 6e-8 the other way).
constexpr float kEx2Low = 3.8e-8f;

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

// A running maximum m with s = sum 2^((x - origin(m)) c), e what its additions rounded
// off; the origin of -inf is 0, so that rows and parts of nothing but -inf sum to
// zero.  (The dozen additions that merge a row's parts are all of the size of its
// likeliest token: without e, logp was off by 7.5e-8 rms instead of 4e-8.)
struct Run {
  float m, s, e;
};
__device__ __forceinline__ void grow(Run& r, float x, float low) {   // s + x, exactly, + low
  const float t = __fadd_rn(r.s, x), b = __fsub_rn(t, r.s);
  r.e += __fadd_rn(__fadd_rn(__fsub_rn(r.s, __fsub_rn(t, b)), __fsub_rn(x, b)), low);
  r.s = t;
}
__device__ __forceinline__ float origin(float m) { return m == kNegInf ? 0.f : m; }
__device__ __forceinline__ void raise(Run& r, float m, const Scale& c) {
  if (m > r.m) {
    const float f = term(r.m - m, c), s = __fmul_rn(r.s, f);
    r.e = fmaf(r.e, f, fmaf(s, kEx2Low, __fmaf_rn(r.s, f, -s)));
    r.s = s;
    r.m = m;
  }
}
// The warp's first N lanes merged (the others hold nothing), for all of those.
template <int N>
__device__ __forceinline__ Run warp_merge(Run r, const Scale& c) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(r.m));
  raise(r, m, c);
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const float s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o), e = __shfl_xor_sync(0xFFFFFFFFu, r.e, o);
    grow(r, s, e);
  }
  r.m = m;
  return r;
}
// Warp 0's first eight lanes get the CTA's.  part: shared, one per warp, of which
// there are at most eight.
__device__ __forceinline__ Run cta_merge(Run r, const Scale& c, Run* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  r = warp_merge<32>(r, c);
  if (blockDim.x == 32) {
    __syncwarp();
    return r;
  }
  if (lane == 0) part[warp] = r;
  __syncthreads();
  if (warp == 0)
    r = warp_merge<8>(lane < (int)(blockDim.x >> 5) ? part[lane] : Run{kNegInf, 0.f, 0.f}, c);
  return r;
}
// Sum of b's terms, two at a time.
template <typename TX, int U>
__device__ __forceinline__ float sum_batch(const uint4 (&b)[U], float o, const Scale& c) {
  constexpr int H = Elem<TX>::kPerVec / 2;
  const float2 hi = make_float2(c.hi, c.hi), lo = make_float2(c.lo, c.lo);
  float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < U; ++k) {
    float2 d[H];
    differences(b[k], o, d);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float2 a = fma2(d[i], hi, mul2(d[i], lo));
      s[i & 1] = add2(s[i & 1], make_float2(ex2(a.x), ex2(a.y)));
    }
  }
  const float2 t = add2(s[0], s[1]);
  return t.x + t.y;
}
// The gradient -g p_j, as coef 2^((x_j - o) c + l2), and g (1 - p) at the target.  (The
// exponential may be off by 2^-24 of its exponent; `fine`: the exponent takes both
// parts of the scale, for an o that may be far from the row's maximum.)
struct Grad {
  float coef, o, l2, at, g;
  Scale c;
};
template <bool FINE>
__device__ __forceinline__ float gradient_one(float x, const Grad& d) {
  const float z = __fadd_rn(x, -d.o);
  const float a = FINE ? __fmaf_rn(z, d.c.lo, __fmaf_rn(z, d.c.hi, d.l2)) : __fmul_rn(z, d.c.hi);
  return __fmul_rn(d.coef, ex2(a));
}
template <typename TX, bool FINE>
__device__ __forceinline__ void put_one(TX* to, float x, const Grad& d, bool target) {
  st_scalar(to, d.g == 0.f ? 0.f : target ? d.at : gradient_one<FINE>(x, d));
}
// A vector of it, for g other than 0; place: the target's element, or out of
// range.
template <typename TX, bool FINE>
__device__ __forceinline__ uint4 gradient(const uint4& b, const Grad& d, int place) {
  constexpr int E = Elem<TX>::kPerVec;
  float q[E];
  float2 z[E / 2];
  differences(b, d.o, z);
  const float2 hi = make_float2(d.c.hi, d.c.hi);
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 y = z[i / 2];
    const float2 a = FINE ? fma2(y, make_float2(d.c.lo, d.c.lo),
                                 fma2(y, hi, make_float2(d.l2, d.l2)))
                          : mul2(y, hi);
    const float2 r = mul2(make_float2(ex2(a.x), ex2(a.y)), make_float2(d.coef, d.coef));
    q[i] = r.x;
    q[i + 1] = r.y;
  }
  if ((unsigned)place < (unsigned)E) {
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] = place == i ? d.at : q[i];
  }
  return pack(q);
}
template <typename TX, int U>
__device__ __forceinline__ void add_batch(Run& r, const uint4 (&b)[U], const Scale& c) {
  raise(r, max_of(b, static_cast<TX*>(nullptr)), c);
  grow(r, sum_batch<TX>(b, origin(r.m), c), 0.f);
}
__device__ __forceinline__ void add_one(Run& r, float q, const Scale& c) {
  raise(r, q, c);
  grow(r, term(q - origin(r.m), c), 0.f);
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

// A value in two fp32 parts, some 45 bits, on the fp32 pipe: the fp64 pipe has two
// lanes a clock for all of an SM's rows, which bounds short ones.  The low part of a
// value that is not finite is 0.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ float finite_or_0(float x) {
  return fabsf(x) < CUDART_INF_F ? x : 0.f;
}
__device__ __forceinline__ Two two_sum(float a, float b, float low) {   // a + b, exactly, + low
  const float h = __fadd_rn(a, b), t = __fsub_rn(h, a);
  const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(h, t)), __fsub_rn(b, t));
  return Two{h, finite_or_0(__fadd_rn(e, low))};
}
__device__ __forceinline__ float value_of(const Two& v) { return __fadd_rn(v.hi, v.lo); }
__device__ __forceinline__ Two minus(const Two& a, const Two& b) {
  return two_sum(a.hi, -b.hi, __fsub_rn(a.lo, b.lo));
}
// v times the temperature's inverse
__device__ __forceinline__ Two scaled(const Two& v, const LossParams& p) {
  const float h = __fmul_rn(v.hi, p.inv_tf);
  const float e = __fmaf_rn(v.hi, p.inv_tf, -h);
  return Two{h, finite_or_0(__fmaf_rn(v.lo, p.inv_tf, __fmaf_rn(v.hi, p.inv_tlo, e)))};
}

// log(s), and what ex2.approx reads low put back (kEx2Low).  The exponent times
// the high part of ln 2 (15 bits) is exact, and the mantissa, in [0.75, 1.5), has a
// logarithm small enough that its rounding is below 2^-25.
__device__ __forceinline__ Two log_sum(const Run& r) {
  const float s = r.s;
  if (!(s > 0.f) || !(s < CUDART_INF_F)) return Two{logf(s), 0.f};
  constexpr float kLn2Hi = 0.693145751953125f, kLn2Lo = 1.428606765330187e-06f;
  const uint32_t b = __float_as_uint(s);
  const int e = (int)(b - 0x3F400000u) >> 23;   // 0x3F400000: 0.75
  const float f = logf(__uint_as_float(b - ((uint32_t)e << 23)));
  const float inv = __fdividef(1.f, s);
  return two_sum((float)e * kLn2Hi, f,
                 fmaf((float)e, kLn2Lo, fmaf(r.e, inv, kEx2Low * (1.f - inv))));
}

// What the losses need of a row besides its sums: loaded at the row's start and
// not touched (no conversion, no comparison, which would wait) before its end.
struct RowIn {
  float old_logp, ref_logp, advantage, weight;
  int64_t begin, end;             // preference: the rows that belong to sequences
};
template <int MODE>
__device__ __forceinline__ RowIn row_in(const LossParams& p, int64_t row) {
  RowIn in{};
  if (MODE == kLossPolicy || MODE == kLossPolicyGrad) {
    in.weight = 1.f;
    if (p.weights) in.weight = p.weights[row];
    in.advantage = p.advantages[row];
    in.old_logp = p.old_logp[row];
  }
  if (MODE == kLossPreference) {
    in.begin = p.cu[0];
    in.end = p.cu[2 * p.pairs];
  }
  if (MODE != kLossLogprob && p.ref_logp) in.ref_logp = p.ref_logp[row];
  return in;
}

struct PolicyTerm {
  float loss, slope;   // of the row, times its weight
};
__device__ __forceinline__ PolicyTerm policy_term(const LossParams& p, const RowIn& in,
                                                  const Two& logp) {
  const float w = in.weight, A = in.advantage;
  if (w == 0.f) return PolicyTerm{0.f, 0.f};
  const float r = expf(value_of(minus(logp, Two{in.old_logp, 0.f})));
  const bool up = A >= 0.f && r > p.ratio_hi, down = A < 0.f && r < p.ratio_lo;
  float loss = -A * (up ? p.ratio_hi : down ? p.ratio_lo : r);
  float slope = up || down ? 0.f : -A * r;
  if (p.ref_logp) {
    const float d = value_of(minus(Two{in.ref_logp, 0.f}, logp)), e = expm1f(d);
    loss = fmaf(p.kl, e - d, loss);
    slope = fmaf(-p.kl, e, slope);
  }
  return PolicyTerm{w * loss, w * slope};
}

// What one thread does with a row's maximum and sum and its target's logit xt
// (NaN for a target past the row): its results, and (policy
// with the gradient) what the row's gradient needs.  Several CTAs may call it for
// the same row; `write` says which of them stores.
template <int MODE>
__device__ __forceinline__ Grad finish_row(const LossParams& p, int64_t row, const Run& r,
                                           float xt, const RowIn& in, bool write) {
  Grad row_grad{};
  const Two ls = log_sum(r);
  const Two logp = minus(scaled(two_sum(xt, -r.m, 0.f), p), ls);
  if (write) {
    p.logp[row] = value_of(logp);
    p.lse[row] = -value_of(logp);
  }
  if (MODE == kLossPolicy || MODE == kLossPolicyGrad) {
    const PolicyTerm q = policy_term(p, in, logp);
    if (write) {
      p.token_loss[row] = q.loss;
      p.dlogp[row] = q.slope;
    }
    const float g = q.slope * p.inv_tf;
    if (MODE == kLossPolicyGrad)
      row_grad = Grad{g == 0.f ? 0.f : __fdividef(-g, r.s), origin(r.m), 0.f,
                     -g * expm1f(value_of(logp)), g, Scale{p.c_hi, p.c_lo}};
  }
  if (MODE == kLossPreference && write)
    p.dlogp[row] = row >= in.begin && row < in.end
                       ? value_of(minus(logp, Two{in.ref_logp, 0.f})) : 0.f;
  return row_grad;
}
template <int MODE>
__device__ __forceinline__ void left_out(const LossParams& p, int64_t row) {
  p.logp[row] = 0.f;
  p.lse[row] = 0.f;
  if (MODE != kLossLogprob) p.dlogp[row] = 0.f;
  if (MODE == kLossPolicy || MODE == kLossPolicyGrad) p.token_loss[row] = 0.f;
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_addr(const void* local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---------------------------------------------------------------- row kernel

template <typename TX, int MODE, int CL>
__global__ void __launch_bounds__(kLossThreads, 4) loss_row_kernel(LossParams p) {
  constexpr int E = Elem<TX>::kPerVec, U = kLossBatch;
  __shared__ Run part[32];
  __shared__ float4 peers[8];
  pdl_begin();
  const int64_t row = blockIdx.x / CL;
  const int rank = CL > 1 ? (int)cta_rank() : 0;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t t = p.targets[row];
  const bool first = rank == 0, last = rank == CL - 1;
  if (t < 0) {   // the row takes no part
    if (first && tid == 0) left_out<MODE>(p, row);
    return;
  }
  if (CL > 1) cluster_arrive();
  const TX* x = static_cast<const TX*>(p.logits) + row * p.ld;
  const Frame f = frame_of(x, p.V);
  const int v0 = CL > 1 ? (int)((int64_t)f.nvec * rank / CL) : 0;
  const int v1 = CL > 1 ? (int)((int64_t)f.nvec * (rank + 1) / CL) : f.nvec;
  const TX* xv = x + f.head;
  RowIn in{};
  TX xt{};
  if (first && tid == 0) {
    in = row_in<MODE>(p, row);
    if (t < p.V) xt = x[t];
  }

  Run r{kNegInf, 0.f, 0.f};
  const Scale c{p.c_hi, p.c_lo};
  int v = v0 + tid;
  for (; v - tid + U * nt <= v1; v += U * nt) {   // whole batches
    uint4 b[U];
#pragma unroll
    for (int k = 0; k < U; ++k) b[k] = ld_stream(xv + (size_t)(v + k * nt) * E);
    add_batch<TX>(r, b, c);
  }
  if (v - tid < v1) {
    uint4 b[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      b[k] = v + k * nt < v1 ? ld_stream(xv + (size_t)(v + k * nt) * E) : neg_inf_vec<TX>();
    add_batch<TX>(r, b, c);
  }
  if (first)
    for (int j = tid; j < f.head; j += nt) add_one(r, ld_scalar(x + j), c);
  if (last)
    for (int j = f.tail0 + tid; j < p.V; j += nt) add_one(r, ld_scalar(x + j), c);
  r = cta_merge(r, c, part);
  if (CL > 1) {
    cluster_wait();   // the first CTA has started
    if (tid == 0)
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                       peer_addr(peers + rank, 0)),
                   "f"(r.m), "f"(r.s), "f"(r.e), "f"(0.f)
                   : "memory");
    cluster_arrive();
    if (!first) return;
    cluster_wait();
    if (tid < 32) {
      const float4 q = tid < CL ? peers[tid] : make_float4(kNegInf, 0.f, 0.f, 0.f);
      r = warp_merge<CL>(Run{q.x, q.y, q.z}, c);
    }
  }
  if (first && tid == 0)
    finish_row<MODE>(p, row, r, t < p.V ? Elem<TX>::to_f32(xt) : CUDART_NAN_F, in, true);
}

// ---------------------------------------------------------------- loss and gradient

__device__ __forceinline__ void copy_async16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The policy loss with the logits' gradient: clusters of CL CTAs of NT threads
// walk the rows, each CTA with its part of every row.  A thread copies the vectors
// it will read itself into its own slots of a shared-memory ring of S batches, on
// past the end of a row, so that loads stay in flight while a row's sums are
// merged and its loss is worked out.  No barrier guards the ring: a thread waits
// for its own copies only.
//
// A row is gone over twice, the second time backwards: its last S batches are
// still in the ring -- all of them, where a CTA's part is no longer -- and only what
// lies before them is fetched again, from L2, where it was a moment ago.  Batch i
// of a row lies in stage base + i, or base - i in every other row: the second pass
// frees the stages in the opposite order, and the next row's batches fill them so.
// Each step of either pass commits one group (an empty one where there is nothing
// to fetch), so the data a step needs is always the S-th last group.
//
// What bounds it.  DRAM would take 285 us for 4096 x 131072 bf16 with a fifth of the
// rows left out; this takes 347 (5.6 TB/s).  A CTA's passes are short, and its
// merges, the exchange with its peers and the loss between them -- some 8000 of a
// row's 25000 clocks -- leave its warps idle, so an SM needs many CTAs at different
// points: 768 threads of it (896 where the ring is shorter) in CTAs as small as a
// row's part allows, the ring of 64 bytes a thread and batch being what 227 KB hold.
// (One CTA of 1024 threads per SM with the same ring 377 us; three quarters of a row
// in the ring 362.)  An SM stores at most 32 bytes a clock, from wherever: 4.4 us for
// a row of 256 KB.
template <typename TX, int NT, int CL, int S>
__global__ void __launch_bounds__(NT, 896 / NT) loss_stream_kernel(LossParams p) {
  constexpr int MODE = kLossPolicyGrad;
  constexpr int E = Elem<TX>::kPerVec, U = kLossBatch;
  extern __shared__ uint4 ring[];   // [S][U][NT]
  __shared__ Run part[2][32];
  __shared__ float4 peers[2][8];   // m, s, e and, from the CTA that has it, the target's logit
  __shared__ uint64_t bar[2];
  __shared__ float target_logit;
  __shared__ Grad row_grad;
  __shared__ int stop;
  pdl_begin();
  const int tid = threadIdx.x;
  const int rank = CL > 1 ? (int)cta_rank() : 0;
  const int64_t row0 = blockIdx.x / CL, rows = gridDim.x / CL;
  const bool first = rank == 0, last = rank == CL - 1;
  const Scale c{p.c_hi, p.c_lo};
  const TX* logits = static_cast<const TX*>(p.logits);
  TX* dlogits = static_cast<TX*>(p.dlogits);
  // rows whose gradient starts like them modulo 16 bytes take the second pass
  auto alike = [&](int64_t row) {
    return ((reinterpret_cast<uintptr_t>(logits + row * p.ld) ^
             reinterpret_cast<uintptr_t>(dlogits + row * p.ld_out)) & 15) == 0;
  };
  // this CTA's part of a row: elements [e0, e1), of which nvec vectors from v0 on
  struct Part {
    int v0, nvec, e0, e1;
  };
  auto part_of = [&](const TX* x) {
    const Frame f = frame_of(x, p.V);
    const int a = CL > 1 ? (int)((int64_t)f.nvec * rank / CL) : 0;
    const int b = CL > 1 ? (int)((int64_t)f.nvec * (rank + 1) / CL) : f.nvec;
    return Part{f.head + a * E, b - a, first ? 0 : f.head + a * E, last ? p.V : f.head + b * E};
  };
  // (whole batches without a comparison per vector)
  auto load = [&](int stage, const TX* xv, int nvec, int batch) {
    uint4* slot = ring + stage * (U * NT) + tid;
    const int v = batch * (U * NT) + tid;
    const TX* src = xv + (size_t)v * E;
    if ((batch + 1) * (U * NT) <= nvec) {
#pragma unroll
      for (int k = 0; k < U; ++k) copy_async16(slot + k * NT, src + k * NT * E);
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (v + k * NT < nvec) copy_async16(slot + k * NT, src + k * NT * E);
    }
  };
  // the targets of the row in hand and of the next two, each read two rows ahead
  auto target = [&](int64_t row) { return row < p.M ? p.targets[row] : (int64_t)-1; };
  int64_t t = target(row0), t1 = target(row0 + rows), t2;
  int64_t next = row0;   // batch i of that row, if it takes part, is what comes after this row's
  Part np{};
  auto load_next = [&](int stage, int i) {
    if (next >= 0) load(stage, logits + next * p.ld + np.v0, np.nvec, i);
  };
  auto set_next = [&](int64_t row, int64_t its_target) {
    next = its_target < 0 ? -1 : row;
    if (next >= 0) np = part_of(logits + next * p.ld);
  };
  auto wrap = [&](int stage) { return stage < 0 ? stage + S : stage >= S ? stage - S : stage; };
  if (CL > 1) {
    if (tid == 0) {
      mbar_init(bar, 1);
      mbar_init(bar + 1, 1);
      mbar_init_fence();
      stop = 0;
    }
    cluster_arrive();   // no push before every CTA's barriers are there
    cluster_wait();
  }
  set_next(row0, t);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    load_next(i, i);
    copy_commit();
  }

  int base = 0, dir = 1;
  uint32_t turn = 0;   // rows merged so far
  for (int64_t row = row0; row < p.M; row += rows, t = t1, t1 = t2) {
    t2 = target(row + 2 * rows);
    const TX* x = logits + row * p.ld;
    TX* dx = dlogits + row * p.ld_out;
    const bool twice = alike(row);
    const Part in_hand = np;
    set_next(row + rows, t1);
    if (t < 0) {   // the ring is empty: the next row's first batches
#pragma unroll
      for (int i = 0; i < S; ++i) {
        load_next(wrap(base + (dir > 0 ? i : -i)), i);
        copy_commit();
      }
      if (first && tid == 0) left_out<MODE>(p, row);
      const Part f = part_of(x);
      if (twice) {
        for (int v = tid; v < f.nvec; v += NT)
          st_stream(dx + f.v0 + (size_t)v * E, make_uint4(0, 0, 0, 0));
        for (int j = f.e0 + tid; j < f.v0; j += NT) st_scalar(dx + j, 0.f);
        for (int j = f.v0 + f.nvec * E + tid; j < f.e1; j += NT) st_scalar(dx + j, 0.f);
      } else {
        for (int j = f.e0 + tid; j < f.e1; j += NT) st_scalar(dx + j, 0.f);
      }
      continue;
    }
    const Part f = in_hand;
    const TX* xv = x + f.v0;
    int nb = (f.nvec + U * NT - 1) / (U * NT);
    if (nb < S) nb = S;   // so that the stages' order holds

    RowIn in{};
    if (tid == 0) in = row_in<MODE>(p, row);
    // the target among the vectors' elements, or out of their range; its vector's
    // batch if that is this thread's
    const bool mine = t >= f.e0 && t < f.e1;
    const int tv = mine ? (int)t - f.v0 : -1, tvec = tv < 0 ? -1 : tv / E;
    const int t_batch = tvec >= 0 && tvec < f.nvec && tvec % NT == tid ? tvec / (U * NT) : -1;
    // the elements before and behind the vectors, one a thread
    const int j_head = f.e0 + tid, j_tail = f.v0 + f.nvec * E + tid;
    const bool has_head = j_head < f.v0, has_tail = j_tail < f.e1;
    const float x_head = has_head ? ld_scalar(x + j_head) : 0.f;
    const float x_tail = has_tail ? ld_scalar(x + j_tail) : 0.f;

    Run r{kNegInf, 0.f, 0.f};
    int stage = base;
    for (int i = 0; i < nb; ++i) {
      copy_wait<S - 1>();
      const uint4* slot = ring + stage * (U * NT) + tid;
      const int v = i * (U * NT) + tid;
      uint4 b[U];
      if ((i + 1) * (U * NT) <= f.nvec) {
#pragma unroll
        for (int k = 0; k < U; ++k) b[k] = ld_shared_v4(slot + k * NT);
      } else {
#pragma unroll
        for (int k = 0; k < U; ++k)
          b[k] = v + k * NT < f.nvec ? ld_shared_v4(slot + k * NT) : neg_inf_vec<TX>();
      }
      if (i == t_batch)
        target_logit = ld_scalar(reinterpret_cast<const TX*>(slot + (tvec / NT % U) * NT) + tv % E);
      add_batch<TX>(r, b, c);
      // the stage is free, unless the second pass begins with what it holds
      if (i + S < nb) load(stage, xv, f.nvec, i + S);
      else if (!twice) load_next(stage, i + S - nb);
      copy_commit();
      stage = wrap(stage + dir);
    }
    if (has_head) add_one(r, x_head, c);
    if (has_tail) add_one(r, x_tail, c);
    if (has_head && j_head == t) target_logit = x_head;
    if (has_tail && j_tail == t) target_logit = x_tail;
    // (part is written again for the row after next, behind the next row's barriers)
    const uint32_t parity = turn & 1;
    r = cta_merge(r, c, part[parity]);
    float xt = mine ? target_logit : CL > 1 && t < p.V ? 0.f : CUDART_NAN_F;
    if (CL > 1 && tid < 32) {
      // Each CTA's (m, s) into a place of every CTA of the cluster, counted on that
      // CTA's barrier: a release at a cluster barrier would wait for this row's
      // predecessor to be stored.  A place is pushed to again two rows on, which
      // its owner allows by its push for the row between, sent after it has read.
      if (tid < CL) {
        if (tid == 0) mbar_arrive_expect_tx(bar + parity, CL * 16u);
        fence_proxy_async_smem();
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
            "[%5];" ::"r"(peer_addr(&peers[parity][rank], tid)),
            "f"(r.m), "f"(r.s), "f"(r.e), "f"(xt), "r"(peer_addr(bar + parity, tid))
            : "memory");
      }
      const bool ok = mbar_wait_bounded(bar + parity, (turn >> 1) & 1, p.wait_limit);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        // (the peers' pushes of this row land before the CTA leaves)
        mbar_wait_bounded(bar + parity, (turn >> 1) & 1, kDrainLimit);
        if (tid == 0) {
          atomicOr(p.status, kStatusWaitTimeout);
          stop = 1;
        }
      } else {
        const float4 q =
            tid < CL ? peers[parity][tid] : make_float4(kNegInf, 0.f, 0.f, 0.f);
        r = warp_merge<CL>(Run{q.x, q.y, q.z}, c);
        xt = group_sum<CL>(q.w);   // the others' are 0, or NaN all of them
      }
    }
    ++turn;
    if (tid == 0) row_grad = finish_row<MODE>(p, row, r, xt, in, first);
    __syncthreads();
    if (CL > 1 && stop) break;   // the peers give up the same way
    const Grad d = row_grad;
    if (!twice) {
      base = stage;
      for (int j = f.e0 + tid; j < f.e1; j += NT)
        put_one<TX, false>(dx + j, ld_scalar(x + j), d, j == t);
      continue;
    }
    for (int i = nb - 1; i >= 0; --i) {
      stage = wrap(stage - dir);   // where batch i lies
      copy_wait<S - 1>();
      const uint4* slot = ring + stage * (U * NT) + tid;
      const int v = i * (U * NT) + tid;
      TX* to = dx + f.v0 + (size_t)v * E;
      auto store = [&](int k) {
        st_stream(to + k * NT * E,
                  gradient<TX, false>(ld_shared_v4(slot + k * NT), d, tv - (v + k * NT) * E));
      };
      if (d.g == 0.f) {
        for (int k = 0; k < U; ++k)
          if (v + k * NT < f.nvec) st_stream(to + k * NT * E, make_uint4(0, 0, 0, 0));
      } else if ((i + 1) * (U * NT) <= f.nvec) {
#pragma unroll
        for (int k = 0; k < U; ++k) store(k);
      } else {
        for (int k = 0; k < U; ++k)
          if (v + k * NT < f.nvec) store(k);
      }
      if (i >= S) load(stage, xv, f.nvec, i - S);
      else load_next(stage, S - 1 - i);
      copy_commit();
    }
    // the next row's batch 0 went to the stage of this row's batch S - 1
    base = wrap(base - dir);
    dir = -dir;
    if (has_head) put_one<TX, false>(dx + j_head, x_head, d, j_head == t);
    if (has_tail) put_one<TX, false>(dx + j_tail, x_tail, d, j_tail == t);
  }
  copy_wait<0>();
  if (CL > 1) {   // no CTA leaves while a peer may still push to it
    cluster_arrive();
    cluster_wait();
  }
}

// ---------------------------------------------------------------- backward

// dlogits_j = g ([j = t] - p_j), g = dlogp scale / temperature, with
// p_j = exp(z_j - z_t - rel), rel the row's log-sum-exp seen from its target (minus
// logp).  The rounding of rel shows as 2^-24 |rel| in every p_j, and |rel| is small
// where p is not (a plain log-sum-exp of 20 would show 1e-6 in each, and 1 - p at a
// confident target is taken from rel by expm1, not from p).  Where the target is so
// unlikely that this would lose digits (rel > kRelFine), or has no probability at
// all, a CTA takes its row's maximum and sum again and uses those.
//
// A CTA takes kLossBatch vectors a thread of a row -- or (p.whole_rows: dlogits is logits, whose
// target another CTA might overwrite) a whole row.  Rows that take no part and
// rows whose g is zero are zeroed without being read.
constexpr float kRelFine = 64.f;
template <typename TX, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) loss_bwd_kernel(LossParams p) {
  constexpr int E = Elem<TX>::kPerVec, U = kLossBatch, per = U * NT;
  __shared__ Run part[32];
  __shared__ Run again;
  pdl_begin();
  const int tid = threadIdx.x;
  const int chunks = (p.V + per * E - 1) / (per * E);
  const int per_row = p.whole_rows ? 1 : chunks;
  const int64_t items = p.M * per_row;
  const float scale = (p.scale ? *p.scale : 1.f) * p.inv_tf;
  const Scale sc{p.c_hi, p.c_lo};
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / per_row;
    const int chunk = (int)(it - row * per_row);
    const int64_t t = p.targets[row];
    const float dlogp = p.dlogp_in[row], rel = p.lse[row];
    const float g = t < 0 ? 0.f : t < p.V ? dlogp * scale : CUDART_NAN_F;
    const TX* x = static_cast<const TX*>(p.logits) + row * p.ld;
    TX* dx = static_cast<TX*>(p.dlogits) + row * p.ld_out;
    const bool alike =
        ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x)) & 15) == 0;
    const bool again_sum = g != 0.f && !(rel <= kRelFine);
    if (again_sum && chunk != 0) continue;   // the row's first CTA takes all of it
    const int c0 = chunk, c1 = p.whole_rows || again_sum ? chunks : chunk + 1;
    // chunks of the row's vectors; the last one is short by the head at most, so
    // the row's `chunks` chunks cover them all
    const Frame f = frame_of(x, p.V);
    int w0 = c0 * per + tid;
    uint4 b[U];
    auto load = [&]() {
      if (g != 0.f && alike) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          if (w0 + k * NT < f.nvec)
            b[k] = ld_rw(x + f.head + (size_t)(w0 + k * NT) * E);
      }
    };
    load();   // on their way while the target's logit is
    Grad d{-g, 0.f, 0.f, 0.f, g, sc};
    if (g != 0.f) {
      const float xt = t < p.V ? ld_scalar(x + t) : CUDART_NAN_F;
      if (!again_sum) {
        d.o = xt;
        d.l2 = -rel * kLog2e;
        d.at = -g * expm1f(-rel);
      } else {
        Run r{kNegInf, 0.f, 0.f};
        for (int j = tid; j < p.V; j += NT) add_one(r, ld_scalar(x + j), sc);
        r = cta_merge(r, sc, part);
        if (tid == 0) again = r;
        __syncthreads();
        d.coef = -g / again.s;
        d.o = origin(again.m);
        d.at = g + gradient_one<true>(xt, d);
      }
      if (p.whole_rows || again_sum)
        __syncthreads();   // xt has been read; and `part`, `again` before another item
    }
    if (!alike) {
      const int e1 = min((int64_t)p.V, (int64_t)c1 * per * E);
      for (int j = c0 * per * E + tid; j < e1; j += NT)
        put_one<TX, true>(dx + j, g == 0.f ? 0.f : ld_scalar(x + j), d, j == t);
      continue;
    }
    const int tv = t < p.V ? (int)t - f.head : -1;   // the target among the vectors' elements
    for (;;) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int w = w0 + k * NT;
        if (w >= f.nvec) break;
        st_stream(dx + f.head + (size_t)w * E,
                  g == 0.f ? make_uint4(0, 0, 0, 0) : gradient<TX, true>(b[k], d, tv - w * E));
      }
      w0 += per;
      if (w0 >= c1 * per) break;
      load();
    }
    if (chunk == 0) {
      auto element = [&](int j) {
        put_one<TX, true>(dx + j, g == 0.f ? 0.f : ld_scalar(x + j), d, j == t);
      };
      for (int j = tid; j < f.head; j += NT) element(j);
      for (int j = f.tail0 + tid; j < p.V; j += NT) element(j);
    }
  }
}

#if RMSN_PAIR == 0
// ---------------------------------------------------------------- sums over rows

constexpr int kSumThreads = 1024;

// A sum in two fp32 parts: each addition's rounding error is exact and goes to
// the low part, so the sum has some 45 bits -- on the fp32 pipe (in fp64 it made a
// policy loss over 4096 rows 16 us longer).
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ void add(Sum2& s, float x, float low = 0.f) {
  const float t = __fadd_rn(s.hi, x), b = __fsub_rn(t, s.hi);
  const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b));
  // (an infinite or NaN sum stays what it is: its error term is NaN)
  s.lo = __fadd_rn(s.lo, fabsf(t) < CUDART_INF_F ? __fadd_rn(e, low) : 0.f);
  s.hi = t;
}
__device__ __forceinline__ float value_of(const Sum2& s) { return s.hi + s.lo; }

// Sum over groups of `n` lanes (a power of two) in a fixed order; all of them get it.
__device__ __forceinline__ Sum2 lanes_sum2(Sum2 v, int n) {
  for (int o = n / 2; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xFFFFFFFFu, v.hi, o);
    const float lo = __shfl_xor_sync(0xFFFFFFFFu, v.lo, o);
    add(v, hi, lo);
  }
  return v;
}
// Sum over groups of `warps` warps (a power of two) in a fixed order; every thread
// gets its group's.
__device__ __forceinline__ Sum2 warps_sum2(Sum2 v, float2* red, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = lanes_sum2(v, 32);
  __syncthreads();   // earlier readers of red are done
  if (lane == 0) red[warp] = make_float2(v.hi, v.lo);
  __syncthreads();
  const float2 q = red[(warp & -warps) + (lane & (warps - 1))];
  return lanes_sum2(Sum2{q.x, q.y}, warps);
}
__device__ __forceinline__ Sum2 cta_sum2(Sum2 v, float2* red) {
  return warps_sum2(v, red, blockDim.x >> 5);
}

__global__ void __launch_bounds__(kSumThreads) loss_sum_kernel(LossParams p) {
  __shared__ float2 red[32];
  pdl_begin();
  Sum2 s{0.f, 0.f};
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < p.M; i += kSumThreads) add(s, p.token_loss[i]);
  s = cta_sum2(s, red);
  if (threadIdx.x == 0) *p.loss = value_of(s);
}

// Rows [a, b) of sequence s, kept inside the batch whatever the offsets say.
__device__ __forceinline__ void rows_of(const LossParams& p, int64_t s, int64_t* a, int64_t* b) {
  *a = min(max(p.cu[s], (int64_t)0), p.M);
  *b = min(max(p.cu[s + 1], *a), p.M);
}

// log(1 + exp(x))
__device__ __forceinline__ float softplus(float x) {
  return (x < 0.f ? 0.f : x) + log1pf(expf(-fabsf(x)));   // (a NaN stays)
}
// A pair's loss; a part of weight 0 is left out: its softplus may be infinite.
__device__ __forceinline__ float pair_loss(const LossParams& p, float h) {
  float s = 0.f;
  if (p.smoothing < 1.f) s = (1.f - p.smoothing) * softplus(-h);
  if (p.smoothing > 0.f) s = fmaf(p.smoothing, softplus(h), s);
  return s;
}

// Pair b, by `n` threads of which this is the i-th: its rows' logp - ref, which the
// row kernel left in dlogp, summed with their sign ...
struct PairRows {
  int64_t a[2], e[2];
};
__device__ __forceinline__ PairRows pair_rows(const LossParams& p, int64_t b) {
  PairRows r;
  for (int side = 0; side < 2; ++side) rows_of(p, b + side * p.pairs, &r.a[side], &r.e[side]);
  return r;
}
__device__ __forceinline__ Sum2 pair_sum(const LossParams& p, const PairRows& r, int i, int n) {
  Sum2 sum{0.f, 0.f};
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (int64_t k = r.a[side] + i; k < r.e[side]; k += n)
      add(sum, side ? -p.dlogp[k] : p.dlogp[k]);
  return sum;
}
// ... and, with margin h = beta times that sum, dlogp itself.
__device__ __forceinline__ void pair_slopes(const LossParams& p, const PairRows& r, float h, int i,
                                            int n) {
  const float slope = (p.smoothing / (1.f + expf(-h)) - (1.f - p.smoothing) / (1.f + expf(h))) *
                      (p.beta / (float)p.pairs);
  for (int side = 0; side < 2; ++side)
#pragma unroll 4
    for (int64_t k = r.a[side] + i; k < r.e[side]; k += n)
      p.dlogp[k] = p.targets[k] < 0 ? 0.f : side ? -slope : slope;
}

__global__ void __launch_bounds__(kLossThreads) loss_pairs_kernel(LossParams p) {
  __shared__ float2 red[32];
  pdl_begin();
  const PairRows r = pair_rows(p, blockIdx.x);
  const float h =
      p.beta * value_of(cta_sum2(pair_sum(p, r, threadIdx.x, kLossThreads), red));
  if (threadIdx.x == 0) p.margins[blockIdx.x] = h;
  pair_slopes(p, r, h, threadIdx.x, kLossThreads);
}

__global__ void __launch_bounds__(kLossThreads) loss_pairs_mean_kernel(LossParams p) {
  __shared__ float2 red[32];
  pdl_begin();
  Sum2 s{0.f, 0.f};
  for (int64_t b = threadIdx.x; b < p.pairs; b += kLossThreads) add(s, pair_loss(p, p.margins[b]));
  s = cta_sum2(s, red);
  if (threadIdx.x == 0) *p.loss = value_of(s) / (float)p.pairs;
}

// All pairs in one CTA: a group of its warps takes one pair at a time.
__global__ void __launch_bounds__(kSumThreads) loss_pairs_all_kernel(LossParams p) {
  __shared__ float2 red[32];
  constexpr int W = kSumThreads / 32;
  pdl_begin();
  int group = W;   // warps per pair
  while (group > 1 && W / group < p.pairs) group /= 2;
  const int warp = threadIdx.x >> 5;
  const int i = threadIdx.x % (32 * group), n = 32 * group;
  Sum2 losses{0.f, 0.f};
  for (int64_t b0 = 0; b0 < p.pairs; b0 += W / group) {
    const int64_t b = b0 + warp / group;
    PairRows r{};
    if (b < p.pairs) r = pair_rows(p, b);
    const float h = p.beta * value_of(warps_sum2(pair_sum(p, r, i, n), red, group));
    if (b < p.pairs) {
      pair_slopes(p, r, h, i, n);
      if (i == 0) {
        p.margins[b] = h;
        add(losses, pair_loss(p, h));
      }
    }
  }
  losses = cta_sum2(losses, red);
  if (threadIdx.x == 0) *p.loss = value_of(losses) / (float)p.pairs;
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
LossKernel pick_stream(int cluster, int threads, int stages) {
  if (stages != loss_stages(threads)) return nullptr;
  switch (cluster * 1000 + threads) {
    case 1032: return loss_stream_kernel<TX, 32, 1, loss_stages(32)>;
    case 1064: return loss_stream_kernel<TX, 64, 1, kLossStages>;
    case 1128: return loss_stream_kernel<TX, 128, 1, kLossStages>;
    case 1256: return loss_stream_kernel<TX, 256, 1, kLossStages>;
    case 2128: return loss_stream_kernel<TX, 128, 2, kLossStages>;
    case 4128: return loss_stream_kernel<TX, 128, 4, kLossStages>;
    case 8128: return loss_stream_kernel<TX, 128, 8, kLossStages>;
    case 2256: return loss_stream_kernel<TX, 256, 2, kLossStages>;
    case 4256: return loss_stream_kernel<TX, 256, 4, kLossStages>;
    case 8256: return loss_stream_kernel<TX, 256, 8, kLossStages>;
    default: return nullptr;
  }
}
template <typename TX>
LossKernel pick_bwd(int threads) {
  switch (threads) {
    case 32: return loss_bwd_kernel<TX, 32>;
    case 64: return loss_bwd_kernel<TX, 64>;
    case 128: return loss_bwd_kernel<TX, 128>;
    default: return loss_bwd_kernel<TX, 256>;
  }
}
template <typename TX>
LossKernel pick_mode(int mode, int cluster, int threads, int stages) {
  switch (mode) {
    case kLossLogprob: return pick_row<TX, kLossLogprob>(cluster);
    case kLossPolicy: return pick_row<TX, kLossPolicy>(cluster);
    case kLossPolicyGrad: return pick_stream<TX>(cluster, threads, stages);
    case kLossPreference: return pick_row<TX, kLossPreference>(cluster);
    default: return nullptr;
  }
}

}  // namespace

#if RMSN_PAIR == 0
LossKernel get_loss_rows_f32(int mode, int cluster, int threads, int stages) {
  return pick_mode<float>(mode, cluster, threads, stages);
}
LossKernel get_loss_bwd_f32(int threads) { return pick_bwd<float>(threads); }
LossKernel get_loss_sum() { return loss_sum_kernel; }
LossKernel get_loss_pairs() { return loss_pairs_kernel; }
LossKernel get_loss_pairs_all() { return loss_pairs_all_kernel; }
LossKernel get_loss_pairs_mean() { return loss_pairs_mean_kernel; }
#else
LossKernel get_loss_rows_bf16(int mode, int cluster, int threads, int stages) {
  return pick_mode<bf16>(mode, cluster, threads, stages);
}
LossKernel get_loss_bwd_bf16(int threads) { return pick_bwd<bf16>(threads); }
#endif

}  // namespace rmsn
