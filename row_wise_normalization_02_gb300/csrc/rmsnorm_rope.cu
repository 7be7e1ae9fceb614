// Rotary positions with several axes over the heads of q and k, alone or
// behind the per-head RMSNorm, forward and backward (sm_103a).
//
//   theta(t, i) = position[axis(i)][t] * inv_freq[i],   i < R / 2
//   forward : z = x (rotation alone) or x * rstd * gamma (per head of D), then
//             the pair (u, v) of frequency i becomes
//             (u cos - v sin, u sin + v cos); columns >= R pass unchanged
//   backward: g = dy rotated by -theta; alone dx = g, with the norm
//             c = rstd^2 / D sum_k gamma_k g_k x_k,
//             dx = rstd (gamma g - x c),  dgamma = sum over rows of g x rstd
// All arithmetic is fp32 on unpacked values with one rounding of the result;
// rstd is recomputed from x, which the row's lanes hold anyway.
//
// Angles.  A position can be millions and the angle has to be right modulo one
// turn, where a 32-bit product has lost every digit.  So the frequency becomes
// a 64-bit fixed-point fraction of a turn per position,
// F = round_down(inv_freq / (2 pi) * 2^64) (freq_turns), and the product
// position * F modulo 2^64 -- an ordinary wrapping integer multiply -- IS the
// angle modulo one turn, off by at most |position| * 2^-64 turns.  Its high
// word, a signed fraction of a turn, goes to sincospif.
//
// What bounds it: memory.  Every element is read once and written once (the
// backward with the norm reads x and dy), against about 4-10 fp32 instructions
// per element.  A warp takes one token (or a chunk of its heads where tokens
// are few): its lanes compute the token's R / 2 sines and cosines once into
// the warp's shared memory, each lane takes the ones of its columns into
// registers, and the warp then walks the heads, 32 / G rows at a time.  A lane
// holds two 16-byte vectors of a row, chosen so that both halves of every pair
// are its own (columns i.. and R/2 + i.. for halves, neighbours for adjacent
// pairs): the rotation needs no exchange.
#include "rmsnorm_device.cuh"
#include "rmsnorm_internal.h"

#ifndef RMSN_PAIR
#error "compile once per dtype pair with -DRMSN_PAIR=0 (f32/f32), 1 (bf16/bf16), 2 (bf16/f32)"
#endif

namespace rmsn {
namespace {

// inv_freq / (2 pi) in units of 2^-64 turn, modulo one turn.  f = m 2^e with a
// 24-bit m, and 1 / (2 pi) = C 2^-66 with C = floor(2^65 / pi) (64 bits), so F is
// the 88-bit product m C shifted by e - 2.  Zero and values that are not finite
// give no rotation (the entry point's contract asks for finite ones).
__device__ __forceinline__ unsigned long long freq_turns(float f) {
  constexpr unsigned long long C = 0xA2F9836E4E441529ull;
  const uint32_t b = __float_as_uint(f);
  const int ex = (int)((b >> 23) & 0xFF);
  if (ex == 255) return 0;
  const uint32_t m = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int s = (ex ? ex : 1) - 150 - 2;   // F = m C 2^s
  const unsigned long long lo = (unsigned long long)m * C, hi = __umul64hi(m, C);
  unsigned long long r;
  if (s <= -128) r = 0;
  else if (s <= -64) r = hi >> (-s - 64);
  else if (s < 0) r = (hi << (64 + s)) | (lo >> -s);
  else r = s < 64 ? lo << s : 0;
  return (b >> 31) ? 0ull - r : r;
}

// Axis of frequency i: blocks of sections[a] frequencies per axis, or
// interleaved -- axis a > 0 takes the i with i % axes == a below
// sections[a] * axes, axis 0 the rest.
__device__ __forceinline__ int freq_axis(const RopeParams& p, int i) {
  if (p.order) {
    const int a = i % p.axes;
    return i < p.sections[a] * p.axes ? a : 0;
  }
  int a = 0, end = p.sections[0];
  while (a + 1 < p.axes && i >= end) end += p.sections[++a];
  return a;
}

// (cos, sign * sin) of frequency i at token t.
__device__ __forceinline__ float2 angle(const RopeParams& p, int64_t t, int i) {
  const int64_t pos = __ldg(p.positions + freq_axis(p, i) * p.pos_st + t);
  const unsigned long long turn = (unsigned long long)pos * freq_turns(__ldg(p.inv_freq + i));
  float s, c;
  sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c, p.sign * s);
}

// The two vectors of unit u of a row (see the note at the top): rotary units
// first, then the unrotated columns two neighbours at a time.
template <int E, bool ADJ>
__device__ __forceinline__ void unit_vectors(const RopeParams& p, int u, int* a, int* b) {
  const int half = p.R / (2 * E);
  if (ADJ || u >= half) {
    *a = 2 * u;
    *b = 2 * u + 1;
  } else {
    *a = u;
    *b = u + half;
  }
}

// Rotate the E pairs a unit holds: halves pair a[i] with b[i], adjacent pairs
// lie side by side in a, then in b.
template <int E, bool ADJ>
__device__ __forceinline__ void rotate(float (&a)[E], float (&b)[E], const float2 (&cs)[E],
                                       float sgn) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    float* u = ADJ ? (i < E / 2 ? &a[2 * i] : &b[2 * i - E]) : &a[i];
    float* v = ADJ ? u + 1 : &b[i];
    const float x = *u, y = *v, s = sgn * cs[i].y;
    *u = x * cs[i].x - y * s;
    *v = x * s + y * cs[i].x;
  }
}

template <typename TW, int E>
__device__ __forceinline__ void load_gamma(const void* gamma, int vec, float (&w)[E]) {
  const char* g = static_cast<const char*>(gamma) + (size_t)vec * E * sizeof(TW);
  if constexpr (sizeof(TW) * E == 16) {
    unpack(ld_cached(g), w);
  } else {   // bf16 activations with fp32 weights
    float lo[4], hi[4];
    unpack(ld_cached(g), lo);
    unpack(ld_cached(g + 16), hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = lo[i];
      w[4 + i] = hi[i];
    }
  }
}

template <int E>
__device__ __forceinline__ float sum_sq(const float (&a)[E], const float (&b)[E]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
  return s;
}

// The warp's angles of token t, one frequency per lane and step, then each
// lane's own E of them.
template <int E>
__device__ __forceinline__ void warp_angles(const RopeParams& p, int64_t t, float2* table, int u,
                                            bool rotary, float2 (&cs)[E]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the previous token's readers are done
  for (int i = lane; i < p.R / 2; i += 32) table[i] = angle(p, t, i);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float4 q = rotary ? *reinterpret_cast<const float4*>(table + u * E + i)
                            : make_float4(1.f, 0.f, 1.f, 0.f);
    cs[i] = make_float2(q.x, q.y);
    cs[i + 1] = make_float2(q.z, q.w);
  }
}

// ---------------------------------------------------------------------------
// Forward, and the backward of the rotation alone (sign -1).  One warp per
// (token, chunk of rows); q's rows come first, k's follow.
template <typename TX, typename TW, int G, bool NORM, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeParams p) {
  constexpr int E = Elem<TX>::kPerVec, RG = 32 / G;
  extern __shared__ float4 smem4[];
  pdl_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = lane % G, rg = lane / G;
  const uint32_t item = blockIdx.x * (kRopeThreads / 32) + warp;
  const uint32_t t32 = item / (uint32_t)p.chunks[0];
  const int64_t t = t32;
  if (t >= p.T) return;
  const int h0 = (int)(item - t32 * (uint32_t)p.chunks[0]) * p.heads_per_chunk[0];
  const int rows = p.v[0].heads + p.v[1].heads;
  const int h1 = min(h0 + p.heads_per_chunk[0], rows);
  const bool has = u < p.D / (2 * E);
  int va, vb;
  unit_vectors<E, ADJ>(p, u, &va, &vb);

  auto load = [&](int r, uint4* a, uint4* b) {
    if (has && r < h1) {
      const RopeView& v = p.v[r >= p.v[0].heads];
      const int h = r - (r >= p.v[0].heads ? p.v[0].heads : 0);
      const TX* x = static_cast<const TX*>(v.x) + t * v.x_st + h * v.x_sh;
      *a = ld_rw(x + va * E);
      *b = ld_rw(x + vb * E);
    } else {
      *a = *b = make_uint4(0, 0, 0, 0);
    }
  };
  uint4 na, nb;
  load(h0 + rg, &na, &nb);   // on its way while the angles are computed
  float2 cs[E];
  warp_angles<E>(p, t, reinterpret_cast<float2*>(smem4) + warp * ((p.R / 2 + 1) & ~1), u,
                 u < p.R / (2 * E), cs);
  for (int r0 = h0; r0 < h1; r0 += RG) {
    const int r = r0 + rg;
    const uint4 xa = na, xb = nb;
    load(r + RG, &na, &nb);
    float a[E], b[E];
    unpack(xa, a);
    unpack(xb, b);
    const RopeView& v = p.v[r >= p.v[0].heads];
    if (NORM) {
      const float rstd = rsqrtf(group_sum<G>(sum_sq(a, b)) * p.inv_d + p.eps);
      if (has && r < h1) {
        float w[E];
        load_gamma<TW>(v.gamma, va, w);
#pragma unroll
        for (int i = 0; i < E; ++i) a[i] *= rstd * w[i];
        load_gamma<TW>(v.gamma, vb, w);
#pragma unroll
        for (int i = 0; i < E; ++i) b[i] *= rstd * w[i];
      }
    }
    rotate<E, ADJ>(a, b, cs, 1.f);
    if (has && r < h1) {
      const int h = r - (r >= p.v[0].heads ? p.v[0].heads : 0);
      TX* y = static_cast<TX*>(v.y) + t * v.y_st + h * v.y_sh;
      st_stream(y + va * E, pack(a));
      st_stream(y + vb * E, pack(b));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward with the norm.  Persistent: each warp walks (token, chunk) items of
// q, then those of k, its lanes keeping the dgamma partials of their columns
// in registers; after each view the CTA adds its lanes' partials in a fixed
// order into its partial row.
template <typename TX, typename TW, int G, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_norm_bwd_kernel(RopeParams p) {
  constexpr int E = Elem<TX>::kPerVec, RG = 32 / G, W = kRopeThreads / 32;
  extern __shared__ float4 smem4[];
  pdl_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = lane % G, rg = lane / G;
  const bool has = u < p.D / (2 * E), rotary = u < p.R / (2 * E);
  int va, vb;
  unit_vectors<E, ADJ>(p, u, &va, &vb);
  float* red = reinterpret_cast<float*>(smem4);                       // [W][D]
  float2* table = reinterpret_cast<float2*>(red + W * p.D) + warp * ((p.R / 2 + 1) & ~1);
  const uint32_t nw = gridDim.x * W, w0 = blockIdx.x * W + warp;
  uint32_t skip = 0;   // items of q, so that k's start where q's ended

  for (int side = 0; side < 2; ++side) {
    const RopeView& v = p.v[side];
    if (v.heads == 0) {   // an absent view: its partial columns are zero
      if (p.partial)
        for (int d = threadIdx.x; d < p.ld_half; d += kRopeThreads)
          p.partial[(size_t)blockIdx.x * 2 * p.ld_half + side * p.ld_half + d] = 0.f;
      continue;
    }
    const uint32_t chunks = (uint32_t)p.chunks[side];
    const uint32_t items = (uint32_t)p.T * chunks;
    float wa[E], wb[E], ga[E], gb[E];
#pragma unroll
    for (int i = 0; i < E; ++i) wa[i] = wb[i] = ga[i] = gb[i] = 0.f;
    if (has) {
      load_gamma<TW>(v.gamma, va, wa);
      load_gamma<TW>(v.gamma, vb, wb);
    }
    for (uint32_t it = (w0 + nw - skip % nw) % nw; it < items; it += nw) {
      const uint32_t t32 = it / chunks;
      const int64_t t = t32;
      const int h0 = (int)(it - t32 * chunks) * p.heads_per_chunk[side];
      const int h1 = min(h0 + p.heads_per_chunk[side], v.heads);
      auto load = [&](int h, uint4 (&x)[2], uint4 (&d)[2]) {
        if (has && h < h1) {
          const TX* xr = static_cast<const TX*>(v.x) + t * v.x_st + h * v.x_sh;
          const TX* dr = static_cast<const TX*>(v.dy) + t * v.dy_st + h * v.dy_sh;
          x[0] = ld_rw(xr + va * E);
          x[1] = ld_rw(xr + vb * E);
          d[0] = ld_rw(dr + va * E);
          d[1] = ld_rw(dr + vb * E);
        } else {
          x[0] = x[1] = d[0] = d[1] = make_uint4(0, 0, 0, 0);
        }
      };
      uint4 nx[2], nd[2];
      load(h0 + rg, nx, nd);
      float2 cs[E];
      warp_angles<E>(p, t, table, u, rotary, cs);
      for (int hb = h0; hb < h1; hb += RG) {
        const int h = hb + rg;
        float a[E], b[E], da[E], db[E];
        unpack(nx[0], a);
        unpack(nx[1], b);
        unpack(nd[0], da);
        unpack(nd[1], db);
        load(h + RG, nx, nd);
        rotate<E, ADJ>(da, db, cs, 1.f);
        float ss = sum_sq(a, b), dot = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          dot = fmaf(wa[i] * da[i], a[i], dot);
          dot = fmaf(wb[i] * db[i], b[i], dot);
        }
        ss = group_sum<G>(ss);
        dot = group_sum<G>(dot);
        const float r = rsqrtf(ss * p.inv_d + p.eps);
        const float c = r * r * p.inv_d * dot;
        if (has && h < h1) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            ga[i] = fmaf(da[i] * a[i], r, ga[i]);
            gb[i] = fmaf(db[i] * b[i], r, gb[i]);
            a[i] = r * fmaf(-a[i], c, wa[i] * da[i]);
            b[i] = r * fmaf(-b[i], c, wb[i] * db[i]);
          }
          TX* y = static_cast<TX*>(v.y) + t * v.y_st + h * v.y_sh;
          st_stream(y + va * E, pack(a));
          st_stream(y + vb * E, pack(b));
        }
      }
    }
    skip += items;
    if (p.partial) {
      __syncthreads();   // the previous view's sums have been read
#pragma unroll
      for (int i = 0; i < E; ++i) {
#pragma unroll
        for (int o = G; o < 32; o <<= 1) {
          ga[i] += __shfl_xor_sync(0xFFFFFFFFu, ga[i], o);
          gb[i] += __shfl_xor_sync(0xFFFFFFFFu, gb[i], o);
        }
        if (has && rg == 0) {
          red[warp * p.D + va * E + i] = ga[i];
          red[warp * p.D + vb * E + i] = gb[i];
        }
      }
      __syncthreads();
      for (int d = threadIdx.x; d < p.ld_half; d += kRopeThreads) {
        float s = 0.f;
        if (d < p.D)
          for (int w = 0; w < W; ++w) s += red[w * p.D + d];
        p.partial[(size_t)blockIdx.x * 2 * p.ld_half + side * p.ld_half + d] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Scalar form of both, for rows or columns that do not fall on 16-byte vectors
// and for more than 64 of them: a CTA per (token, chunk), the angles in shared
// memory, each thread the pairs i = tid, tid + threads, ... and, behind them,
// the unrotated columns.
template <typename TX, typename TW, bool NORM, bool ADJ, bool BWD>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_kernel(RopeParams p) {
  extern __shared__ float4 smem4[];
  __shared__ float red[2 * 2 * 32];
  pdl_begin();
  float2* table = reinterpret_cast<float2*>(smem4);           // [R / 2]
  float* acc = reinterpret_cast<float*>(table + p.R / 2);     // [D], backward only
  const int half = p.R / 2, tid = threadIdx.x, nt = blockDim.x;
  int parity = 0;
  for (int side = 0; side < 2; ++side) {
    const RopeView& v = p.v[side];
    const bool sums = BWD && p.partial;
    if (sums) {
      for (int d = tid; d < p.D; d += nt) acc[d] = 0.f;
      __syncthreads();
    }
    const uint32_t chunks = (uint32_t)p.chunks[side];
    const uint32_t items = v.heads ? (uint32_t)p.T * chunks : 0u;
    for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
      const uint32_t t32 = it / chunks;
      const int64_t t = t32;
      const int h0 = (int)(it - t32 * chunks) * p.heads_per_chunk[side];
      const int h1 = min(h0 + p.heads_per_chunk[side], v.heads);
      __syncthreads();
      for (int i = tid; i < half; i += nt) table[i] = angle(p, t, i);
      __syncthreads();
      for (int h = h0; h < h1; ++h) {
        const TX* x = static_cast<const TX*>(v.x) + t * v.x_st + h * v.x_sh;
        const TX* dy = BWD ? static_cast<const TX*>(v.dy) + t * v.dy_st + h * v.dy_sh : nullptr;
        TX* y = static_cast<TX*>(v.y) + t * v.y_st + h * v.y_sh;
        const TW* w = static_cast<const TW*>(v.gamma);
        // columns (i, j) of step n: a pair, or (n >= half) one plain column
        auto columns = [&](int n, int* i, int* j) {
          if (n >= half) *i = *j = n + half;
          else if (ADJ) *i = 2 * n, *j = 2 * n + 1;
          else *i = n, *j = n + half;
        };
        // the gradient of the step's normed values: dy rotated back
        auto back = [&](int n, int i, int j, float* gi, float* gj) {
          const float a = ld_scalar(dy + i), b = ld_scalar(dy + j);
          *gi = a;
          *gj = b;
          if (n < half) {
            const float2 c = table[n];
            *gi = a * c.x - b * c.y;
            *gj = a * c.y + b * c.x;
          }
        };
        const int steps = p.D - half;
        float rstd = 1.f, c = 0.f;
        if (NORM) {
          float s[2] = {0.f, 0.f};
          for (int n = tid; n < steps; n += nt) {
            int i, j;
            columns(n, &i, &j);
            const float a = ld_scalar(x + i), b = i == j ? 0.f : ld_scalar(x + j);
            s[0] = fmaf(a, a, fmaf(b, b, s[0]));
            if (BWD) {
              float gi, gj;
              back(n, i, j, &gi, &gj);
              s[1] = fmaf(ld_scalar_ro(w + i) * gi, a, s[1]);
              s[1] = fmaf(ld_scalar_ro(w + j) * gj, b, s[1]);
            }
          }
          cta_sum<2>(s, red, parity);
          parity ^= 1;
          rstd = rsqrtf(s[0] * p.inv_d + p.eps);
          c = rstd * rstd * p.inv_d * s[1];
        }
        for (int n = tid; n < steps; n += nt) {
          int i, j;
          columns(n, &i, &j);
          float a = ld_scalar(x + i), b = ld_scalar(x + j);
          if (BWD) {
            float gi, gj;
            back(n, i, j, &gi, &gj);
            if (sums) {
              acc[i] = fmaf(gi * a, rstd, acc[i]);
              if (i != j) acc[j] = fmaf(gj * b, rstd, acc[j]);
            }
            a = rstd * fmaf(-a, c, ld_scalar_ro(w + i) * gi);
            b = rstd * fmaf(-b, c, ld_scalar_ro(w + j) * gj);
          } else {
            if (NORM) {
              a *= rstd * ld_scalar_ro(w + i);
              b *= rstd * ld_scalar_ro(w + j);
            }
            if (n < half) {
              const float2 q = table[n];
              const float a0 = a;
              a = a0 * q.x - b * q.y;
              b = a0 * q.y + b * q.x;
            }
          }
          st_scalar(y + i, a);
          if (i != j) st_scalar(y + j, b);
        }
      }
    }
    if (sums) {
      __syncthreads();
      for (int d = tid; d < p.ld_half; d += nt)
        p.partial[(size_t)blockIdx.x * 2 * p.ld_half + side * p.ld_half + d] =
            d < p.D ? acc[d] : 0.f;
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------

template <typename TX, typename TW, bool NORM, bool ADJ>
RopeKernel pick_fwd(int g) {
  switch (g) {
    case 4: return rope_kernel<TX, TW, 4, NORM, ADJ>;
    case 8: return rope_kernel<TX, TW, 8, NORM, ADJ>;
    case 16: return rope_kernel<TX, TW, 16, NORM, ADJ>;
    case 32: return rope_kernel<TX, TW, 32, NORM, ADJ>;
    case 0: return rope_scalar_kernel<TX, TW, NORM, ADJ, false>;
    default: return nullptr;
  }
}
template <typename TX, typename TW, bool ADJ>
RopeKernel pick_bwd(int g) {
  switch (g) {
    case 4: return rope_norm_bwd_kernel<TX, TW, 4, ADJ>;
    case 8: return rope_norm_bwd_kernel<TX, TW, 8, ADJ>;
    case 16: return rope_norm_bwd_kernel<TX, TW, 16, ADJ>;
    case 32: return rope_norm_bwd_kernel<TX, TW, 32, ADJ>;
    case 0: return rope_scalar_kernel<TX, TW, true, ADJ, true>;
    default: return nullptr;
  }
}
template <typename TX, typename TW>
RopeKernel pick(const RopeKey& k) {
  if (k.bwd) return k.adjacent ? pick_bwd<TX, TW, true>(k.g) : pick_bwd<TX, TW, false>(k.g);
  if (k.norm)
    return k.adjacent ? pick_fwd<TX, TW, true, true>(k.g) : pick_fwd<TX, TW, true, false>(k.g);
#if RMSN_PAIR == 2   // the rotation alone has no weights: the bf16/bf16 unit has it
  return nullptr;
#else
  return k.adjacent ? pick_fwd<TX, TW, false, true>(k.g) : pick_fwd<TX, TW, false, false>(k.g);
#endif
}

}  // namespace

#if RMSN_PAIR == 0
RopeKernel get_rope_kernel_f32_f32(const RopeKey& k) { return pick<float, float>(k); }
#elif RMSN_PAIR == 1
RopeKernel get_rope_kernel_bf16_bf16(const RopeKey& k) { return pick<bf16, bf16>(k); }
#else
RopeKernel get_rope_kernel_bf16_f32(const RopeKey& k) { return pick<bf16, float>(k); }
#endif

}  // namespace rmsn
