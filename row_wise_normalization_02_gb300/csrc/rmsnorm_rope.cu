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

// Vectors of E elements: 16 bytes, or 8, 4 or 2 where rows, strides or halves do
// not fall on 16.
template <int B> struct Raw;
template <> struct Raw<16> { uint4 v; };
template <> struct Raw<8> { uint2 v; };
template <> struct Raw<4> { uint32_t v; };
template <> struct Raw<2> { uint16_t v; };

__device__ __forceinline__ void unpack_raw(const Raw<16>& r, float (&f)[4]) { unpack(r.v, f); }
__device__ __forceinline__ void unpack_raw(const Raw<16>& r, float (&f)[8]) { unpack(r.v, f); }
__device__ __forceinline__ void unpack_raw(const Raw<8>& r, float (&f)[2]) {
  f[0] = __uint_as_float(r.v.x);
  f[1] = __uint_as_float(r.v.y);
}
__device__ __forceinline__ void unpack_raw(const Raw<8>& r, float (&f)[4]) {
  unpack_word_bf16(r.v.x, f[0], f[1]);
  unpack_word_bf16(r.v.y, f[2], f[3]);
}
__device__ __forceinline__ void unpack_raw(const Raw<4>& r, float (&f)[1]) {
  f[0] = __uint_as_float(r.v);
}
__device__ __forceinline__ void unpack_raw(const Raw<4>& r, float (&f)[2]) {
  unpack_word_bf16(r.v, f[0], f[1]);
}
__device__ __forceinline__ void unpack_raw(const Raw<2>& r, float (&f)[1]) {
  f[0] = __uint_as_float((uint32_t)r.v << 16);
}

// Streaming stores of a vector.
__device__ __forceinline__ void store_vec(void* p, const float (&f)[8], bf16*) {
  st_stream(p, pack(f));
}
__device__ __forceinline__ void store_vec(void* p, const float (&f)[4], float*) {
  st_stream(p, pack(f));
}
__device__ __forceinline__ void store_words(void* p, uint32_t a, uint32_t b) {
  asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void store_word(void* p, uint32_t a) {
  asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(p), "r"(a) : "memory");
}
__device__ __forceinline__ void store_vec(void* p, const float (&f)[4], bf16*) {
  store_words(p, pack_word_bf16(f[0], f[1]), pack_word_bf16(f[2], f[3]));
}
__device__ __forceinline__ void store_vec(void* p, const float (&f)[2], bf16*) {
  store_word(p, pack_word_bf16(f[0], f[1]));
}
__device__ __forceinline__ void store_vec(void* p, const float (&f)[1], bf16*) {
  st_scalar(static_cast<bf16*>(p), f[0]);
}
__device__ __forceinline__ void store_vec(void* p, const float (&f)[2], float*) {
  store_words(p, __float_as_uint(f[0]), __float_as_uint(f[1]));
}
__device__ __forceinline__ void store_vec(void* p, const float (&f)[1], float*) {
  store_word(p, __float_as_uint(f[0]));
}

// Global -> shared copy of one vector, which the copying thread reads back itself
// after copy_wait: no barrier.  (Two bytes have no asynchronous form.)
__device__ __forceinline__ void copy_vec(Raw<16>* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_vec(Raw<8>* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_vec(Raw<4>* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_vec(Raw<2>* dst, const void* src) {
  dst->v = *static_cast<const volatile uint16_t*>(src);
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Read of a slot, not to be moved over the copies around it.
template <int B>
__device__ __forceinline__ Raw<B> slot_of(const Raw<B>* p) {
  Raw<B> r;
  if constexpr (B == 16) {
    r.v = ld_shared_v4(p);
  } else if constexpr (B == 8) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(r.v.x), "=r"(r.v.y) : "r"(smem_addr(p)));
  } else if constexpr (B == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.v) : "r"(smem_addr(p)));
  } else {
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r.v) : "r"(smem_addr(p)));
  }
  return r;
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
// lie side by side in a, then in b (single elements: a with b again).
template <int E, bool ADJ>
__device__ __forceinline__ void rotate(float (&a)[E], float (&b)[E], const float2 (&cs)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    constexpr bool kSide = ADJ && E > 1;
    float* u = kSide ? (i < E / 2 ? &a[2 * i] : &b[2 * i - E]) : &a[i];
    float* v = kSide ? u + 1 : &b[i];
    const float x = *u, y = *v;
    *u = x * cs[i].x - y * cs[i].y;
    *v = x * cs[i].y + y * cs[i].x;
  }
}

template <typename TX, typename TW, int E>
__device__ __forceinline__ void load_gamma(const void* gamma, int vec, float (&w)[E]) {
  const TW* g = static_cast<const TW*>(gamma) + (size_t)vec * E;
  if constexpr (E * sizeof(TX) < 16) {
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = ld_scalar_ro(g + i);
  } else if constexpr (sizeof(TW) * E == 16) {
    unpack(ld_cached(g), w);
  } else {   // bf16 activations with fp32 weights
    float lo[4], hi[4];
    unpack(ld_cached(g), lo);
    unpack(ld_cached(g + 4), hi);
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

// The warp's angles of token t, one frequency per lane and step ...
__device__ __forceinline__ void warp_angles(const RopeParams& p, int64_t t, float2* table) {
  __syncwarp();   // the previous token's readers are done
  for (int i = threadIdx.x & 31; i < p.R / 2; i += 32) table[i] = angle(p, t, i);
  __syncwarp();
}
// ... and a unit's E of them.
template <int E>
__device__ __forceinline__ void unit_angles(const float2* table, int u, bool rotary,
                                            float2 (&cs)[E]) {
  if constexpr (E == 1) {
    cs[0] = rotary ? table[u] : make_float2(1.f, 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const float4 q = rotary ? *reinterpret_cast<const float4*>(table + u * E + i)
                              : make_float4(1.f, 0.f, 1.f, 0.f);
      cs[i] = make_float2(q.x, q.y);
      cs[i + 1] = make_float2(q.z, q.w);
    }
  }
}

// ---------------------------------------------------------------------------
// Forward, and the backward of the rotation alone (sign -1).  One warp per
// (token, chunk of rows); q's rows come first, k's follow.  A row is G lanes of L
// units; steps of 32 / G rows go through a ring of S steps per thread.
template <typename TX, typename TW, int E, int G, int L, bool NORM, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeParams p) {
  constexpr int RG = 32 / G, B = E * sizeof(TX), S = kRopeFwdSteps;
  using V = Raw<B>;
  extern __shared__ float4 smem4[];
  pdl_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane % G, rg = lane / G;
  V* ring = reinterpret_cast<V*>(smem4) + tid;   // [S][2 L][threads]
  float2* table = reinterpret_cast<float2*>(reinterpret_cast<V*>(smem4) +
                                            S * 2 * L * kRopeThreads) +
                  warp * ((p.R / 2 + 1) & ~1);
  const uint32_t item = blockIdx.x * (kRopeThreads / 32) + warp;
  const uint32_t t32 = item / (uint32_t)p.chunks[0];
  const int64_t t = t32;
  if (t >= p.T) return;
  const int h0 = (int)(item - t32 * (uint32_t)p.chunks[0]) * p.heads_per_chunk[0];
  const int nq = p.v[0].heads, rows = nq + p.v[1].heads;
  const int h1 = min(h0 + p.heads_per_chunk[0], rows);
  const int units = p.D / (2 * E);
  int va[L], vb[L];
#pragma unroll
  for (int k = 0; k < L; ++k) unit_vectors<E, ADJ>(p, g + k * G, &va[k], &vb[k]);
  const TX* xq = static_cast<const TX*>(p.v[0].x) + t * p.v[0].x_st;
  const TX* xk = static_cast<const TX*>(p.v[1].x) + t * p.v[1].x_st;
  TX* yq = static_cast<TX*>(p.v[0].y) + t * p.v[0].y_st;
  TX* yk = static_cast<TX*>(p.v[1].y) + t * p.v[1].y_st;

  auto load = [&](int stage, int r) {
    if (r < h1) {
      const TX* x = r < nq ? xq + r * p.v[0].x_sh : xk + (r - nq) * p.v[1].x_sh;
      V* slot = ring + stage * (2 * L * kRopeThreads);
#pragma unroll
      for (int k = 0; k < L; ++k)
        if (g + k * G < units) {
          copy_vec(slot + 2 * k * kRopeThreads, x + va[k] * E);
          copy_vec(slot + (2 * k + 1) * kRopeThreads, x + vb[k] * E);
        }
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < S; ++s) load(s, h0 + s * RG + rg);   // on their way while the angles are computed
  warp_angles(p, t, table);
  float2 cs[L][E];
#pragma unroll
  for (int k = 0; k < L; ++k)
    unit_angles<E>(table, g + k * G, g + k * G < p.R / (2 * E), cs[k]);
  int stage = 0;
  for (int r0 = h0; r0 < h1; r0 += RG) {
    const int r = r0 + rg;
    copy_wait<S - 1>();
    const V* slot = ring + stage * (2 * L * kRopeThreads);
    float a[L][E], b[L][E], ss = 0.f;
#pragma unroll
    for (int k = 0; k < L; ++k) {
      if (r < h1 && g + k * G < units) {
        unpack_raw(slot_of(slot + 2 * k * kRopeThreads), a[k]);
        unpack_raw(slot_of(slot + (2 * k + 1) * kRopeThreads), b[k]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) a[k][i] = b[k][i] = 0.f;
      }
      if (NORM) ss += sum_sq(a[k], b[k]);
    }
    load(stage, r + S * RG);
    stage = stage + 1 == S ? 0 : stage + 1;
    if (NORM) ss = rsqrtf(group_sum<G>(ss) * p.inv_d + p.eps);
    if (r >= h1) continue;
    TX* y = r < nq ? yq + r * p.v[0].y_sh : yk + (r - nq) * p.v[1].y_sh;
#pragma unroll
    for (int k = 0; k < L; ++k) {
      if (g + k * G >= units) continue;
      if (NORM) {
        const void* gamma = r < nq ? p.v[0].gamma : p.v[1].gamma;
        float w[E];
        load_gamma<TX, TW>(gamma, va[k], w);
#pragma unroll
        for (int i = 0; i < E; ++i) a[k][i] *= ss * w[i];
        load_gamma<TX, TW>(gamma, vb[k], w);
#pragma unroll
        for (int i = 0; i < E; ++i) b[k][i] *= ss * w[i];
      }
      rotate<E, ADJ>(a[k], b[k], cs[k]);
      store_vec(y + va[k] * E, a[k], static_cast<TX*>(nullptr));
      store_vec(y + vb[k] * E, b[k], static_cast<TX*>(nullptr));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward with the norm.  Persistent: each warp walks (token, chunk) items of
// q, then those of k, its lanes keeping the dgamma partials of their columns
// in registers; after each view the CTA adds its lanes' partials in a fixed
// order into its partial row.
template <typename TX, typename TW, int E, int G, int L, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_norm_bwd_kernel(RopeParams p) {
  constexpr int RG = 32 / G, W = kRopeThreads / 32, B = E * sizeof(TX), S = kRopeBwdSteps;
  using V = Raw<B>;
  extern __shared__ float4 smem4[];
  pdl_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane % G, rg = lane / G;
  const int units = p.D / (2 * E);
  int va[L], vb[L];
#pragma unroll
  for (int k = 0; k < L; ++k) unit_vectors<E, ADJ>(p, g + k * G, &va[k], &vb[k]);
  V* ring = reinterpret_cast<V*>(smem4) + tid;                        // [S][4 L][threads]
  float2* tables = reinterpret_cast<float2*>(reinterpret_cast<V*>(smem4) +
                                             S * 4 * L * kRopeThreads);
  float2* table = tables + warp * ((p.R / 2 + 1) & ~1);
  float* red = reinterpret_cast<float*>(tables + W * ((p.R / 2 + 1) & ~1));   // [W][D]
  const uint32_t nw = gridDim.x * W, w0 = blockIdx.x * W + warp;
  uint32_t skip = 0;   // items of q, so that k's start where q's ended

  for (int side = 0; side < 2; ++side) {
    const RopeView& v = p.v[side];
    if (v.heads == 0) {   // an absent view: its partial columns are zero
      if (p.partial)
        for (int d = tid; d < p.ld_half; d += kRopeThreads)
          p.partial[(size_t)blockIdx.x * 2 * p.ld_half + side * p.ld_half + d] = 0.f;
      continue;
    }
    const uint32_t chunks = (uint32_t)p.chunks[side];
    const uint32_t items = (uint32_t)p.T * chunks;
    float wa[L][E], wb[L][E], ga[L][E], gb[L][E];
#pragma unroll
    for (int k = 0; k < L; ++k) {
#pragma unroll
      for (int i = 0; i < E; ++i) wa[k][i] = wb[k][i] = ga[k][i] = gb[k][i] = 0.f;
      if (g + k * G < units) {
        load_gamma<TX, TW>(v.gamma, va[k], wa[k]);
        load_gamma<TX, TW>(v.gamma, vb[k], wb[k]);
      }
    }
    // what comes next into the ring: a step of an item
    uint32_t f_it = (w0 + nw - skip % nw) % nw;
    int f_h = 0, f_h1 = 0;
    const TX *f_x = nullptr, *f_dy = nullptr;
    auto f_begin = [&]() {
      if (f_it >= items) return;
      const uint32_t t32 = f_it / chunks;
      f_h = (int)(f_it - t32 * chunks) * p.heads_per_chunk[side];
      f_h1 = min(f_h + p.heads_per_chunk[side], v.heads);
      f_x = static_cast<const TX*>(v.x) + (int64_t)t32 * v.x_st;
      f_dy = static_cast<const TX*>(v.dy) + (int64_t)t32 * v.dy_st;
    };
    auto load = [&](int stage) {
      if (f_it < items) {
        const int h = f_h + rg;
        if (h < f_h1) {
          const TX* xr = f_x + h * v.x_sh;
          const TX* dr = f_dy + h * v.dy_sh;
          V* slot = ring + stage * (4 * L * kRopeThreads);
#pragma unroll
          for (int k = 0; k < L; ++k)
            if (g + k * G < units) {
              copy_vec(slot + 4 * k * kRopeThreads, xr + va[k] * E);
              copy_vec(slot + (4 * k + 1) * kRopeThreads, xr + vb[k] * E);
              copy_vec(slot + (4 * k + 2) * kRopeThreads, dr + va[k] * E);
              copy_vec(slot + (4 * k + 3) * kRopeThreads, dr + vb[k] * E);
            }
        }
        f_h += RG;
        if (f_h >= f_h1) {
          f_it += nw;
          f_begin();
        }
      }
      copy_commit();
    };
    uint32_t it = f_it;
    f_begin();
#pragma unroll
    for (int s = 0; s < S; ++s) load(s);
    int stage = 0;
    for (; it < items; it += nw) {
      const uint32_t t32 = it / chunks;
      const int64_t t = t32;
      const int h0 = (int)(it - t32 * chunks) * p.heads_per_chunk[side];
      const int h1 = min(h0 + p.heads_per_chunk[side], v.heads);
      TX* yt = static_cast<TX*>(v.y) + t * v.y_st;
      warp_angles(p, t, table);
      float2 cs[L][E];
#pragma unroll
      for (int k = 0; k < L; ++k)
        unit_angles<E>(table, g + k * G, g + k * G < p.R / (2 * E), cs[k]);
      for (int hb = h0; hb < h1; hb += RG) {
        const int h = hb + rg;
        copy_wait<S - 1>();
        const V* slot = ring + stage * (4 * L * kRopeThreads);
        float a[L][E], b[L][E], da[L][E], db[L][E];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int k = 0; k < L; ++k) {
          if (h < h1 && g + k * G < units) {
            unpack_raw(slot_of(slot + 4 * k * kRopeThreads), a[k]);
            unpack_raw(slot_of(slot + (4 * k + 1) * kRopeThreads), b[k]);
            unpack_raw(slot_of(slot + (4 * k + 2) * kRopeThreads), da[k]);
            unpack_raw(slot_of(slot + (4 * k + 3) * kRopeThreads), db[k]);
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i) a[k][i] = b[k][i] = da[k][i] = db[k][i] = 0.f;
          }
          rotate<E, ADJ>(da[k], db[k], cs[k]);
          ss += sum_sq(a[k], b[k]);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            dot = fmaf(wa[k][i] * da[k][i], a[k][i], dot);
            dot = fmaf(wb[k][i] * db[k][i], b[k][i], dot);
          }
        }
        load(stage);
        stage = stage + 1 == S ? 0 : stage + 1;
        ss = group_sum<G>(ss);
        dot = group_sum<G>(dot);
        const float r = rsqrtf(ss * p.inv_d + p.eps);
        const float c = r * r * p.inv_d * dot;
        if (h >= h1) continue;
        TX* y = yt + h * v.y_sh;
#pragma unroll
        for (int k = 0; k < L; ++k) {
          if (g + k * G >= units) continue;
#pragma unroll
          for (int i = 0; i < E; ++i) {
            ga[k][i] = fmaf(da[k][i] * a[k][i], r, ga[k][i]);
            gb[k][i] = fmaf(db[k][i] * b[k][i], r, gb[k][i]);
            a[k][i] = r * fmaf(-a[k][i], c, wa[k][i] * da[k][i]);
            b[k][i] = r * fmaf(-b[k][i], c, wb[k][i] * db[k][i]);
          }
          store_vec(y + va[k] * E, a[k], static_cast<TX*>(nullptr));
          store_vec(y + vb[k] * E, b[k], static_cast<TX*>(nullptr));
        }
      }
    }
    skip += items;
    if (p.partial) {
      __syncthreads();   // the previous view's sums have been read
#pragma unroll
      for (int k = 0; k < L; ++k) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
#pragma unroll
          for (int o = G; o < 32; o <<= 1) {
            ga[k][i] += __shfl_xor_sync(0xFFFFFFFFu, ga[k][i], o);
            gb[k][i] += __shfl_xor_sync(0xFFFFFFFFu, gb[k][i], o);
          }
          if (g + k * G < units && rg == 0) {
            red[warp * p.D + va[k] * E + i] = ga[k][i];
            red[warp * p.D + vb[k] * E + i] = gb[k][i];
          }
        }
      }
      __syncthreads();
      for (int d = tid; d < p.ld_half; d += kRopeThreads) {
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

// Shapes: vectors of 16 bytes with one unit a lane, smaller ones with up to four.
template <typename TX, typename TW, bool NORM, bool ADJ>
RopeKernel pick_fwd(const RopeKey& k) {
  constexpr int E = Elem<TX>::kPerVec;
  const int id = k.e * 1000 + k.g * 10 + k.l;
  if (id == 0) return rope_scalar_kernel<TX, TW, NORM, ADJ, false>;
  if (id == E * 1000 + 41) return rope_kernel<TX, TW, E, 4, 1, NORM, ADJ>;
  if (id == E * 1000 + 81) return rope_kernel<TX, TW, E, 8, 1, NORM, ADJ>;
  if (id == E * 1000 + 161) return rope_kernel<TX, TW, E, 16, 1, NORM, ADJ>;
  if (id == E * 1000 + 321) return rope_kernel<TX, TW, E, 32, 1, NORM, ADJ>;
#define RMSN_ROPE(E_, G_, L_) \
  if (id == E_ * 1000 + G_ * 10 + L_) return rope_kernel<TX, TW, E_, G_, L_, NORM, ADJ>;
#define RMSN_ROPE_SMALL(E_) \
  RMSN_ROPE(E_, 16, 1) RMSN_ROPE(E_, 32, 1) RMSN_ROPE(E_, 32, 2) RMSN_ROPE(E_, 32, 4)
  RMSN_ROPE_SMALL(1) RMSN_ROPE_SMALL(2)
  if constexpr (E == 8) { RMSN_ROPE_SMALL(4) }
#undef RMSN_ROPE_SMALL
#undef RMSN_ROPE
  return nullptr;
}
template <typename TX, typename TW, bool ADJ>
RopeKernel pick_bwd(const RopeKey& k) {
  constexpr int E = Elem<TX>::kPerVec;
  const int id = k.e * 1000 + k.g * 10 + k.l;
  if (id == 0) return rope_scalar_kernel<TX, TW, true, ADJ, true>;
  if (id == E * 1000 + 41) return rope_norm_bwd_kernel<TX, TW, E, 4, 1, ADJ>;
  if (id == E * 1000 + 81) return rope_norm_bwd_kernel<TX, TW, E, 8, 1, ADJ>;
  if (id == E * 1000 + 161) return rope_norm_bwd_kernel<TX, TW, E, 16, 1, ADJ>;
  if (id == E * 1000 + 321) return rope_norm_bwd_kernel<TX, TW, E, 32, 1, ADJ>;
#define RMSN_ROPE(E_, G_, L_) \
  if (id == E_ * 1000 + G_ * 10 + L_) return rope_norm_bwd_kernel<TX, TW, E_, G_, L_, ADJ>;
#define RMSN_ROPE_SMALL(E_) \
  RMSN_ROPE(E_, 16, 1) RMSN_ROPE(E_, 32, 1) RMSN_ROPE(E_, 32, 2) RMSN_ROPE(E_, 32, 4)
  RMSN_ROPE_SMALL(1) RMSN_ROPE_SMALL(2)
  if constexpr (E == 8) { RMSN_ROPE_SMALL(4) }
#undef RMSN_ROPE_SMALL
#undef RMSN_ROPE
  return nullptr;
}
template <typename TX, typename TW>
RopeKernel pick(const RopeKey& k) {
  if (k.bwd) return k.adjacent ? pick_bwd<TX, TW, true>(k) : pick_bwd<TX, TW, false>(k);
  if (k.norm)
    return k.adjacent ? pick_fwd<TX, TW, true, true>(k) : pick_fwd<TX, TW, true, false>(k);
#if RMSN_PAIR == 2   // the rotation alone has no weights: the bf16/bf16 unit has it
  return nullptr;
#else
  return k.adjacent ? pick_fwd<TX, TW, false, true>(k) : pick_fwd<TX, TW, false, false>(k);
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
