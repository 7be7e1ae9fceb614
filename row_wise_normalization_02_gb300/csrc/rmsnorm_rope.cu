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
// per element.  A warp takes one token (a chunk of its heads where tokens are few, a
// block of tokens where heads are): its lanes compute the R / 2 sines and cosines
// once into the warp's shared memory, each lane takes the ones of its columns into
// registers, and the warp then walks the heads, 32 / G rows at a time.  A lane
// holds L units of two vectors of a row, chosen so that both columns of every pair
// are its own (vectors of either half for halves, within a vector for adjacent
// pairs): the rotation needs no exchange.  Rows arrive by cp.async in a ring of
// which every thread reads back only what it copied itself, so that loads stay in
// flight through the arithmetic and no barrier waits for them.
#include "rmsnorm_device.cuh"
#include "rmsnorm_internal.h"
#include "rmsnorm_operators.h"

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

// (cos, sign * sin) of a position times a frequency's turns.
__device__ __forceinline__ float2 angle_of(long long pos, unsigned long long turns, float sign) {
  const unsigned long long turn = (unsigned long long)pos * turns;
  float s, c;
  sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c, sign * s);
}
// The same for frequency i at token t.
__device__ __forceinline__ float2 angle(const RopeParams& p, int64_t t, int i) {
  return angle_of(__ldg(p.positions + freq_axis(p, i) * p.pos_st + t),
                  freq_turns(__ldg(p.inv_freq + i)), p.sign);
}

// Vectors of E elements: 16 bytes, or 8, 4 or 2 where rows, strides or halves do
// not fall on 16.
template <int B> struct Raw;
template <> struct Raw<16> { uint4 v; };
template <> struct Raw<8> { uint2 v; };
template <> struct Raw<4> { uint32_t v; };
template <> struct Raw<2> { uint16_t v; };

[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<16>& r, float (&f)[4]) {
  unpack(r.v, f);
}
[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<16>& r, float (&f)[8]) {
  unpack(r.v, f);
}
[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<8>& r, float (&f)[2]) {
  f[0] = __uint_as_float(r.v.x);
  f[1] = __uint_as_float(r.v.y);
}
[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<8>& r, float (&f)[4]) {
  unpack_word_bf16(r.v.x, f[0], f[1]);
  unpack_word_bf16(r.v.y, f[2], f[3]);
}
[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<4>& r, float (&f)[1]) {
  f[0] = __uint_as_float(r.v);
}
[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<4>& r, float (&f)[2]) {
  unpack_word_bf16(r.v, f[0], f[1]);
}
[[maybe_unused]] __device__ __forceinline__ void unpack_raw(const Raw<2>& r, float (&f)[1]) {
  f[0] = __uint_as_float((uint32_t)r.v << 16);
}

// Streaming stores of a vector.
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[8], bf16*) {
  st_stream(p, pack(f));
}
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[4], float*) {
  st_stream(p, pack(f));
}
[[maybe_unused]] __device__ __forceinline__ void store_words(void* p, uint32_t a, uint32_t b) {
  asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(a), "r"(b) : "memory");
}
[[maybe_unused]] __device__ __forceinline__ void store_word(void* p, uint32_t a) {
  asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(p), "r"(a) : "memory");
}
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[4], bf16*) {
  store_words(p, pack_word_bf16(f[0], f[1]), pack_word_bf16(f[2], f[3]));
}
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[2], bf16*) {
  store_word(p, pack_word_bf16(f[0], f[1]));
}
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[1], bf16*) {
  st_scalar(static_cast<bf16*>(p), f[0]);
}
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[2], float*) {
  store_words(p, __float_as_uint(f[0]), __float_as_uint(f[1]));
}
[[maybe_unused]] __device__ __forceinline__ void store_vec(void* p, const float (&f)[1], float*) {
  store_word(p, __float_as_uint(f[0]));
}

// Global -> shared copy of one vector, which the copying thread reads back itself
// after copy_wait: no barrier.  (Two bytes have no asynchronous form.)
[[maybe_unused]] __device__ __forceinline__ void copy_vec(Raw<16>* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
[[maybe_unused]] __device__ __forceinline__ void copy_vec(Raw<8>* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
[[maybe_unused]] __device__ __forceinline__ void copy_vec(Raw<4>* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
[[maybe_unused]] __device__ __forceinline__ void copy_vec(Raw<2>* dst, const void* src) {
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

// The two vectors of unit u of a row, such that every pair is within the unit and
// lanes next to each other read next to each other.  Halves: vector u of the first
// half of the rotated columns and vector u of the second; behind them the others,
// two neighbours at a time.  Adjacent pairs lie within a vector: vectors u and u +
// units.  Single elements in adjacent pairs: 2u and 2u + 1.
template <int E, bool ADJ>
__device__ __forceinline__ void unit_vectors(const RopeParams& p, int u, int* a, int* b) {
  const int half = p.R / (2 * E);
  if (ADJ && E > 1) {
    *a = u;
    *b = u + p.D / (2 * E);
  } else if (ADJ || u >= half) {
    *a = 2 * u;
    *b = 2 * u + 1;
  } else {
    *a = u;
    *b = u + half;
  }
}

// Operations on pairs of registers, E / 2 at a time (E = 1: one).
__device__ __forceinline__ float2 pair_at(const float* a, int i) {
  return make_float2(a[i], a[i + 1]);
}
__device__ __forceinline__ void put_pair(float* a, int i, float2 v) {
  a[i] = v.x;
  a[i + 1] = v.y;
}
// o = a * b
template <int E>
__device__ __forceinline__ void mul_all(float (&o)[E], const float (&a)[E], const float (&b)[E]) {
  if constexpr (E == 1) o[0] = a[0] * b[0];
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) put_pair(o, i, __fmul2_rn(pair_at(a, i), pair_at(b, i)));
}
// o = a * s
template <int E>
__device__ __forceinline__ void scale_all(float (&o)[E], const float (&a)[E], float s) {
  if constexpr (E == 1) o[0] = a[0] * s;
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) put_pair(o, i, __fmul2_rn(pair_at(a, i), make_float2(s, s)));
}
// o += a * b
template <int E>
__device__ __forceinline__ void fma_all(float (&o)[E], const float (&a)[E], const float (&b)[E]) {
  if constexpr (E == 1) o[0] = fmaf(a[0], b[0], o[0]);
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2)
    put_pair(o, i, __ffma2_rn(pair_at(a, i), pair_at(b, i), pair_at(o, i)));
}
// o += a * s
template <int E>
__device__ __forceinline__ void axpy_all(float (&o)[E], const float (&a)[E], float s) {
  if constexpr (E == 1) o[0] = fmaf(a[0], s, o[0]);
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2)
    put_pair(o, i, __ffma2_rn(pair_at(a, i), make_float2(s, s), pair_at(o, i)));
}
// Two running sums of a * b.
template <int E>
__device__ __forceinline__ void dot_all(float2& acc, const float (&a)[E], const float (&b)[E]) {
  if constexpr (E == 1) acc.x = fmaf(a[0], b[0], acc.x);
#pragma unroll
  for (int i = 0; i + 1 < E; i += 2) acc = __ffma2_rn(pair_at(a, i), pair_at(b, i), acc);
}

// The cosines and sines of a unit's pairs.
template <int E>
struct Turn {
  float c[E], s[E];
};

// Rotate the E pairs a unit holds: halves pair a[i] with b[i], adjacent pairs
// lie side by side in a, then in b (single elements: a with b again).
template <int E, bool ADJ>
__device__ __forceinline__ void rotate(float (&a)[E], float (&b)[E], const Turn<E>& t) {
  if constexpr (ADJ && E > 1) {
    // (u, v) -> u (c, s) + v (-s, c)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float* u = i < E / 2 ? &a[2 * i] : &b[2 * i - E];
      const float2 p = __fmul2_rn(make_float2(u[1], u[1]), make_float2(-t.s[i], t.c[i]));
      put_pair(u, 0, __ffma2_rn(make_float2(u[0], u[0]), make_float2(t.c[i], t.s[i]), p));
    }
  } else {
    float n[E], x[E], y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) n[i] = -t.s[i];
    mul_all(x, b, n);
    mul_all(y, a, t.s);
    fma_all(x, a, t.c);
    fma_all(y, b, t.c);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      a[i] = x[i];
      b[i] = y[i];
    }
  }
}

// What a CTA of the vectorised kernels keeps in shared memory behind its ring: the
// frequencies as turns and their axes, and each warp's cosines and sines for the
// tokens it is at.
struct Tables {
  unsigned long long* turns;   // [R / 2]
  float2* angles;              // the warp's, [block][R / 2 rounded to 2]
  uint8_t* axis;               // [R / 2]
  int ld_angles;
};
__device__ __forceinline__ Tables make_tables(const RopeParams& p, void* at) {
  Tables t;
  const int half = p.R / 2, warps = kRopeThreads / 32;
  t.ld_angles = (half + 1) & ~1;
  t.angles = static_cast<float2*>(at);
  t.turns = reinterpret_cast<unsigned long long*>(t.angles + warps * p.block * t.ld_angles);
  t.axis = reinterpret_cast<uint8_t*>(t.turns + t.ld_angles);
  t.angles += (threadIdx.x >> 5) * p.block * t.ld_angles;
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    t.turns[i] = freq_turns(__ldg(p.inv_freq + i));
    t.axis[i] = (uint8_t)freq_axis(p, i);
  }
  __syncthreads();
  return t;
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

// Two bf16 products, exact in fp32, from the packed halves by the mixed-precision fma
// (addend -0 keeps a zero's sign) ...
__device__ __forceinline__ float2 products(uint32_t x, uint32_t w) {
  float2 r;
  asm("{\n\t.reg .b16 xl, xh, wl, wh;\n\t"
      "mov.b32 {xl, xh}, %2;\n\t"
      "mov.b32 {wl, wh}, %3;\n\t"
      "fma.rn.f32.bf16 %0, xl, wl, 0f80000000;\n\t"
      "fma.rn.f32.bf16 %1, xh, wh, 0f80000000;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(x), "r"(w));
  return r;
}
// ... and two running sums of squares.
__device__ __forceinline__ void add_squares(float2& acc, uint32_t x) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "fma.rn.f32.bf16 %0, l, l, %0;\n\t"
      "fma.rn.f32.bf16 %1, h, h, %1;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(x));
}
__device__ __forceinline__ void add_squares(float2& acc, const uint4& v) {
  add_squares(acc, v.x);
  add_squares(acc, v.y);
  add_squares(acc, v.z);
  add_squares(acc, v.w);
}
// x gamma rstd of a vector, so.
template <int E>
__device__ __forceinline__ void scale_packed(float (&o)[E], const uint4& x, const uint4& w,
                                             float rstd) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    put_pair(o, 2 * i, __fmul2_rn(products(xs[i], ws[i]), make_float2(rstd, rstd)));
}

// G lanes a row, 32 / G rows at a time: a power of two, or in the normed backward 5,
// 6 or 10, of which a warp's last two lanes have no row.
constexpr int kNoRow = 1 << 20;
// Sum over a row's lanes, in a fixed order, for all of them.
template <int G>
__device__ __forceinline__ float row_sum(float v, int g) {
  if constexpr ((G & (G - 1)) == 0) {
    return group_sum<G>(v);
  } else {
    int n = G;
#pragma unroll
    for (int o = G < 8 ? 4 : 8; o > 0; o >>= 1) {
      const float t = __shfl_down_sync(0xFFFFFFFFu, v, o);
      if (g + o < n) v += t;
      n = o;
    }
    return __shfl_sync(0xFFFFFFFFu, v, (int)(threadIdx.x & 31) - g);
  }
}
// Sum of a lane's value over the rows, in a fixed order, for the first row's lanes.
template <int G>
__device__ __forceinline__ float rows_sum(float v) {
  if constexpr ((G & (G - 1)) == 0) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  } else {
    float s = v;
#pragma unroll
    for (int r = 1; r < 32 / G; ++r) s += __shfl_down_sync(0xFFFFFFFFu, v, r * G);
    return s;
  }
}

// Lane 4 k + a holds the position of token t0 + k on axis a (of up to eight
// tokens), so that it can be asked for long before it is needed.
__device__ __forceinline__ long long lane_position(const RopeParams& p, int64_t t0, int tokens) {
  const int lane = threadIdx.x & 31, k = lane >> 2, a = lane & 3;
  return k < tokens && a < p.axes ? __ldg(p.positions + a * p.pos_st + t0 + k) : 0;
}
// The warp's angles of those tokens, one frequency per lane and step ...
__device__ __forceinline__ void warp_angles(const RopeParams& p, const Tables& tab, long long pos,
                                            int tokens) {
  const int lane = threadIdx.x & 31, half = p.R / 2;
  __syncwarp();   // the previous tokens' readers are done
  for (int k = 0; k < tokens; ++k)
    for (int i0 = 0; i0 < half; i0 += 32) {
      const int i = i0 + lane;
      const long long at = __shfl_sync(0xFFFFFFFFu, pos, 4 * k + (i < half ? tab.axis[i] : 0));
      if (i < half) tab.angles[k * tab.ld_angles + i] = angle_of(at, tab.turns[i], p.sign);
    }
  __syncwarp();
}
// ... and a unit's E of them (adjacent pairs: those of its first vector, then those
// of its second), no turn for columns from R on.
template <int N>
__device__ __forceinline__ void read_angles(const float2* table, bool rotary, float* c, float* s) {
  if constexpr (N == 1) {
    const float2 q = rotary ? table[0] : make_float2(1.f, 0.f);
    c[0] = q.x;
    s[0] = q.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 q = rotary ? *reinterpret_cast<const float4*>(table + i)
                              : make_float4(1.f, 0.f, 1.f, 0.f);
      c[i] = q.x;
      s[i] = q.y;
      c[i + 1] = q.z;
      s[i + 1] = q.w;
    }
  }
}
template <int E, bool ADJ>
__device__ __forceinline__ void unit_angles(const RopeParams& p, const float2* table, int u,
                                            Turn<E>& t) {
  if constexpr (ADJ && E > 1) {
    const int v = u + p.D / (2 * E);
    read_angles<E / 2>(table + u * (E / 2), u < p.R / E, t.c, t.s);
    read_angles<E / 2>(table + v * (E / 2), v < p.R / E, t.c + E / 2, t.s + E / 2);
  } else {
    read_angles<E>(table + u * E, u < p.R / (2 * E), t.c, t.s);
  }
}

// ---------------------------------------------------------------------------
// Forward, and the backward of the rotation alone (sign -1).  A warp takes one
// token, or a chunk of its rows where tokens are few, or a block of tokens where
// rows are; a token's rows are q's, then k's.  A row is G lanes of L units; steps of
// 32 / G rows go through a ring of S steps per thread.
template <typename TX, typename TW, int E, int G, int L, bool NORM, bool ADJ, bool BLOCK>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeParams p) {
  constexpr int RG = 32 / G, B = E * sizeof(TX), S = kRopeFwdSteps;
  using V = Raw<B>;
  extern __shared__ float4 smem4[];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // in a uniform register
  const int g = lane % G, rg = lane / G;
  V* ring = reinterpret_cast<V*>(smem4) + tid;   // [S][2 L][threads]
  const uint32_t item = blockIdx.x * (kRopeThreads / 32) + warp;
  const uint32_t group = item / (uint32_t)p.chunks[0];   // block of tokens
  const int64_t t0 = (int64_t)group * (BLOCK ? p.block : 1);
  const int tokens = (int)max((int64_t)0, min((int64_t)(BLOCK ? p.block : 1), p.T - t0));
  const int h0 = (int)(item - group * (uint32_t)p.chunks[0]) * p.heads_per_chunk[0];
  const int nq = p.v[0].heads, all = nq + p.v[1].heads;
  const int rows = min(p.heads_per_chunk[0], all - h0);   // of each token
  const int total = tokens * rows;
  const int units = p.D / (2 * E);
  int va[L], vb[L];
#pragma unroll
  for (int k = 0; k < L; ++k) unit_vectors<E, ADJ>(p, g + k * G, &va[k], &vb[k]);

  // row j of the item: head r of token t0 + k
  auto place = [&](int j, int* k, int* r) {
    *k = 0;
    *r = h0 + j;
    if (BLOCK) {
      *k = j / rows;
      *r -= *k * rows;
    }
  };
  const TX* xq = static_cast<const TX*>(p.v[0].x) + t0 * p.v[0].x_st;
  const TX* xk = static_cast<const TX*>(p.v[1].x) + t0 * p.v[1].x_st;
  TX* yq = static_cast<TX*>(p.v[0].y) + t0 * p.v[0].y_st;
  TX* yk = static_cast<TX*>(p.v[1].y) + t0 * p.v[1].y_st;
  // The lane's row of a step, RG rows further with every step (and from q to k); worked
  // out for every row where lanes hold several units (16000 tokens of 32 heads of 36
  // bf16: 26 us, stepped on 31).
  constexpr bool STEPPED = !BLOCK && L == 1;
  auto row_of = [&](const RopeView& v, const TX* base, int r, bool out) {
    return base + r * (out ? v.y_sh : v.x_sh);
  };
  auto further = [&](const TX* at, int r, const TX* k0, bool out) {   // r: the new row
    if (r >= nq && r < nq + RG) return row_of(p.v[1], k0, r - nq, out);
    const RopeView& v = p.v[r >= nq];
    return at + RG * (out ? v.y_sh : v.x_sh);
  };
  int r_in = h0 + rg, r_out = r_in;
  const TX* x_row = r_in < nq ? row_of(p.v[0], xq, r_in, false)
                              : row_of(p.v[1], xk, r_in - nq, false);
  const TX* y_row = r_in < nq ? row_of(p.v[0], yq, r_in, true)
                              : row_of(p.v[1], yk, r_in - nq, true);
  auto load = [&](int stage, int j) {
    if (j < total) {
      const TX* x = x_row;
      if (!STEPPED) {
        int tok, r;
        place(j, &tok, &r);
        x = r < nq ? xq + r * p.v[0].x_sh + tok * p.v[0].x_st
                   : xk + (r - nq) * p.v[1].x_sh + tok * p.v[1].x_st;
      }
      V* slot = ring + stage * (2 * L * kRopeThreads);
#pragma unroll
      for (int k = 0; k < L; ++k)
        if (g + k * G < units) {
          copy_vec(slot + 2 * k * kRopeThreads, x + va[k] * E);
          copy_vec(slot + (2 * k + 1) * kRopeThreads, x + vb[k] * E);
        }
    }
    copy_commit();
    if (STEPPED) x_row = further(x_row, r_in += RG, xk, false);
  };
  // the first rows are on their way while the angles are computed
#pragma unroll
  for (int s = 0; s < S; ++s) load(s, s * RG + rg);
  const long long pos = lane_position(p, t0, tokens);
  const Tables tab =
      make_tables(p, reinterpret_cast<V*>(smem4) + S * 2 * L * kRopeThreads);
  warp_angles(p, tab, pos, tokens);
  Turn<E> cs[L];
  auto angles_at = [&](int tok) {
#pragma unroll
    for (int k = 0; k < L; ++k)
      unit_angles<E, ADJ>(p, tab.angles + tok * tab.ld_angles, g + k * G, cs[k]);
  };
  int at = -1;   // the token whose angles cs holds
  if (!BLOCK) angles_at(0);
  int stage = 0;
  // bf16 with bf16 weights: squares and products with gamma straight from the packed words
  constexpr bool PACKED = NORM && B == 16 && sizeof(TX) == 2 && sizeof(TW) == 2;
  for (int j0 = 0; j0 < total; j0 += RG) {
    const int j = j0 + rg;
    int tok, r;
    place(j, &tok, &r);
    const bool live = j < total;
    if (BLOCK && live && tok != at) {
      at = tok;
      angles_at(tok);
    }
    copy_wait<S - 1>();
    const V* slot = ring + stage * (2 * L * kRopeThreads);
    float a[L][E], b[L][E];
    V xa[L], xb[L];
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < L; ++k) {
      if constexpr (PACKED) {
        xa[k].v = xb[k].v = make_uint4(0, 0, 0, 0);
        if (live && g + k * G < units) {
          xa[k] = slot_of(slot + 2 * k * kRopeThreads);
          xb[k] = slot_of(slot + (2 * k + 1) * kRopeThreads);
        }
        add_squares(ss, xa[k].v);
        add_squares(ss, xb[k].v);
        continue;
      }
      if (live && g + k * G < units) {
        unpack_raw(slot_of(slot + 2 * k * kRopeThreads), a[k]);
        unpack_raw(slot_of(slot + (2 * k + 1) * kRopeThreads), b[k]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) a[k][i] = b[k][i] = 0.f;
      }
      if (NORM) {
        dot_all(ss, a[k], a[k]);
        dot_all(ss, b[k], b[k]);
      }
    }
    load(stage, j + S * RG);
    stage = stage + 1 == S ? 0 : stage + 1;
    float rstd = 1.f;
    if (NORM) rstd = rsqrtf(group_sum<G>(ss.x + ss.y) * p.inv_d + p.eps);
    TX* y_at = const_cast<TX*>(y_row);
    if (STEPPED) y_row = further(y_row, r_out += RG, yk, true);
    if (!live) continue;
    TX* y = y_at;
    if (!STEPPED)
      y = r < nq ? yq + r * p.v[0].y_sh + tok * p.v[0].y_st
                 : yk + (r - nq) * p.v[1].y_sh + tok * p.v[1].y_st;
#pragma unroll
    for (int k = 0; k < L; ++k) {
      if (g + k * G >= units) continue;
      if constexpr (PACKED) {
        const TW* w = static_cast<const TW*>(r < nq ? p.v[0].gamma : p.v[1].gamma);
        scale_packed(a[k], xa[k].v, ld_cached(w + va[k] * E), rstd);
        scale_packed(b[k], xb[k].v, ld_cached(w + vb[k] * E), rstd);
      } else if (NORM) {   // gamma from L1: in registers it costs a CTA per SM (116 us for 105)
        float w[E];
        load_gamma<TX, TW>(r < nq ? p.v[0].gamma : p.v[1].gamma, va[k], w);
        scale_all(w, w, rstd);
        mul_all(a[k], a[k], w);
        load_gamma<TX, TW>(r < nq ? p.v[0].gamma : p.v[1].gamma, vb[k], w);
        scale_all(w, w, rstd);
        mul_all(b[k], b[k], w);
      }
      rotate<E, ADJ>(a[k], b[k], cs[k]);
      store_vec(y + va[k] * E, a[k], static_cast<TX*>(nullptr));
      store_vec(y + vb[k] * E, b[k], static_cast<TX*>(nullptr));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward with the norm.  Persistent: each warp walks items (a token, a chunk of
// its rows, or a block of tokens) of q, then those of k, its lanes keeping the
// dgamma partials of their columns in registers; after each view the CTA adds its
// lanes' partials in a fixed order into its partial row.  The ring runs on from
// item to item, and so do the positions, one item ahead.  Small batches, whose items
// take each warp one round at most: the first p.split CTAs take q, the others k.
template <typename TX, typename TW, int E, int G, int L, bool ADJ, bool BLOCK>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_norm_bwd_kernel(RopeParams p) {
  constexpr int RG = 32 / G, W = kRopeThreads / 32, B = E * sizeof(TX), S = kRopeBwdSteps;
  using V = Raw<B>;
  extern __shared__ float4 smem4[];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // in a uniform register
  const int g = lane % G, rg = lane < RG * G ? lane / G : kNoRow;
  const int units = p.D / (2 * E);
  int va[L], vb[L];
#pragma unroll
  for (int k = 0; k < L; ++k) unit_vectors<E, ADJ>(p, g + k * G, &va[k], &vb[k]);
  V* ring = reinterpret_cast<V*>(smem4) + tid;                        // [S][4 L][threads]
  float* red = reinterpret_cast<float*>(reinterpret_cast<V*>(smem4) +
                                        S * 4 * L * kRopeThreads);    // [W][D rounded to 4]
  const int ld_red = (p.D + 3) & ~3;
  const Tables tab = make_tables(p, red + W * ld_red);
  const bool apart = p.split > 0, latter = apart && blockIdx.x >= (unsigned)p.split;
  const uint32_t cta0 = latter ? p.split : 0, cta1 = apart && !latter ? p.split : gridDim.x;
  const uint32_t nw = (cta1 - cta0) * W, w0 = (blockIdx.x - cta0) * W + warp;
  const int block = BLOCK ? p.block : 1;
  const uint32_t groups = (uint32_t)((p.T + block - 1) / block);
  uint32_t skip = 0;   // items of q, so that k's start where q's ended

  for (int side = 0; side < 2; ++side) {
    const RopeView& v = p.v[side];
    if (v.heads == 0 || (apart && side != (int)latter)) {   // its partial columns are zero
      if (p.partial)
        for (int d = tid; d < p.ld_half; d += kRopeThreads)
          p.partial[(size_t)blockIdx.x * 2 * p.ld_half + side * p.ld_half + d] = 0.f;
      continue;
    }
    const uint32_t chunks = (uint32_t)p.chunks[side];
    const uint32_t items = groups * chunks;
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

    // an item: tokens [t0, t0 + tokens), rows [h0, h0 + rows) of each
    struct Item {
      int64_t t0;
      int tokens, h0, rows;
    };
    auto item_at = [&](uint32_t it) {
      const uint32_t group = it / chunks;
      Item m;
      m.t0 = (int64_t)group * block;
      m.tokens = BLOCK ? (int)min((int64_t)block, p.T - m.t0) : 1;
      m.h0 = (int)(it - group * chunks) * p.heads_per_chunk[side];
      m.rows = min(p.heads_per_chunk[side], v.heads - m.h0);
      return m;
    };
    auto place = [&](const Item& m, int j, int* k, int* h) {
      *k = 0;
      *h = m.h0 + j;
      if (BLOCK) {
        *k = j / m.rows;
        *h -= *k * m.rows;
      }
    };
    // what comes next into the ring: row f_j of item f
    uint32_t it = (w0 + nw - skip % nw) % nw, f_it = it;
    int f_j = 0;
    Item f{};
    // The lane's row of a step, stepped on where rows are wide (8000 tokens of 32 heads of
    // 192 bf16: 64 us, worked out for every row 68; heads of 128 and 32768 tokens 176
    // against 164)
    constexpr bool STEPPED = !BLOCK && G >= 16;
    const TX *fx = nullptr, *fd = nullptr;
    auto start = [&]() {
      f = item_at(f_it);
      if (STEPPED) {
        fx = static_cast<const TX*>(v.x) + f.t0 * v.x_st + (f.h0 + rg) * v.x_sh;
        fd = static_cast<const TX*>(v.dy) + f.t0 * v.dy_st + (f.h0 + rg) * v.dy_sh;
      }
    };
    if (f_it < items) start();
    auto load = [&](int stage) {
      if (f_it < items) {
        const int j = f_j + rg;
        if (j < f.tokens * f.rows) {
          const TX *xr = fx, *dr = fd;
          if (!STEPPED) {
            int tok, h;
            place(f, j, &tok, &h);
            xr = static_cast<const TX*>(v.x) + (f.t0 + tok) * v.x_st + h * v.x_sh;
            dr = static_cast<const TX*>(v.dy) + (f.t0 + tok) * v.dy_st + h * v.dy_sh;
          }
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
        f_j += RG;
        fx += RG * v.x_sh;
        fd += RG * v.dy_sh;
        if (f_j >= f.tokens * f.rows) {
          f_j = 0;
          f_it += nw;
          if (f_it < items) start();
        }
      }
      copy_commit();
    };
    long long pos = 0;
    if (it < items) {
      const Item m = item_at(it);
      pos = lane_position(p, m.t0, m.tokens);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) load(s);
    int stage = 0;
    for (; it < items; it += nw) {
      const Item m = item_at(it);
      warp_angles(p, tab, pos, m.tokens);
      if (it + nw < items) {
        const Item n = item_at(it + nw);
        pos = lane_position(p, n.t0, n.tokens);
      }
      Turn<E> cs[L];
      auto angles_at = [&](int tok) {
#pragma unroll
        for (int k = 0; k < L; ++k)
          unit_angles<E, ADJ>(p, tab.angles + tok * tab.ld_angles, g + k * G, cs[k]);
      };
      int at = -1;   // the token whose angles cs holds
      if (!BLOCK) angles_at(0);
      const int total = m.tokens * m.rows;
      TX* yr = static_cast<TX*>(v.y) + m.t0 * v.y_st + (m.h0 + rg) * v.y_sh;
      for (int j0 = 0; j0 < total; j0 += RG, yr += RG * v.y_sh) {
        const int j = j0 + rg;
        int tok, h;
        place(m, j, &tok, &h);
        const bool live = j < total;
        if (BLOCK && live && tok != at) {
          at = tok;
          angles_at(tok);
        }
        copy_wait<S - 1>();
        const V* slot = ring + stage * (4 * L * kRopeThreads);
        float a[L][E], b[L][E], da[L][E], db[L][E];
        float2 ss = make_float2(0.f, 0.f), dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < L; ++k) {
          if (live && g + k * G < units) {
            unpack_raw(slot_of(slot + 4 * k * kRopeThreads), a[k]);
            unpack_raw(slot_of(slot + (4 * k + 1) * kRopeThreads), b[k]);
            unpack_raw(slot_of(slot + (4 * k + 2) * kRopeThreads), da[k]);
            unpack_raw(slot_of(slot + (4 * k + 3) * kRopeThreads), db[k]);
            rotate<E, ADJ>(da[k], db[k], cs[k]);
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i) a[k][i] = b[k][i] = da[k][i] = db[k][i] = 0.f;
          }
          dot_all(ss, a[k], a[k]);
          dot_all(ss, b[k], b[k]);
        }
        load(stage);
        stage = stage + 1 == S ? 0 : stage + 1;
        const float r = rsqrtf(row_sum<G>(ss.x + ss.y, g) * p.inv_d + p.eps);
        // dgamma takes g x r; then g becomes g gamma
#pragma unroll
        for (int k = 0; k < L; ++k) {
          if (g + k * G >= units) continue;
          float x[E];
          scale_all(x, a[k], r);
          fma_all(ga[k], da[k], x);
          mul_all(da[k], da[k], wa[k]);
          dot_all(dot, da[k], a[k]);
          scale_all(x, b[k], r);
          fma_all(gb[k], db[k], x);
          mul_all(db[k], db[k], wb[k]);
          dot_all(dot, db[k], b[k]);
        }
        const float c = r * r * p.inv_d * row_sum<G>(dot.x + dot.y, g);
        if (!live) continue;
        TX* y = STEPPED ? yr : static_cast<TX*>(v.y) + (m.t0 + tok) * v.y_st + h * v.y_sh;
#pragma unroll
        for (int k = 0; k < L; ++k) {
          if (g + k * G >= units) continue;
          axpy_all(da[k], a[k], -c);
          scale_all(da[k], da[k], r);
          axpy_all(db[k], b[k], -c);
          scale_all(db[k], db[k], r);
          store_vec(y + va[k] * E, da[k], static_cast<TX*>(nullptr));
          store_vec(y + vb[k] * E, db[k], static_cast<TX*>(nullptr));
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
          ga[k][i] = rows_sum<G>(ga[k][i]);
          gb[k][i] = rows_sum<G>(gb[k][i]);
          if (g + k * G < units && rg == 0) {
            red[warp * ld_red + va[k] * E + i] = ga[k][i];
            red[warp * ld_red + vb[k] * E + i] = gb[k][i];
          }
        }
      }
      __syncthreads();
      for (int d = tid; d < p.ld_half; d += kRopeThreads) {
        float s = 0.f;
        if (d < p.D)
          for (int w = 0; w < W; ++w) s += red[w * ld_red + d];
        p.partial[(size_t)blockIdx.x * 2 * p.ld_half + side * p.ld_half + d] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Scalar form of both, for rows that reach further than the vectors of their
// alignment do: a CTA per (token, chunk), the angles in shared
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

// Shapes: vectors of 16 bytes with one unit a lane, smaller ones with three or
// four, because a step of few bytes is bound by its instructions (16384 tokens x 40
// heads, forward / backward with the norm: 36 bf16 columns in single elements, 32
// lanes of one unit 92 / 251 us, 8 of three 64 / 101; 36 fp32 in pairs 49 / 81, 49 /
// 62).  Vectors of four in the backward keep to two: three spill (80 bf16
// columns 130 us, one unit 101).
template <typename TX, typename TW, bool NORM, bool ADJ, bool BWD, int E, int G, int L, bool BLOCK>
RopeKernel kernel_of() {
  if constexpr (BWD) return rope_norm_bwd_kernel<TX, TW, E, G, L, ADJ, BLOCK>;
  else return rope_kernel<TX, TW, E, G, L, NORM, ADJ, BLOCK>;
}
template <typename TX, typename TW, bool NORM, bool ADJ, bool BWD, int E>
RopeKernel pick_small(int id) {
#define RMSN_ROPE(G_, L_) \
  if (id == G_ * 10 + L_) return kernel_of<TX, TW, NORM, ADJ, BWD, E, G_, L_, false>();
  if constexpr (BWD && E == 4) {
    RMSN_ROPE(4, 2) RMSN_ROPE(8, 2) RMSN_ROPE(16, 2) RMSN_ROPE(32, 2)
  } else {
    RMSN_ROPE(4, 3) RMSN_ROPE(4, 4) RMSN_ROPE(8, 3) RMSN_ROPE(8, 4)
    RMSN_ROPE(16, 3) RMSN_ROPE(16, 4) RMSN_ROPE(32, 3) RMSN_ROPE(32, 4)
  }
#undef RMSN_ROPE
  return nullptr;
}
template <typename TX, typename TW, bool NORM, bool ADJ, bool BWD>
RopeKernel pick_shape(const RopeKey& k) {
  constexpr int E = Elem<TX>::kPerVec;
  if (k.e == 0) return rope_scalar_kernel<TX, TW, NORM, ADJ, BWD>;
  if (k.e == E && k.l == 1) {
#define RMSN_ROPE(G_) \
  if (k.g == G_)      \
    return k.block ? kernel_of<TX, TW, NORM, ADJ, BWD, E, G_, 1, true>() \
                   : kernel_of<TX, TW, NORM, ADJ, BWD, E, G_, 1, false>();
    RMSN_ROPE(4) RMSN_ROPE(8) RMSN_ROPE(16) RMSN_ROPE(32)
    if constexpr (BWD) { RMSN_ROPE(5) RMSN_ROPE(6) RMSN_ROPE(10) }
#undef RMSN_ROPE
    return nullptr;
  }
  if (k.block) return nullptr;
  const int id = k.g * 10 + k.l;
  if (k.e == 1) return pick_small<TX, TW, NORM, ADJ, BWD, 1>(id);
  if (k.e == 2) return pick_small<TX, TW, NORM, ADJ, BWD, 2>(id);
  if constexpr (E == 8)
    if (k.e == 4) return pick_small<TX, TW, NORM, ADJ, BWD, 4>(id);
  return nullptr;
}
template <typename TX, typename TW>
RopeKernel pick(const RopeKey& k) {
  if (k.bwd)
    return k.adjacent ? pick_shape<TX, TW, true, true, true>(k)
                      : pick_shape<TX, TW, true, false, true>(k);
  if (k.norm)
    return k.adjacent ? pick_shape<TX, TW, true, true, false>(k)
                      : pick_shape<TX, TW, true, false, false>(k);
#if RMSN_PAIR == 2   // the rotation alone has no weights: the bf16/bf16 unit has it
  return nullptr;
#else
  return k.adjacent ? pick_shape<TX, TW, false, true, false>(k)
                    : pick_shape<TX, TW, false, false, false>(k);
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
