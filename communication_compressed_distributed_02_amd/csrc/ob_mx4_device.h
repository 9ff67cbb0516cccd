// Loads, stores and conversions that the ob_mx4 kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_random.h"

namespace ob {
namespace mx4 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Wide accesses at the alignment of one element, which gfx950 takes.
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));

struct bf16 {
  uint16_t bits;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ void load8(const float* p, float* c) {
  const f32x4 a = *(const f32x4_at4*)p, b = *(const f32x4_at4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = a[i], c[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const bf16* p, float* c) {
  const u32x4 w = *(const u32x4_at2*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = __uint_as_float(w[i] << 16);
    c[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// The same past the caches.
__device__ __forceinline__ void load8_stream(const float* p, float* c) {
  const f32x4 a = __builtin_nontemporal_load((const f32x4_at4*)p);
  const f32x4 b = __builtin_nontemporal_load((const f32x4_at4*)(p + 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = a[i], c[4 + i] = b[i];
}
__device__ __forceinline__ void load8_stream(const bf16* p, float* c) {
  const u32x4 w = __builtin_nontemporal_load((const u32x4_at2*)p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[2 * i] = __uint_as_float(w[i] << 16);
    c[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8_stream(float* p, const float* c) {
  __builtin_nontemporal_store(f32x4{c[0], c[1], c[2], c[3]}, (f32x4_at4*)p);
  __builtin_nontemporal_store(f32x4{c[4], c[5], c[6], c[7]}, (f32x4_at4*)(p + 4));
}
// The first n of them, zeros after.
template <typename T>
__device__ __forceinline__ void load8_some(const T* p, int n, float* c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 0.0f;
    if (i < n) c[i] = widen(p[i]);
  }
}
__device__ __forceinline__ void store8(float* p, const float* c) {
  *(f32x4_at4*)p = f32x4{c[0], c[1], c[2], c[3]};
  *(f32x4_at4*)(p + 4) = f32x4{c[4], c[5], c[6], c[7]};
}
__device__ __forceinline__ void store8(bf16* p, const float* c) {
  *(u32x4_at2*)p = u32x4{pack_bf16(c[0], c[1]), pack_bf16(c[2], c[3]), pack_bf16(c[4], c[5]),
                         pack_bf16(c[6], c[7])};
}
__device__ __forceinline__ void store1(float* p, float c) { *p = c; }
__device__ __forceinline__ void store1(bf16* p, float c) {
  p->bits = (uint16_t)pack_bf16(c, c);
}

// Blocks go to the 8 dies in turn: the block's place in an order that gives each
// die a run of neighbours, which then share its cache.
__device__ __forceinline__ uint32_t on_one_die(uint32_t block, uint32_t all) {
  constexpr uint32_t kDies = 8;
  const uint32_t per = all / kDies, more = all % kDies, die = block % kDies;
  return die * per + (die < more ? die : more) + block / kDies;
}

// What this wave wrote to LDS is there for all its lanes.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Largest value over the four lanes of a quad, and over 8 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
  return y > x ? y : x;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  return max_with<0x4E>(max_with<0xB1>(x));  // lanes 1 0 3 2, then 2 3 0 1
}
__device__ __forceinline__ uint32_t oct_max(uint32_t x) {
  return max_with<0x141>(quad_max(x));  // halves of 8 lanes mirrored
}

// The scale byte of a block from the bit pattern of its largest magnitude: the
// exponent of the least power of two of which it is below 7 times (or at most
// 6 times), as patterns: what exceeds 1.75 (1.5) of a power of two carries
// into the exponent.  255 where a value is not finite.
template <bool STOCHASTIC>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int e = (int)((top + (STOCHASTIC ? 0x3FFFFFu : 0x200000u)) >> 23) - 2;
  return top >= 0x7f800000u ? 255u : (uint32_t)(e < 0 ? 0 : e);
}
// What the conversions divide by: they take its exponent field alone, so that 0
// stands for 2^-127.  (Their results are dropped for 255.)
__device__ __forceinline__ float divisor(uint32_t byte) { return __uint_as_float(byte << 23); }
// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 255u ? __builtin_nanf("")
                      : __uint_as_float(byte == 0u ? 0x400000u : byte << 23);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Of pairs of bfloat16 values, as pairs; the larger of a pair as fp32's pattern.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 magnitudes(uint32_t w) {
  return __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t larger(u16x2 m) {
  const uint32_t w = __builtin_bit_cast(uint32_t, m), high = w & 0xffff0000u, low = w << 16;
  return high > low ? high : low;
}
template <int N>
__device__ __forceinline__ uint32_t largest(const float* c) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w = magnitude(c[i]);
    top = w > top ? w : top;
  }
  return top;
}

// Codes of 8 consecutive elements of a block with this scale byte, zeros for 255.
__device__ __forceinline__ uint32_t encode8(const float* c, uint32_t byte) {
  const float s = divisor(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[0], c[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[2], c[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[4], c[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[6], c[7], s, 3);
  return byte == 255u ? 0u : r;
}
// Of 4, in the low 16 bits.
__device__ __forceinline__ uint32_t encode4(const float* c, uint32_t byte) {
  const float s = divisor(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[0], c[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[2], c[3], s, 1);
  return byte == 255u ? 0u : r;
}
// From pairs of bfloat16 values.
__device__ __forceinline__ bf16x2 pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }
__device__ __forceinline__ uint32_t encode8(u32x4 w, uint32_t byte) {
  const float s = divisor(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(w[0]), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(w[1]), s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(w[2]), s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(w[3]), s, 3);
  return byte == 255u ? 0u : r;
}
__device__ __forceinline__ uint32_t encode4(u32x2 w, uint32_t byte) {
  const float s = divisor(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(w[0]), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(w[1]), s, 1);
  return byte == 255u ? 0u : r;
}

// Stochastically: the instruction adds the top bits of its 32 random ones below
// the kept bits of its first value, and those from bit 30 on to its second.
// Each element has 16 random bits of its own, so a pair is converted twice and
// gives one code each time.  Only byte 0 of a result counts: the builtin does
// not keep the old value's other bytes, so they are joined by permutations.
// (The form for bfloat16 values rounds otherwise where they are small beside
// their block's scale, so they are widened.)
__device__ __forceinline__ uint32_t pair_stochastic(float x, float y, uint32_t word, float s) {
  const f32x2 v = {x, y};
  const uint32_t a = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, v, word << 16, s, 0);
  const uint32_t b =
      __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, v, word >> 1 & 0x7fff8000u, s, 0);
  return (a & 15u) | (b & ~15u);
}
__device__ __forceinline__ uint32_t pair_stochastic(uint32_t w, uint32_t word, float s) {
  return pair_stochastic(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u), word, s);
}
// The random words of 4 elements.  WIDE: their index may pass 2^32.
struct Words {
  uint32_t a, b;
};
template <bool WIDE>
__device__ __forceinline__ Words random_words(uint64_t quad, Keys k) {
  Words w;
  w.a = first_word((uint32_t)quad, WIDE ? high_key(quad, k.k0) : k.k0);
  w.b = next_word(w.a, k.k1, 1);
  return w;
}
__device__ __forceinline__ uint32_t join2(uint32_t p0, uint32_t p1) {
  return __builtin_amdgcn_perm(p1, p0, 0x0c0c0400u);
}
__device__ __forceinline__ uint32_t join4(uint32_t p0, uint32_t p1, uint32_t p2, uint32_t p3) {
  return join2(p0, p1) | __builtin_amdgcn_perm(p3, p2, 0x04000c0cu);
}
// quad: index of the first four elements.
template <bool WIDE>
__device__ __forceinline__ uint32_t encode4_stochastic(const float* c, uint32_t byte, uint64_t quad,
                                                       Keys k) {
  const float s = divisor(byte);
  const Words r = random_words<WIDE>(quad, k);
  const uint32_t p0 = pair_stochastic(c[0], c[1], r.a, s), p1 = pair_stochastic(c[2], c[3], r.b, s);
  return byte == 255u ? 0u : join2(p0, p1);
}
template <bool WIDE>
__device__ __forceinline__ uint32_t encode8_stochastic(const float* c, uint32_t byte, uint64_t quad,
                                                       Keys k) {
  const float s = divisor(byte);
  const Words q = random_words<WIDE>(quad, k), r = random_words<WIDE>(quad + 1, k);
  const uint32_t p0 = pair_stochastic(c[0], c[1], q.a, s), p1 = pair_stochastic(c[2], c[3], q.b, s);
  const uint32_t p2 = pair_stochastic(c[4], c[5], r.a, s), p3 = pair_stochastic(c[6], c[7], r.b, s);
  return byte == 255u ? 0u : join4(p0, p1, p2, p3);
}
template <bool WIDE>
__device__ __forceinline__ uint32_t encode4_stochastic(u32x2 w, uint32_t byte, uint64_t quad,
                                                       Keys k) {
  const float s = divisor(byte);
  const Words r = random_words<WIDE>(quad, k);
  const uint32_t p0 = pair_stochastic(w[0], r.a, s), p1 = pair_stochastic(w[1], r.b, s);
  return byte == 255u ? 0u : join2(p0, p1);
}
template <bool WIDE>
__device__ __forceinline__ uint32_t encode8_stochastic(u32x4 w, uint32_t byte, uint64_t quad,
                                                       Keys k) {
  const float s = divisor(byte);
  const Words q = random_words<WIDE>(quad, k), r = random_words<WIDE>(quad + 1, k);
  const uint32_t p0 = pair_stochastic(w[0], q.a, s), p1 = pair_stochastic(w[1], q.b, s);
  const uint32_t p2 = pair_stochastic(w[2], r.a, s), p3 = pair_stochastic(w[3], r.b, s);
  return byte == 255u ? 0u : join4(p0, p1, p2, p3);
}

// 8 codes without their scale, and their values.
__device__ __forceinline__ void grid8(uint32_t codes, float* v) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}
__device__ __forceinline__ void decode8(uint32_t codes, float scale, float* v) {
  grid8(codes, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= scale;
}

}  // namespace mx4
}  // namespace ob
