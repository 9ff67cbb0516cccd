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

// Largest value over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xf, 0xf, false);  // 1 0 3 2
  x = y > x ? y : x;
  const uint32_t z = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xf, 0xf, false);  // 2 3 0 1
  return z > x ? z : x;
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
// 2^(127 - byte), exact for all bytes that scale_byte gives; 0 for 255.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 255u ? __builtin_nanf("")
                      : __uint_as_float(byte == 0u ? 0x400000u : byte << 23);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t largest8(const float* c) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = magnitude(c[i]);
    top = w > top ? w : top;
  }
  return top;
}

// Codes of 8 consecutive elements, c times inv (a power of two; 0 for a block
// that is not finite).
__device__ __forceinline__ uint32_t encode8(const float* c, float inv) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[0] * inv, c[1] * inv, 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[2] * inv, c[3] * inv, 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[4] * inv, c[5] * inv, 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c[6] * inv, c[7] * inv, 1.0f, 3);
  return inv == 0.0f ? 0u : r;
}
// Stochastically: the instruction adds the top bits of its 32 random ones below
// the kept bits of its first value, and those from bit 30 on to its second.
// Each element has 16 random bits of its own, so each is converted beside a
// zero, which stays one.  Only byte 0 of a result counts: the builtin does not
// keep the old value's other bytes, so they are joined by permutations.
__device__ __forceinline__ uint32_t convert_stochastic(float x, float y, uint32_t word) {
  return __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{x, 0.0f}, word << 16, 1.0f, 0) |
         __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, f32x2{0.0f, y}, (word >> 16) << 15, 1.0f,
                                                     0);
}
// quad: index of elements 0..3 (4..7 follow), even: its neighbour has the same
// upper half.
__device__ __forceinline__ uint32_t encode8_stochastic(const float* c, float inv, uint64_t quad,
                                                       Keys k) {
  const uint32_t key = high_key(quad, k.k0);
  const uint32_t a0 = first_word((uint32_t)quad, key), a1 = next_word(a0, k.k1, 1);
  const uint32_t b0 = first_word((uint32_t)quad + 1u, key), b1 = next_word(b0, k.k1, 1);
  const uint32_t p0 = convert_stochastic(c[0] * inv, c[1] * inv, a0);
  const uint32_t p1 = convert_stochastic(c[2] * inv, c[3] * inv, a1);
  const uint32_t p2 = convert_stochastic(c[4] * inv, c[5] * inv, b0);
  const uint32_t p3 = convert_stochastic(c[6] * inv, c[7] * inv, b1);
  const uint32_t r = __builtin_amdgcn_perm(p1, p0, 0x0c0c0400u) |
                     __builtin_amdgcn_perm(p3, p2, 0x04000c0cu);
  return inv == 0.0f ? 0u : r;
}

// The values of 8 codes.
__device__ __forceinline__ void decode8(uint32_t codes, float scale, float* v) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
  v[0] = a.x * scale, v[1] = a.y * scale, v[2] = b.x * scale, v[3] = b.y * scale;
  v[4] = c.x * scale, v[5] = c.y * scale, v[6] = d.x * scale, v[7] = d.y * scale;
}

}  // namespace mx4
}  // namespace ob
