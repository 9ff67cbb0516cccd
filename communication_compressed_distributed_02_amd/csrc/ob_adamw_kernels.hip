// gfx950 kernels of AdamW's step over many tensors and of the gradient norm.
// The arithmetic contract is stated in include/ob_adamw.h.
//
// Mapping: work is listed in chunks of 4096 elements of one tensor, made of 16
// groups of 256, of which a lane takes 4 consecutive elements.  A group is the
// unit that shares the exponents of an 8-bit state, so its maximum is a
// reduction over one wave's lanes, in registers.  A wave takes 4 groups of the
// norm, 1 or 2 of a step over many chunks (kStepGroups) and 1 or 4 of a step
// over few (kFewChunks).  The list of chunks (tensor, place, length,
// hyperparameter group) is made once per plan; the tensors' pointers come by
// value with each launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ob_adamw_kernels.h"

namespace ob {
namespace adamw {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kGroups = kRowElems / kScaleElems;  // groups of 256 in a row of 1024

struct bf16 {
  uint16_t bits;
};

// Index of this wavefront in its block, as a wave-uniform (scalar) value.
__device__ __forceinline__ int wave_in_block() {
  return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __uint_as_float((uint32_t)x.bits << 16); }

// Two fp32 values as bfloat16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 h = __builtin_convertvector(f32x2{a, b}, bf16x2);
  return __builtin_bit_cast(uint32_t, h);
}

template <typename T>
__device__ __forceinline__ T ld_stream(const T* p) { return __builtin_nontemporal_load(p); }
template <typename T>
__device__ __forceinline__ void st_stream(T* p, T v) { __builtin_nontemporal_store(v, p); }

// Four elements from p, which may be aligned to one of them only: gfx950
// takes wide accesses at any address, so an unaligned tensor costs the lines
// that its accesses straddle and no other code.
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
__device__ __forceinline__ f32x4 load4(const float* p) {
  return __builtin_nontemporal_load((const f32x4_at4*)p);
}
__device__ __forceinline__ u32x2 load_packed(const bf16* p) {
  return __builtin_nontemporal_load((const u32x2_at2*)p);
}
// The same through the caches.
__device__ __forceinline__ f32x4 load4_cached(const float* p) { return *(const f32x4_at4*)p; }
__device__ __forceinline__ f32x4 widen2(u32x2 w) {
  return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
               __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 load4(const bf16* p) {
  return widen2(load_packed(p));
}
__device__ __forceinline__ f32x4 load4_cached(const bf16* p) {
  return widen2(*(const u32x2_at2*)p);
}
// The first n (0 to 4) of them at element alignment, zeros after.
template <typename T>
__device__ __forceinline__ f32x4 load_some(const T* p, int n) {
  f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) r[k] = widen(p[k]);
  return r;
}

// Random bits: a 32-bit word hashed from the quad's index and the step's
// first key, and more words from the word before and the second key.  The
// multipliers are digits of sqrt(5), sqrt(3) and the golden ratio; every
// input bit flips every output bit with probability 1/2 within the noise of
// 65536 quads, and no two bits of the four words correlate above it.
__device__ __forceinline__ uint32_t first_word(uint32_t quad, uint32_t key) {
  uint32_t h = quad ^ key;
  h = (h ^ (h >> 16)) * 0x3C6EF373u;
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}
__device__ __forceinline__ uint32_t next_word(uint32_t word, uint32_t key, uint32_t i) {
  const uint32_t h = (word ^ key) * 0x9E3779B9u + i;
  return h ^ (h >> 15);
}
// Quads past 2^32 take another key.
__device__ __forceinline__ uint32_t high_key(uint64_t quad, uint32_t key) {
  return key ^ ((uint32_t)(quad >> 32) * 0x9E3779B9u);
}
__device__ __forceinline__ uint32_t random16(uint32_t a, uint32_t b, int k) {
  const uint32_t w = k < 2 ? a : b;
  return k & 1 ? w >> 16 : w & 0xffffu;
}

// The low 16 bits of x's fp32 pattern rounded stochastically away.  What is
// not finite keeps its pattern (an arithmetic NaN has its quiet bit above).
__device__ __forceinline__ uint32_t round_stochastic(float x, uint32_t r16) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x7f800000u) == 0x7f800000u ? b : b + r16;
}

// Largest value over the wave's 64 lanes, as a scalar: four shifts within
// rows of 16 lanes, then row 0 and 2's last lane to the next row, then lane 31
// to the upper half; lane 63 ends with all of them.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  const auto step = [&](auto ctrl, auto rows) {
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)x, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
    x = y > x ? y : x;
  };
  step(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());  // row_shr:1
  step(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());  // row_shr:2
  step(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());  // row_shr:4
  step(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());  // row_shr:8
  step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());  // row_bcast:15
  step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

__device__ __forceinline__ bool finite_bits(uint32_t b) { return (b & 0x7f800000u) != 0x7f800000u; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// ---------------------------------------------------------- 8-bit codes --
// First moment, a group's four elements of this lane.  e: the group's
// exponent byte; scaling by a power of two is exact, so the e4m3 conversion
// is the only rounding.
__device__ __forceinline__ f32x4 decode_m(uint32_t codes, uint32_t e) {
  const float s = __uint_as_float((e - 7u) << 23);
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  return f32x4{lo.x * s, lo.y * s, hi.x * s, hi.y * s};
}

__device__ __forceinline__ uint32_t codes_m(f32x4 m, uint32_t e) {
  const float s = __uint_as_float((261u - e) << 23);
  const int c = __builtin_amdgcn_cvt_pk_fp8_f32(m.x * s, m.y * s, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(m.z * s, m.w * s, c, true);
}

// The wave's largest |m|, as a pattern.
__device__ __forceinline__ uint32_t top_m(f32x4 m) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) top = umax(top, __float_as_uint(m[k]) & 0x7fffffffu);
  return wave_max(top);
}

// Codes and exponent of a group whose elements lane by lane are m, top =
// top_m(m).
__device__ __forceinline__ uint32_t encode_m(f32x4 m, uint32_t top, uint32_t* e_out) {
  if (top >= 0x7f800000u) {  // something is not finite: held as NaN, the others keep their scale
    f32x4 rest = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!finite_bits(__float_as_uint(m[k]))) {
        rest[k] = 0.0f;
        m[k] = __uint_as_float(0x7fc00000u);
      }
    }
    top = top_m(rest);
  }
  const uint32_t e = umax(top >> 23, (uint32_t)kMinExpM);
  *e_out = e;
  return codes_m(m, e);
}

// Second moment: the code counts eighths of a binade up from the group's
// floor, so decoding is an addition to the fp32 pattern's upper bits.
__device__ __forceinline__ uint32_t floor_v(uint32_t e) { return (e - 31u) * 8u + 1u; }

__device__ __forceinline__ f32x4 decode_v(uint32_t codes, uint32_t e) {
  const uint32_t low = floor_v(e);
  f32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t c = (codes >> (8 * k)) & 255u;
    uint32_t b = c == 0 ? 0u : (c + low) << 20;
    if (c == 255u) b = 0x7fc00000u;
    v[k] = __uint_as_float(b);
  }
  return v;
}

// A v's pattern with `noise` added, less its low 20 bits: rounded to the codes'
// steps.  The sign goes, so that no NaN's pattern wraps around to a small one.
__device__ __forceinline__ uint32_t rounded_v(float v, uint32_t noise) {
  return ((__float_as_uint(v) & 0x7fffffffu) + noise) >> 20;
}
// 16 random bits as that noise, half a unit up: no bias.
__device__ __forceinline__ uint32_t noise_v(uint32_t a, uint32_t b, int k) {
  return (random16(a, b, k) << 4) | 8u;
}

// Codes and exponent of a group whose elements lane by lane are v, rounded to
// q, top the wave's largest q.
__device__ __forceinline__ uint32_t encode_v(f32x4 v, uint32_t (&q)[4], uint32_t top,
                                             uint32_t* e_out) {
  uint32_t odd = 0;  // bit k: element k is not finite
  if (top >= 2040u) {  // something is not finite, or the largest fp32 values round up to infinity
    top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (finite_bits(__float_as_uint(v[k]))) {
        q[k] = umin(q[k], 2039u);
        top = umax(top, q[k]);
      } else {
        odd |= 1u << k;
      }
    }
    top = wave_max(top);
  }
  const uint32_t e = umax(top >> 3, (uint32_t)kMinExpV);
  const int low = (int)floor_v(e);
  uint32_t codes = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    int c = (int)q[k] - low;
    c = c < 1 ? 1 : (c > 254 ? 254 : c);
    if (v[k] == 0.0f) c = 0;
    if ((odd >> k) & 1u) c = 255;
    codes |= (uint32_t)c << (8 * k);
  }
  *e_out = e;
  return codes;
}

// ------------------------------------------------------------------ step --
__device__ __forceinline__ float moment1(float m, float g, float b1, float ob1) {
  return (b1 * m) + (ob1 * g);
}
__device__ __forceinline__ float moment2(float v, float g, float b2, float ob2) {
  return (b2 * v) + (ob2 * (g * g));
}
__device__ __forceinline__ float updated(float x, float m, float v, float decay, float rate,
                                         float rbc2, float eps) {
  const float den = (sqrtf(v) * rbc2) + eps;
  return (x * decay) - (rate * (m / den));
}

// What lies behind the tensor's last element (this lane's n-th) stays zero.
__device__ __forceinline__ void clear_behind(int n, f32x4& m, f32x4& v, f32x4& x) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k >= n) m[k] = v[k] = x[k] = 0.0f;
}

// The same beside 8-bit moments, whose own steps are 2^-4 of them, for 2^-30
// <= eps, v < 2^100 and |m| < 2^90: v_sqrt_f32 and v_rcp_f32 as they are (an
// ulp each, so m/den is within 7 roundings; below 2^-126 v counts as 0, which
// eps hides), without the scaling and the Newton steps of the general forms.
// The step is bound by the ALU otherwise: 1.56B bfloat16 parameters take
// 3.10 ms in the general form, 2.65 with correctly rounded results but no
// scaling, and 2.49 (6.3 TB/s) as here.
__device__ __forceinline__ float updated_plain(float x, float m, float v, float decay, float rate,
                                               float rbc2, float eps) {
  const float den = (__builtin_amdgcn_sqrtf(v) * rbc2) + eps;
  return (x * decay) - (rate * (m * __builtin_amdgcn_rcpf(den)));
}

// Four elements as they were loaded: bfloat16 stays packed until it is used.
template <typename T, bool WHOLE>
struct Quad {
  f32x4 x;
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (WHOLE) x = load4(p);
    else x = load_some(p, n);
  }
  __device__ __forceinline__ f32x4 values() const { return x; }
};
template <>
struct Quad<bf16, true> {
  u32x2 w;
  __device__ __forceinline__ void load(const bf16* p, int) { w = load_packed(p); }
  __device__ __forceinline__ f32x4 values() const { return widen2(w); }
};

template <bool WHOLE>
__device__ __forceinline__ void store_param(float* p, f32x4 x, int n) {
  if constexpr (WHOLE) {
    __builtin_nontemporal_store(x, (f32x4_at4*)p);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) p[k] = x[k];
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store_param(bf16* p, u32x2 w, int n) {
  if constexpr (WHOLE) {
    __builtin_nontemporal_store(w, (u32x2_at2*)p);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) p[k].bits = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
  }
}

// A step's scalars, the same for every element of a row.
struct Scalars {
  float gs, decay, rate, rbc2;
  uint32_t key0, key1;
  bool skip;
};

// The four random words of this lane's quad of group u.
struct Words {
  uint32_t w[4];
  template <int N>
  __device__ __forceinline__ void make(uint64_t quad0, int u, int lane, uint32_t key0,
                                       uint32_t key1) {
    w[0] = first_word((uint32_t)quad0 + u * (kScaleElems / 4) + lane, key0);
#pragma unroll
    for (int i = 1; i < N; ++i) w[i] = next_word(w[i - 1], key1, i);
  }
};

// Rounds four updated parameters as SR says (ODD: they may not be finite) and
// stores them.
template <bool SR, bool ODD, bool WHOLE>
__device__ __forceinline__ void put(float* p, f32x4 x, int n, const Words&) {
  store_param<WHOLE>(p, x, n);
}
template <bool SR, bool ODD, bool WHOLE>
__device__ __forceinline__ void put(bf16* p, f32x4 x, int n, const Words& w) {
  if constexpr (SR) {
    uint32_t s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t r = random16(w.w[2], w.w[3], k);
      s[k] = ODD ? round_stochastic(x[k], r) : __float_as_uint(x[k]) + r;
    }
    // the upper halves of two words
    store_param<WHOLE>(p, u32x2{__builtin_amdgcn_perm(s[1], s[0], 0x07060302u),
                                __builtin_amdgcn_perm(s[3], s[2], 0x07060302u)}, n);
  } else {
    store_param<WHOLE>(p, u32x2{pack_bf16(x.x, x.y), pack_bf16(x.z, x.w)}, n);
  }
}

// Nonzero in a lane where one of the four codes of v is 0 or 255.
__device__ __forceinline__ uint32_t special_codes(uint32_t c) {
  const uint32_t low = c - 0x01010101u, high = 0xfefefefeu - c;  // borrow out of a 0, of a 255
  return ((low & ~c) | (high & c)) & 0x80808080u;
}

// The exponent bytes of a wave's groups, as one value.
template <int GROUPS>
using exps_t = std::conditional_t<GROUPS == 1, uint8_t,
                                  std::conditional_t<GROUPS == 2, uint16_t, uint32_t>>;

// GROUPS groups of 256 elements of one tensor, whose state starts at element
// 256*group.  WHOLE: all of them are the tensor's.  scalars() is called when
// the loads are under way.
template <typename PT, typename GT, int BITS, bool MASTER, bool SR, int GROUPS, bool WHOLE,
          typename F>
__device__ __forceinline__ void step_groups(const GT* g, PT* p, const State& s, int64_t group,
                                            int left, F scalars) {
  const int lane = threadIdx.x & 63;
  const int at = lane * 4;
  float* master = s.master + group * kScaleElems + at;
  float* m32 = (float*)s.m + group * kScaleElems + at;
  float* v32 = (float*)s.v + group * kScaleElems + at;
  uint8_t* m8 = (uint8_t*)s.m + group * kScaleElems + at;
  uint8_t* v8 = (uint8_t*)s.v + group * kScaleElems + at;
  g += at;
  p += at;
  Quad<GT, WHOLE> gq[GROUPS];
  Quad<PT, WHOLE> pq[GROUPS];
  f32x4 xm[GROUPS], mv[GROUPS], vv[GROUPS];
  uint32_t mc[GROUPS], vc[GROUPS], me = 0, ve = 0;
#pragma unroll
  for (int u = 0; u < GROUPS; ++u) {
    const int o = u * kScaleElems, n = left - o - at;
    if (!WHOLE && o >= left) break;  // groups behind the tensor's last element
    gq[u].load(g + o, n);
    if constexpr (MASTER) xm[u] = load4(master + o);
    else pq[u].load(p + o, n);
    if constexpr (BITS == 32) {
      mv[u] = load4(m32 + o);
      vv[u] = load4(v32 + o);
    } else {
      mc[u] = ld_stream((const uint32_t*)(m8 + o));
      vc[u] = ld_stream((const uint32_t*)(v8 + o));
    }
  }
  if constexpr (BITS == 8) {
    me = *(const exps_t<GROUPS>*)(s.m_exp + group);
    ve = *(const exps_t<GROUPS>*)(s.v_exp + group);
  }
  const Scalars c = scalars();
  if (c.skip) return;
  const float b1 = s.beta1, ob1 = 1.0f - b1, b2 = s.beta2, ob2 = 1.0f - b2;
  const uint64_t quad0 = (uint64_t)group * (kScaleElems / 4);
  const uint32_t key0 = high_key(quad0, c.key0), key1 = c.key1;
  const bool plain_scalars =
      s.eps >= 0x1p-30f && b2 >= 0x1p-10f && (b1 == 0.0f || b1 >= 0x1p-8f);
  uint32_t new_me = 0, new_ve = 0;
#pragma unroll
  for (int u = 0; u < GROUPS; ++u) {
    const int o = u * kScaleElems, n = left - o - at;
    if (!WHOLE && o >= left) {  // they hold zeros and keep them
      new_me |= (uint32_t)kMinExpM << (8 * u);
      new_ve |= (uint32_t)kMinExpV << (8 * u);
      continue;
    }
    const f32x4 gv = gq[u].values() * c.gs;
    f32x4 x, m, v;
    if constexpr (MASTER) x = xm[u];
    else x = pq[u].values();
    Words w;
    if constexpr (SR) w.make<4>(quad0, u, lane, key0, key1);
    else if constexpr (BITS == 8) w.make<2>(quad0, u, lane, key0, key1);
    if constexpr (BITS == 32) {
      m = mv[u];
      v = vv[u];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = moment1(m[k], gv[k], b1, ob1);
        v[k] = moment2(v[k], gv[k], b2, ob2);
        x[k] = updated(x[k], m[k], v[k], c.decay, c.rate, c.rbc2, s.eps);
      }
      if constexpr (!WHOLE) clear_behind(n, m, v, x);
      put<SR, true, WHOLE>(p + o, x, n, w);
      st_stream((f32x4*)(m32 + o), m);
      st_stream((f32x4*)(v32 + o), v);
    } else {
      const uint32_t em = (me >> (8 * u)) & 255u, ev = (ve >> (8 * u)) & 255u;
      // No code of v is special and m's scale (at least 2^-118) times b1 is a
      // normal number or 0: then v stays above zero and decoding needs no
      // exceptions.  (A v that is not finite comes from such a gradient, and so
      // with such an m.)
      bool plain = plain_scalars && em >= 16u && __ballot(special_codes(vc[u])) == 0;
      if (plain) {
        // b1 * (code * 2^k) rounds as (b1 * 2^k) * code does
        const float bs = b1 * __uint_as_float((em - 7u) << 23);
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[u], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[u], true);
        m = f32x4{bs * lo.x, bs * lo.y, bs * hi.x, bs * hi.y};
        const uint32_t low = floor_v(ev);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = __uint_as_float((((vc[u] >> (8 * k)) & 255u) + low) << 20);
      } else {
        m = decode_m(mc[u], em) * b1;
        v = decode_v(vc[u], ev);
      }
      uint32_t q[4], tv = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = m[k] + (ob1 * gv[k]);
        v[k] = moment2(v[k], gv[k], b2, ob2);
      }
      if constexpr (!WHOLE) {
        f32x4 unused = x;
        clear_behind(n, m, v, unused);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[k] = rounded_v(v[k], noise_v(w.w[0], w.w[1], k));
        tv = umax(tv, q[k]);
      }
      const uint32_t tm = top_m(m);
      tv = wave_max(tv);
      uint32_t cm, cv, e;
      if (plain && tm < (217u << 23) && tv < (227u << 3) && WHOLE) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = updated_plain(x[k], m[k], v[k], c.decay, c.rate, c.rbc2, s.eps);
        put<SR, false, WHOLE>(p + o, x, n, w);
        e = umax(tm >> 23, (uint32_t)kMinExpM);
        new_me |= e << (8 * u);
        cm = codes_m(m, e);
        e = umax(tv >> 3, (uint32_t)kMinExpV);
        new_ve |= e << (8 * u);
        // q less the floor, at least 1: a saturating difference to one above it
        const uint32_t one = floor_v(e) + 1u;
        cv = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) cv |= __builtin_elementwise_sub_sat(q[k], one) << (8 * k);
        cv += 0x01010101u;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = updated(x[k], m[k], v[k], c.decay, c.rate, c.rbc2, s.eps);
        if constexpr (!WHOLE) clear_behind(n, m, v, x);
        put<SR, true, WHOLE>(p + o, x, n, w);
        cm = encode_m(m, tm, &e);
        new_me |= e << (8 * u);
        cv = encode_v(v, q, tv, &e);
        new_ve |= e << (8 * u);
      }
      st_stream((uint32_t*)(m8 + o), cm);
      st_stream((uint32_t*)(v8 + o), cv);
    }
    if constexpr (MASTER) st_stream((f32x4*)(master + o), x);
  }
  if constexpr (BITS == 8) {
    if (lane == 0) {
      *(exps_t<GROUPS>*)(s.m_exp + group) = (exps_t<GROUPS>)new_me;
      *(exps_t<GROUPS>*)(s.v_exp + group) = (exps_t<GROUPS>)new_ve;
    }
  }
}

// This wave's share of a chunk, from its element `begin` on: `left` elements, of
// which it takes GROUPS groups.
template <typename PT, typename GT, int BITS, bool MASTER, bool SR, int GROUPS, typename F>
__device__ __forceinline__ void step_wave(const GT* g, PT* p, const State& s, uint32_t row,
                                          uint32_t state_row, int begin, int left, F scalars) {
  const int64_t group = (int64_t)state_row * kGroups + begin / kScaleElems;
  g += (int64_t)row * kRowElems + begin;
  p += (int64_t)row * kRowElems + begin;
  if (left >= GROUPS * kScaleElems)
    step_groups<PT, GT, BITS, MASTER, SR, GROUPS, true>(g, p, s, group, left, scalars);
  else
    step_groups<PT, GT, BITS, MASTER, SR, GROUPS, false>(g, p, s, group, left, scalars);
}

// Groups that a wave of a step over many chunks takes, and blocks of a chunk.
// 32-bit states, 1, 2 and 4 groups: 1458, 1480 and 1505 us on 334M parameters in
// 390 tensors, 73, 74 and 77 on 13M in 61.  8-bit ones: 39.8, 38.3 and 41.2 on
// the 61, 3.43, 3.00 and 2.98 ms on 1.56B (the scalars' share of a wave's
// instructions).
template <int BITS>
constexpr int kStepGroups = BITS == 32 ? 1 : 2;
template <int BITS>
constexpr int kStepBlocks = kGroups / kStepGroups<BITS>;

template <typename PT, typename GT, int BITS, bool MASTER, bool SR>
__global__ void __launch_bounds__(kBlock)
    step_kernel(StepPtrs ptrs, State s, uint32_t t0, int64_t c0) {
  constexpr int kShare = kStepGroups<BITS> * kScaleElems;  // of a wave
  const Control* __restrict__ ctl = s.control;
  const ChunkRec rec = s.recs[c0 + blockIdx.x / kStepBlocks<BITS>];
  const GT* g = (const GT*)ptrs.g[rec.tensor - t0];
  PT* p = (PT*)ptrs.p[rec.tensor - t0];
  if (g == nullptr || ctl->skip) return;
  const int begin =
      ((int)(blockIdx.x % kStepBlocks<BITS>) * (kBlock / 64) + wave_in_block()) * kShare;
  const int left = (int)rec.count - begin;
  if (left <= 0) return;
  step_wave<PT, GT, BITS, MASTER, SR, kStepGroups<BITS>>(
      g, p, s, rec.row, rec.state_row, begin, left, [&] {
        return Scalars{ctl->gscale, ctl->decay[rec.group], ctl->rate[rec.group], ctl->rbc2,
                       ctl->k0,     ctl->k1,               false};
      });
}

// ------------------------------------------------------------------ norm --
// The block's sum in a fixed order: lanes by an xor butterfly, then the four
// waves.
__device__ __forceinline__ double block_sum(double acc, double* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) acc = acc + __shfl_xor(acc, o, 64);
  __syncthreads();  // red may still be read from the call before
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ double add_squares(double acc, const f32x4 (&v)[kGroups]) {
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double d = (double)v[u][k];  // the square is exact in fp64
      acc = __builtin_fma(d, d, acc);
    }
  }
  return acc;
}

// Sum of this lane's squares of a row, `left` of whose elements there are.
template <typename GT>
__device__ __forceinline__ double row_sum(const GT* p, int left, int at) {
  f32x4 v[kGroups];
  if (left >= kRowElems) {
#pragma unroll
    for (int u = 0; u < kGroups; ++u) v[u] = load4(p + u * kScaleElems);
  } else {
#pragma unroll
    for (int u = 0; u < kGroups; ++u) v[u] = load_some(p + u * kScaleElems,
                                                       left - u * kScaleElems - at);
  }
  return add_squares(0.0, v);
}

// In front of a step (BACKWARDS) a span's chunks go from the last to the first
// and are loaded through the caches: the step starts on the gradients that were
// read last and finds part of them in the 256 MB memory-side cache.  Clipped
// steps with that, backwards past the caches, and forwards past them: 334M
// parameters 1457, 1477 and 1478 us (32-bit states, bfloat16 gradients), 1085,
// 1098 and 1100 (8-bit, fp32), 13M in 61 tensors 73.2, 74.8 and 75.0, 38.7, 38.8
// and 39.6; 1.56B parameters 7.635, 7.641 and 7.643 ms, but with 8-bit states
// 3.031, 3.012 and 3.016.  A norm on its own goes forwards past the caches, 1 %
// faster than backwards (6.2 GB: 936 and 945 us).
template <typename GT, bool BACKWARDS>
__global__ void __launch_bounds__(kBlock)
    norm_kernel(NormPtrs ptrs, const ChunkRec* __restrict__ recs, uint32_t t0, int64_t c0,
                int64_t n, double* __restrict__ partials) {
  __shared__ double red[kBlock / 64];
  const int wave = wave_in_block();
  const int at = (threadIdx.x & 63) * 4;
  const auto chunk = [&](int64_t i) { return BACKWARDS ? c0 + n - 1 - i : c0 + i; };
  double acc = 0.0;
  int64_t i = blockIdx.x;
  ChunkRec rec = recs[chunk(i)];
  const GT* g = (const GT*)ptrs.g[rec.tensor - t0];
  while (i < n) {
    const int left = g == nullptr ? 0 : (int)rec.count - wave * kRowElems;
    const GT* p = g + ((int64_t)rec.row + wave) * kRowElems + at;
    f32x4 v[kGroups];
    if (left >= kRowElems) {
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if constexpr (BACKWARDS) v[u] = load4_cached(p + u * kScaleElems);
        else v[u] = load4(p + u * kScaleElems);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kGroups; ++u) v[u] = load_some(p + u * kScaleElems,
                                                         left - u * kScaleElems - at);
    }
    // the next chunk's record and pointer arrive while this one's data do
    i += gridDim.x;
    if (i < n) {
      rec = recs[chunk(i)];
      g = (const GT*)ptrs.g[rec.tensor - t0];
    }
    acc = add_squares(acc, v);
  }
  acc = block_sum(acc, red);
  if (threadIdx.x == 0) partials[blockIdx.x] = acc;
}

// Sum of n partials by one block, in an order fixed by n.  Eight loads are
// under way at a time: with one, 2048 partials took 5 us, a tenth of a clipped
// step over 13M parameters.
__device__ __forceinline__ double fold_partials(const double* partials, int64_t n, double* red) {
  double acc = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 8 * kBlock) {
    double p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = i + k * kBlock < n ? partials[i + k * kBlock] : 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc = acc + p[k];
  }
  return block_sum(acc, red);
}

__global__ void __launch_bounds__(kBlock)
    norm_finish_kernel(const double* __restrict__ partials, int64_t n, float grad_scale,
                       double* sumsq, float* norm) {
  __shared__ double red[kBlock / 64];
  const double total = fold_partials(partials, n, red);
  if (threadIdx.x != 0) return;
  if (sumsq != nullptr) *sumsq = total;
  if (norm != nullptr) *norm = (float)(sqrt(total) * (double)grad_scale);
}

__device__ __forceinline__ uint64_t mix64(uint64_t z, uint64_t mul) {
  z ^= z >> 31;
  return z * mul;
}

// What a step does with S: the clipping factor, the bias corrections and the
// keys of its random bits, from the counts before it.
struct Derived {
  double norm, p1, p2;
  float gscale, rbc2;
  uint32_t k0, k1;
  bool skip;
};
__device__ __forceinline__ Derived derive(const ControlArgs& a, double total, int64_t steps,
                                          double p1, double p2) {
  Derived d;
  d.norm = sqrt(total) * (double)a.grad_scale;
  d.skip = a.skip_nonfinite && !(total <= 1.7976931348623157e308);
  d.p1 = p1 * (double)a.beta1;
  d.p2 = p2 * (double)a.beta2;
  double coef = 1.0;
  if (a.max_norm > 0.0f && !(d.norm <= (double)a.max_norm)) coef = (double)a.max_norm / d.norm;
  d.gscale = (float)((double)a.grad_scale * coef);
  d.rbc2 = (float)(1.0 / sqrt(1.0 - d.p2));
  // the multipliers are digits of the square roots of 2, 3 and 5
  uint64_t z = a.seed * 0x6A09E667F3BCC909ull + (uint64_t)(steps + 1) * 0xBB67AE8584CAA73Bull;
  z = mix64(z, 0x3C6EF372FE94F82Bull);
  z = mix64(z, 0x6A09E667F3BCC909ull);
  z ^= z >> 32;
  d.k0 = (uint32_t)z;
  d.k1 = (uint32_t)(z >> 32);
  return d;
}
// The factors of group i.  A NaN rate becomes the canonical one: stochastic
// rounding adds to bit patterns and must not carry out of a NaN.
__device__ __forceinline__ void derive_group(const ControlArgs& a, int i, double p1, float* decay,
                                             float* rate) {
  double lr = (double)(a.lr_device != nullptr ? a.lr_device[i] : a.lr[i]);
  if (lr != lr) lr = __builtin_nan("");
  *decay = (float)(1.0 - lr * (double)a.wd[i]);
  *rate = (float)(lr / (1.0 - p1));
}

// One block: S and the scalars of the step that follows on the stream.
__global__ void __launch_bounds__(kBlock) control_kernel(Control* c, ControlArgs a) {
  __shared__ double red[kBlock / 64];
  double total = 0.0;
  if (a.partials != nullptr) {
    total = fold_partials(a.partials, a.n_partials, red);
  } else if (a.sumsq != nullptr) {
    total = *a.sumsq;
  }
  const int64_t steps = c->steps;
  const Derived d = derive(a, total, steps, c->p1, c->p2);
  __syncthreads();  // every thread has read the counts before thread 0 writes
  if ((int)threadIdx.x < a.n_groups)
    derive_group(a, threadIdx.x, d.p1, &c->decay[threadIdx.x], &c->rate[threadIdx.x]);
  if (threadIdx.x != 0) return;
  if (a.norm != nullptr) *a.norm = (float)d.norm;
  c->skip = d.skip ? 1u : 0u;
  if (d.skip) {
    c->skipped += 1;
    return;
  }
  c->gscale = d.gscale;
  c->rbc2 = d.rbc2;
  c->k0 = d.k0;
  c->k1 = d.k1;
  c->steps = steps + 1;
  c->p1 = d.p1;
  c->p2 = d.p2;
}

// ---------------------------------------------------------- small launches --
// Loads and stores past the caches, which each XCD has of its own: what one
// block leaves here another finds, once the store is done.
template <typename T>
__device__ __forceinline__ T ld_shared_state(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(double* p, double v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // done before what follows
}

// True for the last of `all` callers: each adds `one` (1) once, in one counter
// where they are few, else over kLeaves of them whose last callers meet at a
// root (a counter takes an atomic every 12 ns).  The counters are left at 0.
// `id` numbers the callers from 0.
__device__ __forceinline__ bool last_ticket(Control* c, uint32_t id, uint32_t all, uint32_t one) {
  const uint32_t leaves = all > 64 ? kLeaves : 1;
  const uint32_t leaf = id % leaves;
  const uint32_t n = __hip_atomic_fetch_add(&c->leaf[leaf][0], one, __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT);
  if (n != (all + leaves - 1 - leaf) / leaves - 1) return false;
  c->leaf[leaf][0] = 0;
  if (leaves == 1) return true;
  if (__hip_atomic_fetch_add(&c->root, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) !=
      leaves - 1)
    return false;
  c->root = 0;
  return true;
}

// Control and update in one launch, for the latency of steps over few
// elements.  Every wave derives the scalars for itself from the counts before
// the step while its row is being loaded, and takes a ticket once it has
// them; the wave with the last ticket moves the counts on.  Nothing waits for
// another wave.
template <typename PT, typename GT, int BITS, bool MASTER, bool SR, int GROUPS>
__global__ void __launch_bounds__(kBlock) small_step_kernel(SmallStep k) {
  constexpr int kShare = GROUPS * kScaleElems;             // of a wave
  constexpr int kWaves = kChunkElems / kShare;             // of a chunk
  const int id = blockIdx.x * (kBlock / 64) + wave_in_block();
  const ChunkRec rec = k.s.recs[id / kWaves];
  const GT* g = (const GT*)k.g[rec.tensor];
  PT* p = (PT*)k.p[rec.tensor];
  const ControlArgs& a = k.a;
  Control* ctl = k.s.control;
  const int lane = threadIdx.x & 63;
  const int begin = id % kWaves * kShare;
  const int left = (int)rec.count - begin;
  const int64_t steps = ld_shared_state(&ctl->steps);
  const double p1 = ld_shared_state(&ctl->p1), p2 = ld_shared_state(&ctl->p2);
  double part = 0.0;
  if (a.partials != nullptr) {
    for (int i = lane; i < (int)a.n_partials; i += 64) part = part + a.partials[i];
  } else if (a.sumsq != nullptr && lane == 0) {
    part = *a.sumsq;
  }
  const auto scalars = [&] {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) part = part + __shfl_xor(part, o, 64);
    const Derived d = derive(a, part, steps, p1, p2);
    Scalars c;
    derive_group(a, rec.group, d.p1, &c.decay, &c.rate);
    c.gs = d.gscale;
    c.rbc2 = d.rbc2;
    c.key0 = d.k0;
    c.key1 = d.k1;
    c.skip = d.skip;
    if (lane == 0) {
      // What is added depends on the loaded counts, so the ticket is taken
      // after they have arrived; none of them is ever negative.
      const uint32_t one = steps >= 0 && p1 >= 0.0 && p2 >= 0.0 ? 1u : 2u;
      if (last_ticket(ctl, id, gridDim.x * (kBlock / 64), one)) {
        if (a.norm != nullptr) *a.norm = (float)d.norm;
        if (d.skip) {
          ctl->skipped += 1;
        } else {
          ctl->steps = steps + 1;
          ctl->p1 = d.p1;
          ctl->p2 = d.p2;
        }
      }
    }
    return c;
  };
  if (g == nullptr || left <= 0) {
    scalars();
    return;
  }
  step_wave<PT, GT, BITS, MASTER, SR, GROUPS>(g, p, k.s, rec.row, rec.state_row, begin, left,
                                              scalars);
}

// A chunk a block; the block with the last ticket, which each takes when its
// partial sum has been stored, folds the sums.  At 256 chunks 4.4 us, 7.9 with
// tickets that release and acquire (they write back and empty an L2 each), 6.1
// with a kernel for the fold.
template <typename GT>
__global__ void __launch_bounds__(kBlock) small_norm_kernel(SmallNorm k) {
  __shared__ double red[kBlock / 64];
  __shared__ bool last;
  const ChunkRec rec = k.recs[blockIdx.x];
  const GT* g = (const GT*)k.g[rec.tensor];
  const int wave = wave_in_block();
  const int at = (threadIdx.x & 63) * 4;
  const int left = g == nullptr ? 0 : (int)rec.count - wave * kRowElems;
  const double acc = block_sum(row_sum(g + ((int64_t)rec.row + wave) * kRowElems + at, left, at),
                               red);
  if (threadIdx.x == 0) {
    publish(k.partials + blockIdx.x, acc);
    last = last_ticket(k.control, blockIdx.x, gridDim.x, 1u);
  }
  __syncthreads();
  if (!last) return;
  static_assert(kSmallChunks <= kBlock, "a partial sum a thread");
  const double total = block_sum(
      threadIdx.x < gridDim.x ? ld_shared_state(k.partials + threadIdx.x) : 0.0, red);
  if (threadIdx.x != 0) return;
  if (k.sumsq != nullptr) *k.sumsq = total;
  if (k.norm != nullptr) *k.norm = (float)(sqrt(total) * (double)k.grad_scale);
}

__global__ void set_steps_kernel(Control* c, int64_t steps, double p1, double p2) {
  c->steps = steps;
  c->skipped = 0;
  c->p1 = p1;
  c->p2 = p2;
}

__global__ void __launch_bounds__(kBlock)
    fill_kernel(uint32_t* __restrict__ dst, uint32_t word, uint64_t words) {
  const uint64_t stride = (uint64_t)gridDim.x * kBlock;
  for (uint64_t k = (uint64_t)blockIdx.x * kBlock + threadIdx.x; k < words; k += stride)
    dst[k] = word;
}

__global__ void __launch_bounds__(kBlock)
    master_kernel(StepPtrs ptrs, State s, uint32_t t0, int64_t c0) {
  const ChunkRec rec = s.recs[c0 + blockIdx.x];
  const bf16* p = (const bf16*)ptrs.p[rec.tensor - t0] + (int64_t)rec.row * kRowElems;
  float* dst = s.master + (int64_t)rec.state_row * kRowElems;
  for (int k = threadIdx.x; k < (int)rec.count; k += kBlock) dst[k] = widen(p[k]);
}

// ------------------------------------------------------- state in and out --
template <int BITS, int FIELD>
__device__ __forceinline__ float state_value(const State& s, int64_t i) {
  if constexpr (FIELD == OB_ADAMW_MASTER) {
    return s.master[i];
  } else if constexpr (BITS == 32) {
    return ((const float*)(FIELD == OB_ADAMW_M ? s.m : s.v))[i];
  } else if constexpr (FIELD == OB_ADAMW_M) {
    return decode_m(((const uint8_t*)s.m)[i], s.m_exp[i / kScaleElems]).x;
  } else {
    return decode_v(((const uint8_t*)s.v)[i], s.v_exp[i / kScaleElems]).x;
  }
}

// Any offset and alignment, an element a thread; `done` elements of dst are
// there already.
template <int BITS, int FIELD, bool BF16>
__global__ void __launch_bounds__(kBlock)
    get_kernel(State s, int64_t offset, int64_t done, int64_t count, void* __restrict__ dst) {
  const int64_t stride = (int64_t)gridDim.x * kBlock;
  for (int64_t k = done + (int64_t)blockIdx.x * kBlock + threadIdx.x; k < count; k += stride) {
    const float v = state_value<BITS, FIELD>(s, offset + k);
    if constexpr (BF16)
      ((uint16_t*)dst)[k] = (uint16_t)pack_bf16(v, 0.0f);
    else
      ((float*)dst)[k] = v;
  }
}

// `eights` runs of 8 elements from a multiple of 8 into a 16-byte aligned dst,
// one a thread and round, all of a thread's loads ahead of its stores: 1.56B
// codes to bfloat16 in 0.77 ms (6.0 TB/s; 0.89 ms with one run a round over a
// grid of 8192 blocks).
constexpr int kGetRounds = 4;
constexpr int kGetElems = 8 * kBlock * kGetRounds;
constexpr int64_t kGetBlocks = int64_t(1) << 22;  // of one launch, far below the grid's limit

template <int BITS, int FIELD, bool BF16>
__global__ void __launch_bounds__(kBlock)
    get_blocks_kernel(State s, int64_t offset, int64_t eights, void* __restrict__ dst) {
  const int64_t first = (int64_t)blockIdx.x * (kGetElems / 8) + threadIdx.x;
  constexpr bool kF32 = FIELD == OB_ADAMW_MASTER || BITS == 32;
  const void* src = FIELD == OB_ADAMW_MASTER ? s.master : (FIELD == OB_ADAMW_M ? s.m : s.v);
  f32x4 a[kGetRounds], b[kGetRounds];
  u32x2 c[kGetRounds];
  uint32_t e[kGetRounds];
#pragma unroll
  for (int r = 0; r < kGetRounds; ++r) {
    if (first + r * kBlock >= eights) break;
    const int64_t i = offset + 8 * (first + r * kBlock);
    if constexpr (kF32) {
      a[r] = load4((const float*)src + i);
      b[r] = load4((const float*)src + i + 4);
    } else {
      c[r] = ld_stream((const u32x2*)((const uint8_t*)src + i));
      e[r] = (FIELD == OB_ADAMW_M ? s.m_exp : s.v_exp)[i / kScaleElems];
    }
  }
#pragma unroll
  for (int r = 0; r < kGetRounds; ++r) {
    const int64_t k = first + r * kBlock;
    if (k >= eights) break;
    if constexpr (!kF32) {
      a[r] = FIELD == OB_ADAMW_M ? decode_m(c[r].x, e[r]) : decode_v(c[r].x, e[r]);
      b[r] = FIELD == OB_ADAMW_M ? decode_m(c[r].y, e[r]) : decode_v(c[r].y, e[r]);
    }
    if constexpr (BF16) {
      st_stream((u32x4*)dst + k, u32x4{pack_bf16(a[r].x, a[r].y), pack_bf16(a[r].z, a[r].w),
                                       pack_bf16(b[r].x, b[r].y), pack_bf16(b[r].z, b[r].w)});
    } else {
      st_stream((f32x4*)dst + 2 * k, a[r]);
      st_stream((f32x4*)dst + 2 * k + 1, b[r]);
    }
  }
}

// Whole groups of 256, one per wave and round, from fp32.
template <int FIELD>
__global__ void __launch_bounds__(kBlock)
    set_codes_kernel(State s, int64_t group0, int64_t groups, const float* __restrict__ src) {
  const int wave = wave_in_block();
  const int lane = threadIdx.x & 63;
  for (int64_t i = (int64_t)blockIdx.x * (kBlock / 64) + wave; i < groups;
       i += (int64_t)gridDim.x * (kBlock / 64)) {
    f32x4 x = load_some(src + i * kScaleElems + lane * 4, 4);
    uint32_t e, c;
    if constexpr (FIELD == OB_ADAMW_M) {
      c = encode_m(x, top_m(x), &e);
    } else {
      uint32_t q[4], top = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = x[k] <= 0.0f ? 0.0f : x[k];  // NaN stays
        q[k] = rounded_v(x[k], 1u << 19);   // to nearest
        top = umax(top, q[k]);
      }
      c = encode_v(x, q, wave_max(top), &e);
    }
    const int64_t at = group0 + i;
    ((uint32_t*)(FIELD == OB_ADAMW_M ? s.m : s.v))[at * 64 + lane] = c;
    if (lane == 0) (FIELD == OB_ADAMW_M ? s.m_exp : s.v_exp)[at] = (uint8_t)e;
  }
}

__global__ void __launch_bounds__(kBlock)
    set_f32_kernel(float* __restrict__ dst, int64_t count, const float* __restrict__ src,
                   int non_negative) {
  const int64_t stride = (int64_t)gridDim.x * kBlock;
  for (int64_t k = (int64_t)blockIdx.x * kBlock + threadIdx.x; k < count; k += stride) {
    const float x = src[k];
    dst[k] = non_negative && x <= 0.0f ? 0.0f : x;
  }
}

int grid_for(int64_t threads) {
  const int64_t blocks = (threads + kBlock - 1) / kBlock;
  return (int)(blocks < 1 ? 1 : (blocks > 8192 ? 8192 : blocks));
}

// A wave of a small step takes one group where there are so few chunks, four
// else: the latency of one wave's instructions shows below, four times the
// tickets above.  One and four groups, 32-bit states: 16 chunks 4.4 and 5.3 us,
// 64 chunks 5.8 and 6.0, 128 chunks 7.4 and 6.5, 256 chunks 10.6 and 7.3; 8-bit
// ones: 4.4 and 5.8, 5.7 and 5.9, 7.0 and 6.4, 10.2 and 7.4.
constexpr int64_t kFewChunks = 64;

// fn(types and kinds of the plan's step as compile-time values).
template <typename PT, typename GT, int BITS, bool MASTER, bool SR>
struct Kind {
  static void step(const StepPtrs& ptrs, const State& s, uint32_t t0, int64_t c0, int64_t n,
                   hipStream_t stream) {
    step_kernel<PT, GT, BITS, MASTER, SR>
        <<<(unsigned)n * kStepBlocks<BITS>, kBlock, 0, stream>>>(ptrs, s, t0, c0);
  }
  static void small(const SmallStep& k, int64_t n, hipStream_t stream) {
    if (n <= kFewChunks)
      small_step_kernel<PT, GT, BITS, MASTER, SR, 1>
          <<<(unsigned)n * kGroups, kBlock, 0, stream>>>(k);
    else
      small_step_kernel<PT, GT, BITS, MASTER, SR, kGroups><<<(unsigned)n, kBlock, 0, stream>>>(k);
  }
};
template <typename PT, typename GT, int BITS, typename F>
void with_rounding(const State& s, F fn) {
  if constexpr (sizeof(PT) == 2) {
    if (s.has_master) return fn(Kind<PT, GT, BITS, true, false>());
    if (s.stochastic) return fn(Kind<PT, GT, BITS, false, true>());
  }
  fn(Kind<PT, GT, BITS, false, false>());
}
template <int BITS, typename F>
void with_types(const State& s, F fn) {
  if (s.param_bf16)
    s.grad_bf16 ? with_rounding<bf16, bf16, BITS>(s, fn) : with_rounding<bf16, float, BITS>(s, fn);
  else
    s.grad_bf16 ? with_rounding<float, bf16, BITS>(s, fn)
                : with_rounding<float, float, BITS>(s, fn);
}
template <typename F>
hipError_t with_kind(const State& s, F fn) {
  s.state_bits == 32 ? with_types<32>(s, fn) : with_types<8>(s, fn);
  return hipGetLastError();
}

template <int BITS, int FIELD, bool BF16>
hipError_t get_as(const State& s, int64_t offset, int64_t count, void* dst, hipStream_t stream) {
  int64_t done = 0;
  if (offset % 8 == 0 && (uintptr_t)dst % 16 == 0) {
    const int64_t eights = count / 8, per = kGetBlocks * (kGetElems / 8);
    for (int64_t at = 0; at < eights; at += per) {
      const int64_t n = eights - at < per ? eights - at : per;
      const unsigned grid = (unsigned)((n + kGetElems / 8 - 1) / (kGetElems / 8));
      get_blocks_kernel<BITS, FIELD, BF16><<<grid, kBlock, 0, stream>>>(
          s, offset + 8 * at, n, (char*)dst + 8 * at * (BF16 ? 2 : 4));
    }
    done = 8 * eights;
  }
  if (done < count)
    get_kernel<BITS, FIELD, BF16><<<grid_for(count - done), kBlock, 0, stream>>>(s, offset, done,
                                                                              count, dst);
  return hipGetLastError();
}
template <int BITS, int FIELD>
hipError_t get_of(const State& s, int64_t offset, int64_t count, bool bf16_out, void* dst,
                  hipStream_t stream) {
  return bf16_out ? get_as<BITS, FIELD, true>(s, offset, count, dst, stream)
                  : get_as<BITS, FIELD, false>(s, offset, count, dst, stream);
}

}  // namespace

hipError_t launch_step(const State& s, const StepPtrs& ptrs, uint32_t t0, int64_t c0, int64_t n,
                       hipStream_t stream) {
  return with_kind(s, [&](auto kind) { kind.step(ptrs, s, t0, c0, n, stream); });
}

hipError_t launch_small(const SmallStep& k, int64_t n, hipStream_t stream) {
  return with_kind(k.s, [&](auto kind) { kind.small(k, n, stream); });
}

hipError_t launch_norm(const State& s, const NormPtrs& ptrs, uint32_t t0, int64_t c0, int64_t n,
                       int64_t at, bool backwards, hipStream_t stream) {
  const unsigned grid = (unsigned)norm_partials(n);
  const auto kernel =
      s.grad_bf16 ? (backwards ? norm_kernel<bf16, true> : norm_kernel<bf16, false>)
                  : (backwards ? norm_kernel<float, true> : norm_kernel<float, false>);
  kernel<<<grid, kBlock, 0, stream>>>(ptrs, s.recs, t0, c0, n, s.partials + at);
  return hipGetLastError();
}

hipError_t launch_control(const State& s, const ControlArgs& a, hipStream_t stream) {
  control_kernel<<<1, kBlock, 0, stream>>>(s.control, a);
  return hipGetLastError();
}

hipError_t launch_norm_finish(const State& s, int64_t n_partials, float grad_scale, double* sumsq,
                              float* norm, hipStream_t stream) {
  norm_finish_kernel<<<1, kBlock, 0, stream>>>(s.partials, n_partials, grad_scale, sumsq, norm);
  return hipGetLastError();
}

hipError_t launch_small_norm(const SmallNorm& k, bool grad_bf16, int64_t n, hipStream_t stream) {
  if (grad_bf16)
    small_norm_kernel<bf16><<<(unsigned)n, kBlock, 0, stream>>>(k);
  else
    small_norm_kernel<float><<<(unsigned)n, kBlock, 0, stream>>>(k);
  return hipGetLastError();
}

hipError_t launch_set_steps(const State& s, int64_t steps, double p1, double p2,
                            hipStream_t stream) {
  set_steps_kernel<<<1, 1, 0, stream>>>(s.control, steps, p1, p2);
  return hipGetLastError();
}

hipError_t launch_fill(void* dst, uint32_t word, uint64_t words, hipStream_t stream) {
  if (words == 0) return hipSuccess;
  fill_kernel<<<grid_for((int64_t)words), kBlock, 0, stream>>>((uint32_t*)dst, word, words);
  return hipGetLastError();
}

hipError_t launch_master(const State& s, const StepPtrs& ptrs, uint32_t t0, int64_t c0, int64_t n,
                         hipStream_t stream) {
  master_kernel<<<(unsigned)n, kBlock, 0, stream>>>(ptrs, s, t0, c0);
  return hipGetLastError();
}

hipError_t launch_get(const State& s, int field, int64_t offset, int64_t count, bool bf16_out,
                      void* dst, hipStream_t stream) {
  if (field == OB_ADAMW_MASTER)
    return get_of<32, OB_ADAMW_MASTER>(s, offset, count, bf16_out, dst, stream);
  if (s.state_bits == 32)
    return field == OB_ADAMW_M ? get_of<32, OB_ADAMW_M>(s, offset, count, bf16_out, dst, stream)
                               : get_of<32, OB_ADAMW_V>(s, offset, count, bf16_out, dst, stream);
  return field == OB_ADAMW_M ? get_of<8, OB_ADAMW_M>(s, offset, count, bf16_out, dst, stream)
                             : get_of<8, OB_ADAMW_V>(s, offset, count, bf16_out, dst, stream);
}

hipError_t launch_set(const State& s, int field, int64_t offset, int64_t count, const float* src,
                      hipStream_t stream) {
  if (field != OB_ADAMW_MASTER && s.state_bits == 8) {
    const int64_t groups = count / kScaleElems;
    const int grid = grid_for(groups * 64);
    if (field == OB_ADAMW_M)
      set_codes_kernel<OB_ADAMW_M><<<grid, kBlock, 0, stream>>>(s, offset / kScaleElems, groups,
                                                                src);
    else
      set_codes_kernel<OB_ADAMW_V><<<grid, kBlock, 0, stream>>>(s, offset / kScaleElems, groups,
                                                                src);
    return hipGetLastError();
  }
  float* dst = field == OB_ADAMW_MASTER ? s.master
                                        : (float*)(field == OB_ADAMW_M ? s.m : s.v);
  set_f32_kernel<<<grid_for(count), kBlock, 0, stream>>>(dst + offset, count, src,
                                                         field == OB_ADAMW_V);
  return hipGetLastError();
}

}  // namespace adamw
}  // namespace ob
