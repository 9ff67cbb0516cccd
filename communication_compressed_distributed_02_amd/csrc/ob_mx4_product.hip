// gfx950 kernels of the product of two matrices in microscaled 4-bit floating
// point, out = a b^T.  The arithmetic contract is stated in include/ob_mx4.h.
//
// The matrix instruction takes 32 rows of each side by 64 elements of the sum,
// 4 bits each, with a scale byte for every row's 32: lane l holds row l % 32,
// elements 32 * (l / 32) to + 31 (16 bytes), and that block's scale.  b is its
// first operand, so that the four consecutive results of a lane lie along a row
// of out: lane l has row l % 32 of a, register 4 * q + i row 8 * q + 4 * (l /
// 32) + i of b.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ob_mx4_device.h"
#include "ob_mx4_kernels.h"

namespace ob {
namespace mx4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;       // the instruction's number for these elements

// acc += 32 x 32 products over 64 elements; the scales are byte BYTE of sa, sb.
template <int BYTE>
__device__ __forceinline__ f32x16 multiply(u32x4 b, u32x4 a, f32x16 acc, uint32_t sb, uint32_t sa) {
  const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc, kFp4, kFp4, BYTE, (int)sb,
                                                         BYTE, (int)sa);
}

// acc += 16 x 16 products over 128 elements.
__device__ __forceinline__ f32x4 multiply16(u32x4 b, u32x4 a, f32x4 acc, uint32_t sb, uint32_t sa) {
  const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, acc, kFp4, kFp4, 0, (int)sb, 0,
                                                          (int)sa);
}

template <AType A>
struct Raw {
  typedef float type;
};
template <>
struct Raw<kABf16> {
  typedef bf16 type;
};

__device__ __forceinline__ void store_wide(float* p, const float* c, std::integral_constant<int, 4>) {
  *(f32x4_at4*)p = f32x4{c[0], c[1], c[2], c[3]};
}
__device__ __forceinline__ void store_wide(bf16* p, const float* c, std::integral_constant<int, 8>) {
  store8(p, c);
}
__device__ __forceinline__ void store_wide(bf16* p, const float* c, std::integral_constant<int, 4>) {
  *(u32x2_at2*)p = u32x2{pack_bf16(c[0], c[1]), pack_bf16(c[2], c[3])};
}

// N results from column `at` on of a row of out, of which `left` columns exist.
template <int N, typename T>
__device__ __forceinline__ void write_out(T* row, int at, int64_t left, int32_t accumulate,
                                          float* v) {
  if (at >= left) return;
  T* out = row + at;
  if (accumulate) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at + k < left) v[k] += widen(out[k]);
  }
  if (at + N <= left) {
    store_wide(out, v, std::integral_constant<int, N>());
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at + k < left) store1(out + k, v[k]);
  }
}

// Products with few rows of a (m <= 16 * MT), bound by reading b: a block takes 16
// rows of b, its waves every kWaves-th 256 elements of the sum (lines of 128
// bytes), kAhead of them in loads at a time, and they add up through LDS in their
// order.  The instruction of 16 rows by 16 and 128 elements: lane l holds row
// l % 16, elements 32 * (l / 16) to + 31 and their scale; of the results, row
// l % 16 of a and 4 * (l / 16) + i of b.  An a that is not quantised is, by every
// block for itself, into LDS, while its first loads of b are on their way.
// One row through 6400 x 1600 3.2 us (3.8 with its quantising), of which a launch
// is 2; through 4096 x 4096 4.0, 16 rows 4.9.
constexpr int kWaves = 8, kAhead = 2;
template <int MT, AType A, typename T>
__global__ void __launch_bounds__(kWaves * 64) narrow_kernel(ProductArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = (int)threadIdx.x & 63, row = lane & 15, block = lane >> 4;
  const int64_t rc = row_codes(p.k), rs = row_scales(p.k);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int units = (int)(rc / 64), pairs = (units + 1) / 2;  // of 128 elements, of 256
  // rows behind the last are read as the last, and their results dropped
  const int64_t bn = n0 + row < p.n ? n0 + row : p.n - 1;
  const uint8_t* b_codes = p.b_codes + bn * rc + block * 16;
  const uint8_t* b_scales = p.b_scales + bn * rs;
  u32x4 b[kAhead][2];
  u32x2 sb[kAhead];
  const auto load = [&](int p0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = p0 + i * kWaves;
      if (at >= pairs) continue;
      b[i][0] = *(const u32x4*)(b_codes + (int64_t)at * 128);
      if (2 * at + 1 < units) b[i][1] = *(const u32x4*)(b_codes + (int64_t)at * 128 + 64);
      sb[i] = *(const u32x2*)(b_scales + (int64_t)at * 8);
    }
  };
  load(wave);
  // rows of a in LDS: codes, 16 bytes apart so that rows start in other banks,
  // then the scales
  const int lc = units * 64 + 16, ls = pairs * 8;
  uint8_t* lds_scales = lds + (int)p.m * lc;
  if constexpr (A != kAPacked) {
    using X = typename Raw<A>::type;
    const int groups = units * 16;  // of 8 elements; a block's four lie on a quad of lanes
    for (int i = (int)threadIdx.x; i < (int)p.m * groups; i += kWaves * 64) {
      const int r = i / groups, at = i - r * groups;
      const int64_t k = (int64_t)at * 8;
      const X* x = (const X*)p.a + r * p.a_stride + k;
      float c[8];
      if (k + 8 <= p.k)
        load8(x, c);
      else
        load8_some(x, (int)(p.k > k ? p.k - k : 0), c);
      const uint32_t byte = scale_byte<false>(quad_max(largest<8>(c)));
      *(uint32_t*)(lds + r * lc + at * 4) = encode8(c, byte);
      lds_scales[r * ls + at / 4] = (uint8_t)byte;
    }
    __syncthreads();
  }
  int am[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) am[i] = i * 16 + row < (int)p.m ? i * 16 + row : (int)p.m - 1;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int p0 = wave; p0 < pairs; p0 += kAhead * kWaves) {
    if (p0 != wave) load(p0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = p0 + i * kWaves;
      if (at >= pairs) continue;
      const bool two = 2 * at + 1 < units;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const uint8_t *codes, *scales;
        if constexpr (A == kAPacked) {
          codes = p.a_codes + am[j] * rc + (int64_t)at * 128 + block * 16;
          scales = p.a_scales + am[j] * rs + (int64_t)at * 8;
        } else {
          codes = lds + am[j] * lc + at * 128 + block * 16;
          scales = lds_scales + am[j] * ls + at * 8;
        }
        const u32x2 sa = *(const u32x2*)scales;
        acc[j] = multiply16(b[i][0], *(const u32x4*)codes, acc[j], sb[i].x >> (8 * block),
                            sa.x >> (8 * block));
        if (two)
          acc[j] = multiply16(b[i][1], *(const u32x4*)(codes + 64), acc[j], sb[i].y >> (8 * block),
                              sa.y >> (8 * block));
      }
    }
  }
  if constexpr (A != kAPacked) __syncthreads();
  f32x4* part = (f32x4*)lds;
#pragma unroll
  for (int j = 0; j < MT; ++j) part[(wave * MT + j) * 64 + lane] = acc[j];
  __syncthreads();
  if (wave >= MT) return;
  f32x4 sum = part[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += part[(w * MT + wave) * 64 + lane];
  const int64_t i = wave * 16 + row, j = n0 + 4 * block;
  float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  if (i < p.m) write_out<4>((T*)p.out + i * p.out_stride + j, 0, p.n - j, p.accumulate, v);
}

// Large products.  A block of WM x WN waves takes a tile of TM x TN, each wave
// MT x NT of the instruction's tiles, so that a 16-byte read from LDS feeds NT (or
// MT) instructions.  Codes come into LDS by direct loads in units of 256 elements
// (whole lines of 128 bytes), STAGES units deep, scales for two units at a time, 16
// bytes a row.  A unit is multiplied in four steps of 64 elements; during each
// the next one's registers are read.  At the end of the third step a unit is
// in registers altogether: one barrier, behind which the next unit is there and
// the one STAGES behind may be loaded over this one.  A row's eight 16-byte pieces
// lie in LDS permuted by (row / 2) % 8: lanes of consecutive rows that read the
// same piece then meet all banks evenly.  The permutation is made by the
// addresses that the lanes load from, since direct loads write LDS in the order
// of the lanes.
//
// 256 x 256 (8 waves of 128 x 64): 8192 x 8192 x 16384 in 465-485 us, 4.55-4.72
// PFLOP/s, with operands in the caches, in 509-547 out of memory.  The instruction alone, on random operands in registers, makes 6.2
// (355 us): the card lowers its clock for it, from 2.4 to 1.6 GHz (9.0 on constant
// ones); without its loads the kernel takes 375-390: what separates it from the
// instruction are loads that arrive late, the matrix pipes are busy in 62 % of the
// cycles.  With units of 128 elements,
// half a line each, it took 577, and 514 once the loads and reads were spread
// among the products.  128 x 128 (4 waves of 64 x 64, two blocks on a CU) moves
// twice as much into LDS: 623.  Where there is one block of those for a CU at most
// and the sum is long, four units lie in LDS and three of them are on their way, for
// a unit takes less time there than a load: 1600 x 1600 x 16384 40 us, with two 51.  Short sums are bound by writing out: 16384 x
// 6400 x 1600 117 us, 210 MB of them.  Results that went out from the registers,
// in pieces of 32 bytes: 133; blocks that went on from tile to tile: 117.
template <int WM_, int WN_, int MT_, int NT_, int STAGES_>
struct Tile {
  static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
  static constexpr int STAGES = STAGES_;  // units in LDS
  static constexpr int TM = WM * MT * 32, TN = WN * NT * 32, WAVES = WM * WN;
  static constexpr int LA = TM / 8 / WAVES, LB = TN / 8 / WAVES;  // loads of a unit, a wave
  static constexpr int SCALE_CHUNKS = (TM + TN) / 64;             // loads of two units' scales
  static constexpr int LS = (SCALE_CHUNKS + WAVES - 1) / WAVES;
  static constexpr int UNIT = (TM + TN) * 128, SCALES = (TM + TN) * 16;
  static constexpr int STRIP = NT * 32 + 4;  // floats of a row on the way out
  static constexpr int LOOP_BYTES = STAGES * (UNIT + SCALES);
  static constexpr int OUT_BYTES = WAVES * 32 * STRIP * 4;
  static constexpr int LDS = LOOP_BYTES > OUT_BYTES ? LOOP_BYTES : OUT_BYTES;
  static_assert(LA % 2 == 0 && LB % 2 == 0 && TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0, "");
  static_assert(LDS <= 160 * 1024, "");
};

// 16 bytes of each of the lanes in `lanes` (uniform) from base + offset into LDS
// at `lds`, in the lanes' order.  With no lane it moves nothing.  m0 is named as
// written, so that no use of the compiler's own is moved around it; that it is not
// preserved, of which the compiler warns, is what is meant.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds,
                                            uint64_t lanes) {
  uint64_t all;
  asm volatile(
      "s_mov_b32 m0, %1\n\ts_mov_b64 %0, exec\n\ts_mov_b64 exec, %4\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %2, %3\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "s"(lds), "v"(offset), "s"(base), "s"(lanes)
      : "memory", "m0");
}
#pragma clang diagnostic pop
// This wave's reads are done, and its loads but for the last N, and so are those of
// all the block's waves.  Not `steady` (uniform): all loads, since some of the last N
// may have had no lanes.  The branch stays in here, unseen by the compiler, which would
// move products past it.
template <int N>
__device__ __forceinline__ void arrived(bool steady) {
  if constexpr (N == 0) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  } else {
    const int s = __builtin_amdgcn_readfirstlane(steady ? 1 : 0);
    asm volatile(
        "s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(0)\n1:\n\t"
        "s_waitcnt vmcnt(%1) lgkmcnt(0)\n\ts_barrier" ::"s"(s),
        "n"(N)
        : "memory", "scc");
  }
}
// A uniform 64-bit value in scalar registers.
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(x >> 32)) << 32;
}

// Tiles in an order that keeps neighbours on one die: a die's run goes down kGroup
// tiles of a before it moves along b.  6 and not a power of two, with which the tiles that
// run together meet in the same memory channels: out of memory that is not in
// the caches, 16384 x 6400 x 1600 125 us (8: 148, 4: 134, 7: 123, 12: 131), 8192
// x 8192 x 1024 56 (8 and 4: 67), 16384 x 1600 x 6400 102 (8: 112, 4: 98, 7: 112).
constexpr int kGroup = 6;
__device__ __forceinline__ void tile_of(uint32_t block, uint32_t tiles_m, uint32_t tiles_n,
                                        uint32_t* tm, uint32_t* tn) {
  const uint32_t t = on_one_die(block, tiles_m * tiles_n);
  const uint32_t in_group = kGroup * tiles_n, g = t / in_group, r = t - g * in_group;
  const uint32_t high = tiles_m - g * kGroup < kGroup ? tiles_m - g * kGroup : kGroup;
  *tn = r / high;
  *tm = g * kGroup + (r - *tn * high);
}

template <typename T, typename C>
__global__ void __launch_bounds__(C::WAVES * 64) tile_kernel(ProductArgs p, uint32_t tiles_m,
                                                             uint32_t tiles_n, int per_split) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = (int)threadIdx.x & 63, row = lane & 31, half = lane >> 5;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int64_t m0 = (int64_t)tm * C::TM, n0 = (int64_t)tn * C::TN;
  const uint32_t rc = (uint32_t)row_codes(p.k), rs = (uint32_t)row_scales(p.k);
  // this split's units, an even number in front of it, so that its scales start
  // at a multiple of 16 bytes
  const int first = (int)blockIdx.y * per_split, all = (int)(rc + 127) / 128;
  const int units = all - first < per_split ? all - first : per_split;
  const bool odd = rc % 128 != 0 && first + units == all;  // the last unit is half a one
  const uint32_t last_m = (uint32_t)(p.m - m0 < C::TM ? p.m - m0 : C::TM) - 1;
  const uint32_t last_n = (uint32_t)(p.n - n0 < C::TN ? p.n - n0 : C::TN) - 1;
  const uint8_t* a_codes = p.a_codes + m0 * rc + (int64_t)first * 128;
  const uint8_t* b_codes = p.b_codes + n0 * rc + (int64_t)first * 128;
  const uint8_t* a_scales = p.a_scales + m0 * rs + (int64_t)first * 8;
  const uint8_t* b_scales = p.b_scales + n0 * rs + (int64_t)first * 8;

  // where this lane's loads come from; rows behind the last are read as the last
  uint32_t from_a[C::LA], from_b[C::LB], from_s[C::LS];
#pragma unroll
  for (int i = 0; i < C::LA; ++i) {
    const uint32_t r = (wave * C::LA + i) * 8 + (lane >> 3);
    from_a[i] = (r < last_m ? r : last_m) * rc + ((lane & 7) ^ ((i & 1) * 4 + (lane >> 4))) * 16;
  }
#pragma unroll
  for (int i = 0; i < C::LB; ++i) {
    const uint32_t r = (wave * C::LB + i) * 8 + (lane >> 3);
    from_b[i] = (r < last_n ? r : last_n) * rc + ((lane & 7) ^ ((i & 1) * 4 + (lane >> 4))) * 16;
  }
#pragma unroll
  for (int i = 0; i < C::LS; ++i) {
    const int chunk = wave * C::LS + i;
    const uint32_t r = (chunk < C::TM / 64 ? chunk : chunk - C::TM / 64) * 64 + lane;
    const uint32_t last = chunk < C::TM / 64 ? last_m : last_n;
    from_s[i] = (r < last ? r : last) * rs;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  // Load i of unit u.  Of half a unit only the lanes with pieces 0 to 3 take part,
  // behind the last unit none, and no branch is needed.
  constexpr int kLoads = C::LS + C::LA + C::LB;
  const auto load = [&](int u, int i) {
    const uint32_t to = lds0 + u % C::STAGES * C::UNIT;
    if (i < C::LS) {
      const int chunk = wave * C::LS + i;
      const bool wanted = !(u & 1) && u < units && chunk < C::SCALE_CHUNKS;
      load_to_lds((chunk < C::TM / 64 ? a_scales : b_scales) + u * 8, from_s[i],
                  lds0 + C::STAGES * C::UNIT + (u >> 1) % C::STAGES * C::SCALES + chunk * 1024,
                  uniform(wanted ? ~uint64_t(0) : 0));
      return;
    }
    const int k = i - C::LS < C::LA ? i - C::LS : i - C::LS - C::LA;
    const uint64_t low = k & 1 ? 0xf0f0f0f0f0f0f0f0u : 0x0f0f0f0f0f0f0f0fu;
    const uint64_t lanes = uniform(u + (odd ? 1 : 0) < units ? ~uint64_t(0) : u < units ? low : 0);
    if (i - C::LS < C::LA)
      load_to_lds(a_codes + (int64_t)u * 128, from_a[k], to + (wave * C::LA + k) * 1024, lanes);
    else
      load_to_lds(b_codes + (int64_t)u * 128, from_b[k],
                  to + C::TM * 128 + (wave * C::LB + k) * 1024, lanes);
  };

  struct Step {
    u32x4 a[C::MT], b[C::NT];
  };
  struct Scales {
    u32x2 a[C::MT], b[C::NT];
  };
  // Read i of step h of unit u (piece 2 * h + half of this lane's rows), and of the
  // unit's scales.
  constexpr int kReads = C::MT + C::NT;
  const auto read = [&](int u, int h, int i, Step* f) {
    const uint8_t* from =
        lds + u % C::STAGES * C::UNIT + row * 128 + (((2 * h + half) ^ (row >> 1 & 7)) * 16);
    if (i < C::MT)
      f->a[i] = *(const u32x4*)(from + (wm * C::MT + i) * 4096);
    else
      f->b[i - C::MT] = *(const u32x4*)(from + C::TM * 128 + (wn * C::NT + i - C::MT) * 4096);
  };
  const auto read_scale = [&](int u, int i, Scales* s) {
    const uint8_t* from =
        lds + C::STAGES * C::UNIT + (u >> 1) % C::STAGES * C::SCALES + row * 16 + (u & 1) * 8;
    if (i < C::MT)
      s->a[i] = *(const u32x2*)(from + (wm * C::MT + i) * 512);
    else
      s->b[i - C::MT] = *(const u32x2*)(from + C::TM * 16 + (wn * C::NT + i - C::MT) * 512);
  };
  // This lane's bytes of a row's four to places 0 and 2.
  const auto shifted = [&](const Scales& s) {
    Scales r;
#pragma unroll
    for (int i = 0; i < C::MT; ++i) r.a[i] = s.a[i] >> (uint32_t)(8 * half);
#pragma unroll
    for (int i = 0; i < C::NT; ++i) r.b[i] = s.b[i] >> (uint32_t)(8 * half);
    return r;
  };
  f32x16 acc[C::MT][C::NT];
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
  // The products of step H, `ops` other operations spread among them: a wave
  // issues in order, and a queue that is full would hold up its products.
  const auto multiply_step = [&](auto step, const Step& f, const Scales& sc, auto ops, auto op) {
    constexpr int kSlots = C::MT * C::NT, kOps = decltype(ops)::value, H = decltype(step)::value;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
#pragma unroll
      for (int k = 0; k < kOps; ++k)
        if (k * kSlots / kOps == t) op(k);
      const int i = t / C::NT, j = t % C::NT;
      acc[i][j] = multiply<H % 2 * 2>(f.b[j], f.a[i], acc[i][j], sc.b[j][H / 2], sc.a[i][H / 2]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> k0{};
  constexpr integral_constant<int, 1> k1{};
  constexpr integral_constant<int, 2> k2{};
  constexpr integral_constant<int, 3> k3{};
  constexpr integral_constant<int, kReads> kOnlyReads{};
  // loads of a unit that go with the last step of the unit before its predecessor,
  // and with its predecessor's first
  constexpr int kL1 = kLoads * 2 / 3, kL2 = kLoads - kL1;
  Step f0, f1;
  Scales s0, s1;
  // steps of unit u, each with the reads of the next step
  const auto step3 = [&](int u) {
    multiply_step(k3, f1, s0, integral_constant<int, 2 * kReads + kL1>(), [&](int k) {
      if (k < kReads)
        read_scale(u + 1, k, &s1);
      else if (k < 2 * kReads)
        read(u + 1, 0, k - kReads, &f0);
      else
        load(u + C::STAGES, k - 2 * kReads);
    });
    s0 = shifted(s1);
  };
  const auto step0 = [&](int u) {
    multiply_step(k0, f0, s0, integral_constant<int, kReads + kL2>(), [&](int k) {
      if (k < kReads)
        read(u, 1, k, &f1);
      else
        load(u + C::STAGES - 1, k - kReads + kL1);
    });
  };
  const auto step1 = [&](int u) {
    multiply_step(k1, f1, s0, kOnlyReads, [&](int k) { read(u, 2, k, &f0); });
  };
  const auto step2 = [&](int u) {
    multiply_step(k2, f0, s0, kOnlyReads, [&](int k) { read(u, 3, k, &f1); });
  };

  // loads of codes of the units that may be in flight behind the one awaited; those
  // of scales are left out, as not every unit and wave has them
  constexpr int kBehind = (C::STAGES - 2) * (C::LA + C::LB);
  const auto await = [&](int u) { arrived<kBehind>(u + C::STAGES - 2 < units); };
#pragma unroll
  for (int u = 0; u < C::STAGES - 1; ++u)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(u, i);
  await(0);
#pragma unroll
  for (int i = 0; i < kReads; ++i) read_scale(0, i, &s1);
#pragma unroll
  for (int i = 0; i < kReads; ++i) read(0, 0, i, &f0);
#pragma unroll
  for (int i = 0; i < kL1; ++i) load(C::STAGES - 1, i);
  s0 = shifted(s1);
  __builtin_amdgcn_sched_barrier(0);
  step0(0);
  step1(0);
  const int full = units - (odd ? 1 : 0);
  if (full > 0) {
    step2(0);
#pragma unroll 1
    for (int u = 0; u + 1 < full; ++u) {
      await(u + 1);
      step3(u);
      step0(u + 1);
      step1(u + 1);
      step2(u + 1);
    }
    await(full);
    step3(full - 1);  // behind the last unit what it reads is not used
    if (odd) {
      step0(full);
      step1(full);
    }
  }
  arrived<0>(true);
  // Out by strips of 32 rows through this wave's part of LDS, 16 bytes a lane.
  float* strip = (float*)lds + wave * 32 * C::STRIP;
  constexpr int kWide = sizeof(T) == 2 ? 8 : 4;  // results a lane stores
  constexpr int kLanes = C::NT * 32 / kWide;     // lanes of a row
#pragma unroll
  for (int i = 0; i < C::MT; ++i) {
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)&strip[row * C::STRIP + j * 32 + q * 8 + half * 4] =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                  acc[i][j][4 * q + 3]};
    wave_fence();
#pragma unroll
    for (int r = 0; r < 32 * kLanes / 64; ++r) {
      const int lr = r * (64 / kLanes) + lane / kLanes, lc = lane % kLanes * kWide;
      const int64_t gi = m0 + (wm * C::MT + i) * 32 + lr, gj = n0 + wn * C::NT * 32 + lc;
      float v[kWide];
#pragma unroll
      for (int k = 0; k < kWide; k += 4)
        *(f32x4*)&v[k] = *(const f32x4*)&strip[lr * C::STRIP + lc + k];
      if (gi < p.m)
        write_out<kWide>((T*)p.out + (blockIdx.y * p.m + gi) * p.out_stride + gj, 0, p.n - gj,
                         p.accumulate, v);
    }
    wave_fence();
  }
}

// Sums of the splits, in their order: of 300 x 1000 x 16384 in 8 parts 2.4 of 17 us.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(ProductArgs p, const float* parts, int splits) {
  const int64_t quads = (p.n + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / quads, col = (i - row * quads) * 4;
  if (row >= p.m) return;
  const int64_t stride = up(p.n, 4);
  f32x4 sum = *(const f32x4*)(parts + row * stride + col);
  for (int s = 1; s < splits; ++s)
    sum += *(const f32x4*)(parts + (s * p.m + row) * stride + col);
  float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  write_out<4>((T*)p.out + row * p.out_stride + col, 0, p.n - col, p.accumulate, v);
}

template <typename T, typename C>
hipError_t tiles(const ProductArgs& p, int splits, int per_split, hipStream_t stream) {
  const uint32_t tm = (uint32_t)((p.m + C::TM - 1) / C::TM);
  const uint32_t tn = (uint32_t)((p.n + C::TN - 1) / C::TN);
  tile_kernel<T, C><<<dim3(tm * tn, splits), C::WAVES * 64, 0, stream>>>(p, tm, tn, per_split);
  return hipGetLastError();
}
template <typename T>
hipError_t tiles(const ProductArgs& p, Shape shape, int splits, int per_split, hipStream_t stream) {
  if (shape == kTiles256) return tiles<T, Tile<2, 4, 4, 2, 2>>(p, splits, per_split, stream);
  if (shape == kTiles128) return tiles<T, Tile<2, 2, 2, 2, 2>>(p, splits, per_split, stream);
  return tiles<T, Tile<2, 2, 2, 2, 4>>(p, splits, per_split, stream);
}

template <typename T>
__global__ void __launch_bounds__(256) empty_kernel(ProductArgs p) {
  for (int u = 0; u < 16; ++u) {
    const int64_t i = ((int64_t)blockIdx.x * 16 + u) * 256 + threadIdx.x;
    const int64_t row = i / p.n;
    if (row < p.m) store1((T*)p.out + row * p.out_stride + (i - row * p.n), 0.0f);
  }
}

template <int MT, typename T>
hipError_t narrow(const ProductArgs& p, AType a, hipStream_t stream) {
  const dim3 grid((uint32_t)((p.n + 15) / 16));
  int64_t bytes = kWaves * 64 * MT * 4 * 4;
  if (a != kAPacked && narrow_lds(p.m, p.k) > bytes) bytes = narrow_lds(p.m, p.k);
  if (bytes > kNarrowLds) return hipErrorInvalidValue;
  if (a == kAPacked)
    narrow_kernel<MT, kAPacked, T><<<grid, kWaves * 64, bytes, stream>>>(p);
  else if (a == kABf16)
    narrow_kernel<MT, kABf16, T><<<grid, kWaves * 64, bytes, stream>>>(p);
  else
    narrow_kernel<MT, kAF32, T><<<grid, kWaves * 64, bytes, stream>>>(p);
  return hipGetLastError();
}
template <typename T>
hipError_t narrow(const ProductArgs& p, AType a, hipStream_t stream) {
  if (p.m <= 16) return narrow<1, T>(p, a, stream);
  if (p.m <= 32) return narrow<2, T>(p, a, stream);
  return narrow<4, T>(p, a, stream);
}

}  // namespace

hipError_t launch_product_narrow(const ProductArgs& p, AType a, bool out_bf16,
                                 hipStream_t stream) {
  if (p.m > kNarrowRows) return hipErrorInvalidValue;
  return out_bf16 ? narrow<bf16>(p, a, stream) : narrow<float>(p, a, stream);
}

hipError_t launch_product_tiles(const ProductArgs& p, Shape shape, int splits, int per_split,
                                float* parts, bool out_bf16, hipStream_t stream) {
  if (splits == 1)
    return out_bf16 ? tiles<bf16>(p, shape, 1, per_split, stream)
                    : tiles<float>(p, shape, 1, per_split, stream);
  ProductArgs q = p;  // the parts: splits * m rows
  q.out = parts;
  q.out_stride = up(p.n, 4);
  q.accumulate = 0;
  const hipError_t e = tiles<float>(q, shape, splits, per_split, stream);
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)((p.m * ((p.n + 3) / 4) + 255) / 256));
  if (out_bf16)
    join_kernel<bf16><<<grid, 256, 0, stream>>>(p, parts, splits);
  else
    join_kernel<float><<<grid, 256, 0, stream>>>(p, parts, splits);
  return hipGetLastError();
}

hipError_t launch_product_empty(const ProductArgs& p, bool out_bf16, hipStream_t stream) {
  if (p.accumulate) return hipSuccess;
  const dim3 grid((uint32_t)((p.m * p.n + 4095) / 4096));
  if (out_bf16)
    empty_kernel<bf16><<<grid, 256, 0, stream>>>(p);
  else
    empty_kernel<float><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace mx4
}  // namespace ob
