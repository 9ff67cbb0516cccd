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

#include "ob_mx4_device.h"
#include "ob_mx4_kernels.h"

namespace ob {
namespace mx4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;       // the instruction's number for these elements
constexpr int kUnit = 128;    // elements of the sum that the padding makes whole

// acc += 32 x 32 products over 64 elements; the scales are byte BYTE of sa, sb.
template <int BYTE>
__device__ __forceinline__ f32x16 multiply(u32x4 b, u32x4 a, f32x16 acc, uint32_t sb, uint32_t sa) {
  const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, acc, kFp4, kFp4, BYTE, (int)sb,
                                                         BYTE, (int)sa);
}

template <AType A>
struct Raw {
  typedef float type;
};
template <>
struct Raw<kABf16> {
  typedef bf16 type;
};

// Elements k to k + 31 of a row of a (zeros behind its end), quantised to
// nearest on one lane: the codes, and the scale byte returned.
template <typename T>
__device__ __forceinline__ uint32_t quantize_block(const ProductArgs& p, int64_t row, int64_t k,
                                                   u32x4* codes) {
  const T* x = (const T*)p.a + row * p.a_stride + k;
  float c[kBlockElems];
#pragma unroll
  for (int i = 0; i < kBlockElems; i += 8) {
    if (k + i + 8 <= p.k)
      load8(x + i, c + i);
    else
      load8_some(x + i, (int)(p.k > k + i ? p.k - k - i : 0), c + i);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kBlockElems; ++i) {
    const uint32_t w = magnitude(c[i]);
    top = w > top ? w : top;
  }
  const uint32_t byte = scale_byte<false>(top);
  const float inv = inverse_scale(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) (*codes)[i] = encode8(c + 8 * i, inv);
  return byte;
}

// Four results along a row of out, of which `n` exist.
template <typename T>
__device__ __forceinline__ void store4(T* p, const float* v, int64_t n) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) store1(p + i, v[i]);
}

// Tiles of 32 x 32, one a block; its waves take every kWaves-th unit of the sum
// and add up through LDS in their order.
constexpr int kWaves = 4;
template <AType A, typename T>
__global__ void __launch_bounds__(kWaves * 64) narrow_kernel(ProductArgs p) {
  __shared__ float part[kWaves][64][17];  // 17: lanes do not meet in a bank
  const int64_t tiles_n = (p.n + 31) / 32;
  const int64_t tm = (int64_t)blockIdx.x / tiles_n, tn = (int64_t)blockIdx.x - tm * tiles_n;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = (int)threadIdx.x & 63, row = lane & 31, half = lane >> 5;
  const int64_t rc = row_codes(p.k), rs = row_scales(p.k);
  // rows behind the last are read as the last, and their results dropped
  const int64_t am = tm * 32 + row < p.m ? tm * 32 + row : p.m - 1;
  const int64_t bn = tn * 32 + row < p.n ? tn * 32 + row : p.n - 1;
  const uint8_t* b_codes = p.b_codes + bn * rc + half * 16;
  const uint8_t* b_scales = p.b_scales + bn * rs;
  f32x16 acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  const int64_t units = rc / 64;
#pragma unroll 1
  for (int64_t u = wave; u < units; u += kWaves) {
    const u32x4 b0 = *(const u32x4*)(b_codes + u * 64);
    const u32x4 b1 = *(const u32x4*)(b_codes + u * 64 + 32);
    const uint32_t sb = *(const uint32_t*)(b_scales + u * 4) >> (8 * half);
    u32x4 a0, a1;
    uint32_t sa;
    if constexpr (A == kAPacked) {
      a0 = *(const u32x4*)(p.a_codes + am * rc + u * 64 + half * 16);
      a1 = *(const u32x4*)(p.a_codes + am * rc + u * 64 + half * 16 + 32);
      sa = *(const uint32_t*)(p.a_scales + am * rs + u * 4) >> (8 * half);
    } else {
      const int64_t k = u * kUnit + half * kBlockElems;
      const uint32_t s0 = quantize_block<typename Raw<A>::type>(p, am, k, &a0);
      const uint32_t s1 = quantize_block<typename Raw<A>::type>(p, am, k + 64, &a1);
      sa = s0 | s1 << 16;
    }
    acc = multiply<0>(b0, a0, acc, sb, sa);
    acc = multiply<2>(b1, a1, acc, sb, sa);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) part[wave][lane][i] = acc[i];
  __syncthreads();
  // this wave's quarter of the results: registers 4 * wave to + 3
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = part[0][lane][4 * wave + i];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v[i] += part[w][lane][4 * wave + i];
  }
  const int64_t i = tm * 32 + row, j = tn * 32 + 8 * wave + 4 * half;
  if (i >= p.m || j >= p.n) return;
  T* out = (T*)p.out + i * p.out_stride + j;
  if (p.accumulate) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (j + k < p.n) v[k] += widen(out[k]);
  }
  store4(out, v, p.n - j);
}

template <typename T>
__global__ void __launch_bounds__(256) empty_kernel(ProductArgs p) {
  for (int u = 0; u < 4; ++u) {
    const int64_t i = ((int64_t)blockIdx.x * 4 + u) * 256 + threadIdx.x;
    const int64_t row = i / p.n;
    if (row < p.m) store1((T*)p.out + row * p.out_stride + (i - row * p.n), 0.0f);
  }
}

template <typename T>
hipError_t narrow(const ProductArgs& p, AType a, hipStream_t stream) {
  const dim3 grid((uint32_t)((p.m + 31) / 32 * ((p.n + 31) / 32)));
  if (a == kAPacked)
    narrow_kernel<kAPacked, T><<<grid, kWaves * 64, 0, stream>>>(p);
  else if (a == kABf16)
    narrow_kernel<kABf16, T><<<grid, kWaves * 64, 0, stream>>>(p);
  else
    narrow_kernel<kAF32, T><<<grid, kWaves * 64, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_narrow(const ProductArgs& p, AType a, bool out_bf16,
                                 hipStream_t stream) {
  return out_bf16 ? narrow<bf16>(p, a, stream) : narrow<float>(p, a, stream);
}

hipError_t launch_product_empty(const ProductArgs& p, bool out_bf16, hipStream_t stream) {
  if (p.accumulate) return hipSuccess;
  const dim3 grid((uint32_t)((p.m * p.n + 1023) / 1024));
  if (out_bf16)
    empty_kernel<bf16><<<grid, 256, 0, stream>>>(p);
  else
    empty_kernel<float><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace mx4
}  // namespace ob
