// Launchers of the gfx950 kernels behind the ob_mx4 C interface.
// Internal to the library; every launcher enqueues on `stream` and returns
// hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_mx4_plan.h"

namespace ob {
namespace mx4 {

struct QuantizeArgs {
  const void* x;
  float* residual;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  const uint64_t* seed_device;
  uint64_t seed;
  int64_t rows, cols, stride;
};
// One direction: rows of x, with or without a residual.
hipError_t launch_quantize_rows(const QuantizeArgs& a, bool bf16, bool stochastic,
                                hipStream_t stream);
// The transposed matrix and, where codes is not null, the rows too.
hipError_t launch_quantize_tiles(const QuantizeArgs& a, bool bf16, bool stochastic,
                                 hipStream_t stream);

struct AverageArgs {
  const uint8_t* codes[kMaxMessages];
  const uint8_t* scales[kMaxMessages];
  void* out;
  int64_t rows, cols, stride;
  int32_t n;
  float factor;
};
hipError_t launch_average(const AverageArgs& a, bool bf16, hipStream_t stream);

struct ProductArgs {
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
  const void* a;
  void* out;
  int64_t m, n, k, a_stride, out_stride;
  int32_t accumulate;
};
// a_type: how a is given.
enum AType { kAPacked, kAF32, kABf16 };
// m <= kNarrowRows; an a that is not packed takes narrow_lds(m, k) <= kNarrowLds.
hipError_t launch_product_narrow(const ProductArgs& p, AType a_type, bool out_bf16,
                                 hipStream_t stream);
// Large tiles, packed a; each split takes per_split units of 256 elements (even
// where there are several).  parts: splits * m * up(n, 4) floats where splits > 1.
hipError_t launch_product_tiles(const ProductArgs& p, Shape shape, int splits, int per_split,
                                float* parts, bool out_bf16, hipStream_t stream);
// out = 0, or left as it is with accumulate.
hipError_t launch_product_empty(const ProductArgs& p, bool out_bf16, hipStream_t stream);

}  // namespace mx4
}  // namespace ob
