// Host side of the ob_mx4 C interface: validation and the choice of kernels.
// See include/ob_mx4.h for the contract; the kernels are in ob_mx4_kernels.hip
// and ob_mx4_product.hip.
#include "ob_mx4.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_mx4_kernels.h"

namespace {

namespace mx = ob::mx4;

ob_status status(hipError_t e) { return e == hipSuccess ? OB_OK : OB_ERR_HIP; }

}  // namespace

extern "C" {

ob_status ob_mx4_layout(int64_t rows, int64_t cols, int64_t* row_codes, int64_t* row_scales) {
  if (row_codes == nullptr || row_scales == nullptr) return OB_ERR_ARG;
  if (!mx::shape(rows, cols)) return OB_ERR_SHAPE;
  *row_codes = mx::row_codes(cols);
  *row_scales = mx::row_scales(cols);
  return OB_OK;
}

ob_status ob_mx4_quantize(const ob_mx4_quantize_args* a, void* stream) {
  const ob_status st = mx::check_quantize(a);
  if (st != OB_OK) return st;
  if (a->rows == 0 || a->cols == 0) return OB_OK;
  mx::QuantizeArgs q{};
  q.x = a->x;
  q.residual = a->residual;
  q.codes = (uint8_t*)a->codes;
  q.scales = (uint8_t*)a->scales;
  q.codes_t = (uint8_t*)a->codes_t;
  q.scales_t = (uint8_t*)a->scales_t;
  q.seed_device = a->seed_device;
  q.seed = a->seed;
  q.rows = a->rows;
  q.cols = a->cols;
  q.stride = a->stride;
  const bool bf16 = a->dtype == OB_MX4_BF16, stochastic = a->stochastic != 0;
  return status(a->codes_t == nullptr
                    ? mx::launch_quantize_rows(q, bf16, stochastic, (hipStream_t)stream)
                    : mx::launch_quantize_tiles(q, bf16, stochastic, (hipStream_t)stream));
}

ob_status ob_mx4_average(const void* const* codes, const void* const* scales, int32_t n,
                         int64_t rows, int64_t cols, int32_t dtype, void* out, int64_t stride,
                         void* stream) {
  const ob_status st = mx::check_average(codes, scales, n, rows, cols, dtype, out, stride);
  if (st != OB_OK) return st;
  if (rows == 0 || cols == 0) return OB_OK;
  mx::AverageArgs a{};
  for (int32_t i = 0; i < n; ++i) {
    a.codes[i] = (const uint8_t*)codes[i];
    a.scales[i] = (const uint8_t*)scales[i];
  }
  a.out = out;
  a.rows = rows;
  a.cols = cols;
  a.stride = stride;
  a.n = n;
  a.factor = (float)(1.0 / n);
  return status(mx::launch_average(a, dtype == OB_MX4_BF16, (hipStream_t)stream));
}

ob_status ob_mx4_matmul_workspace(const ob_mx4_matmul_args* a, uint64_t* bytes) {
  if (bytes == nullptr) return OB_ERR_ARG;
  mx::Product plan;
  const ob_status st = mx::plan_product(a, &plan);
  if (st == OB_OK) *bytes = plan.ws_bytes;
  return st;
}

ob_status ob_mx4_matmul(const ob_mx4_matmul_args* a, void* stream) {
  mx::Product plan;
  ob_status st = mx::plan_product(a, &plan);
  if (st == OB_OK) st = mx::check_product(a, plan);
  if (st != OB_OK || plan.empty) return st;
  mx::ProductArgs p{};
  p.a_codes = (const uint8_t*)a->a_codes;
  p.a_scales = (const uint8_t*)a->a_scales;
  p.b_codes = (const uint8_t*)a->b_codes;
  p.b_scales = (const uint8_t*)a->b_scales;
  p.a = a->a;
  p.out = a->out;
  p.m = a->m;
  p.n = a->n;
  p.k = a->k;
  p.a_stride = a->a_stride;
  p.out_stride = a->out_stride;
  p.accumulate = a->accumulate;
  const bool out_bf16 = a->out_dtype == OB_MX4_BF16;
  if (a->k == 0) return status(mx::launch_product_empty(p, out_bf16, (hipStream_t)stream));
  mx::AType type = a->a_codes != nullptr ? mx::kAPacked
                         : a->a_dtype == OB_MX4_BF16 ? mx::kABf16 : mx::kAF32;
  if (plan.quantize) {
    mx::QuantizeArgs q{};
    q.x = p.a;
    q.codes = (uint8_t*)a->workspace;
    q.scales = (uint8_t*)a->workspace + plan.a_scales;
    q.rows = p.m;
    q.cols = p.k;
    q.stride = p.a_stride;
    const hipError_t e = mx::launch_quantize_rows(q, type == mx::kABf16, false, (hipStream_t)stream);
    if (e != hipSuccess) return OB_ERR_HIP;
    p.a_codes = q.codes;
    p.a_scales = q.scales;
    type = mx::kAPacked;
  }
  if (plan.shape == mx::kNarrow)
    return status(mx::launch_product_narrow(p, type, out_bf16, (hipStream_t)stream));
  return status(mx::launch_product_tiles(p, plan.shape, plan.splits, plan.per_split,
                                         (float*)((char*)a->workspace + plan.parts), out_bf16,
                                         (hipStream_t)stream));
}

}  // extern "C"
