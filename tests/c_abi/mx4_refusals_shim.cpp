// Test access to the argument checks of ob_mx4 (ob_mx4_plan.h), which have no HIP
// in them: built with g++ and the sanitizers, called through ctypes.
#include "ob_mx4_plan.h"

using namespace ob::mx4;

extern "C" {

int shim_layout(int64_t rows, int64_t cols, int64_t* out) {
  if (!shape(rows, cols)) return OB_ERR_SHAPE;
  out[0] = row_codes(cols);
  out[1] = row_scales(cols);
  return OB_OK;
}
int shim_quantize(const ob_mx4_quantize_args* a) { return check_quantize(a); }
int shim_average(const void* const* codes, const void* const* scales, int32_t n, int64_t rows,
                 int64_t cols, int32_t type, const void* out, int64_t stride) {
  return check_average(codes, scales, n, rows, cols, type, out, stride);
}
int shim_product(const ob_mx4_matmul_args* a, int64_t* ws_bytes) {
  Product p;
  const ob_status st = plan_product(a, &p);
  if (st != OB_OK) return st;
  *ws_bytes = (int64_t)p.ws_bytes;
  return check_product(a, p);
}

}  // extern "C"
