// Test access to the host arithmetic behind ob_mx4 (ob_mx4_plan.h), which has no
// HIP in it: built with g++ and the sanitizers, called through ctypes.
#include "ob_mx4_plan.h"

using namespace ob::mx4;

extern "C" {

int shim_plan(const ob_mx4_matmul_args* a, int64_t* out) {
  Product p;
  const ob_status st = plan_product(a, &p);
  if (st != OB_OK) return st;
  const int64_t all[] = {p.empty, p.quantize, p.shape, p.splits, p.per_split,
                         (int64_t)p.a_scales, (int64_t)p.parts, (int64_t)p.ws_bytes};
  for (int i = 0; i < 8; ++i) out[i] = all[i];
  return OB_OK;
}

int64_t shim_narrow_lds(int64_t m, int64_t k) { return narrow_lds(m, k); }
int shim_quantize(const ob_mx4_quantize_args* a) { return check_quantize(a); }
int shim_product(const ob_mx4_matmul_args* a) {
  Product p;
  const ob_status st = plan_product(a, &p);
  return st != OB_OK ? st : check_product(a, p);
}

}  // extern "C"
