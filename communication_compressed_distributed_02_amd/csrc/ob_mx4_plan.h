// The host side's arithmetic behind the ob_mx4 C interface: validation, the
// layout of quantised matrices and the choice of a product's kernel.  No HIP
// in it, so that it is tested on its own.
#pragma once

#include <stdint.h>

#include "ob_mx4.h"

namespace ob {
namespace mx4 {

constexpr int kBlockElems = 32;   // elements of one scale
constexpr int kPadElems = 128;    // a row of codes is padded to so many elements
constexpr int kScalePad = 16;     // and a row of scales to so many bytes
constexpr int kMaxMessages = OB_MX4_MAX_MESSAGES;
// Elements in padded rows: a launch counts at most 2^32 threads, and the kernels
// that take fewest, 4096 a block of 256, stay below half of that.
constexpr int64_t kMaxElems = int64_t(1) << 35;
constexpr int64_t kMaxK = int64_t(1) << 24;      // 255 rows of k / 2 bytes stay below 2^32

constexpr int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
constexpr int64_t padded(int64_t cols) { return up(cols, kPadElems); }
constexpr int64_t row_codes(int64_t cols) { return padded(cols) / 2; }
constexpr int64_t row_scales(int64_t cols) { return up(cols, kBlockElems * kScalePad) / kBlockElems; }
inline uint64_t size_of(int32_t dtype) { return dtype == OB_MX4_BF16 ? 2 : 4; }

inline bool aligned(const void* p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
inline bool dtype(int32_t v) { return v == OB_MX4_F32 || v == OB_MX4_BF16; }
inline bool flag(int32_t v) { return v == 0 || v == 1; }

// Rows and columns that a quantised matrix may have, in that order.
inline bool shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxElems || cols > kMaxElems) return false;
  return rows == 0 || padded(cols) <= kMaxElems / rows;
}

// A stride that keeps every offset of rows x cols elements below 2^60.
inline bool stride(int64_t rows, int64_t least, int64_t s) {
  return s >= least && (rows <= 1 || s <= (int64_t(1) << 58) / rows);
}

// Memory that a call reads or writes; empty where it is null.
struct Range {
  uintptr_t begin, end;
  bool written;
};
inline Range range(const void* p, uint64_t bytes, bool written) {
  return {(uintptr_t)p, (uintptr_t)p + (p != nullptr ? bytes : 0), written};
}
inline uint64_t strided_bytes(int64_t rows, int64_t cols, int64_t s, int32_t type) {
  return rows == 0 || cols == 0 ? 0 : ((uint64_t)(rows - 1) * s + cols) * size_of(type);
}
template <int N>
inline bool disjoint(const Range (&r)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if ((r[i].written || r[j].written) && r[i].begin < r[j].end && r[j].begin < r[i].end &&
          r[i].begin < r[i].end && r[j].begin < r[j].end)
        return false;
  return true;
}

inline ob_status check_quantize(const ob_mx4_quantize_args* a) {
  if (a == nullptr || !dtype(a->dtype) || !flag(a->stochastic)) return OB_ERR_ARG;
  if (!shape(a->rows, a->cols) || (a->codes_t != nullptr && !shape(a->cols, a->rows)))
    return OB_ERR_SHAPE;
  if (!stride(a->rows, 0, a->stride)) return OB_ERR_ARG;
  if ((a->codes == nullptr) != (a->scales == nullptr) ||
      (a->codes_t == nullptr) != (a->scales_t == nullptr))
    return OB_ERR_ARG;
  if (a->rows == 0 || a->cols == 0) return OB_OK;
  if (a->codes == nullptr && a->codes_t == nullptr) return OB_ERR_ARG;
  if (a->x == nullptr || !aligned(a->x, size_of(a->dtype))) return OB_ERR_ARG;
  if (a->residual != nullptr && (a->codes_t != nullptr || !aligned(a->residual, 4)))
    return OB_ERR_ARG;
  if (!aligned(a->seed_device, 8) || !aligned(a->codes, 16) || !aligned(a->scales, 16) ||
      !aligned(a->codes_t, 16) || !aligned(a->scales_t, 16))
    return OB_ERR_ARG;
  const Range r[] = {
      range(a->x, strided_bytes(a->rows, a->cols, a->stride, a->dtype), false),
      range(a->seed_device, 8, false),
      range(a->residual, (uint64_t)a->rows * a->cols * 4, true),
      range(a->codes, (uint64_t)a->rows * row_codes(a->cols), true),
      range(a->scales, (uint64_t)a->rows * row_scales(a->cols), true),
      range(a->codes_t, (uint64_t)a->cols * row_codes(a->rows), true),
      range(a->scales_t, (uint64_t)a->cols * row_scales(a->rows), true)};
  return disjoint(r) ? OB_OK : OB_ERR_ARG;
}

inline ob_status check_average(const void* const* codes, const void* const* scales, int32_t n,
                               int64_t rows, int64_t cols, int32_t type, const void* out,
                               int64_t s) {
  if (codes == nullptr || scales == nullptr || !dtype(type)) return OB_ERR_ARG;
  if (n < 1 || n > kMaxMessages || !shape(rows, cols)) return OB_ERR_SHAPE;
  if (!stride(rows, cols, s)) return OB_ERR_ARG;
  if (rows == 0 || cols == 0) return OB_OK;
  if (out == nullptr || !aligned(out, size_of(type))) return OB_ERR_ARG;
  const Range o = range(out, strided_bytes(rows, cols, s, type), true);
  for (int32_t i = 0; i < n; ++i) {
    if (codes[i] == nullptr || scales[i] == nullptr || !aligned(codes[i], 16) ||
        !aligned(scales[i], 16))
      return OB_ERR_ARG;
    const Range r[] = {o, range(codes[i], (uint64_t)rows * row_codes(cols), false),
                       range(scales[i], (uint64_t)rows * row_scales(cols), false)};
    if (!disjoint(r)) return OB_ERR_ARG;
  }
  return OB_OK;
}

// How a product is computed, from its sizes and types alone.
enum Shape { kNarrow, kTiles128, kTiles256, kTiles128Deep };  // Deep: four units in LDS
struct Product {
  bool empty;              // nothing to compute
  bool quantize;           // a is quantised into the workspace first
  Shape shape;
  int splits, per_split;   // of the sum, in units of 256 elements
  uint64_t a_scales, parts, ws_bytes;  // places in the workspace (a's codes at 0)
};

constexpr int kNarrowRows = 64;        // rows of a that the narrow kernel takes at most
constexpr int64_t kNarrowCols = int64_t(1) << 26;  // 16 a block of 512 threads
constexpr int kNarrowLds = 32 * 1024;  // bytes of LDS that it uses at most
// Elements of an a that it quantises itself, by every block: 16 rows of 1024
// 4.4 us, 2.0 and 3.1 in two launches; 16 of 1600 8.2, and 2.0 and 4.4.
constexpr int64_t kNarrowElems = 24 * 1024;
inline int64_t narrow_lds(int64_t m, int64_t k) { return m * (padded(k) / 128 * 72 + 24); }

// Units from which a block alone on its CU holds four of them in LDS and not two,
// so that the loads of three are on their way: 1600 x 1600 x 16384, 64 units, 40.3
// us, with two 50.9; 16 units of 4096 x 1024 15.2 and 17.1; 12 of 1200 x 2000 12.2
// and 11.9, 8 of 2048 x 2048 9.7 and 9.5.
constexpr int kDeepUnits = 16;
// Tiles of 128 x 128 or 256 x 256, and into how many parts the sum goes: the
// shortest by an estimate in ns, a round of tiles at a time.  The figures are
// those of 8192 x 8192 x 16384 (both shapes) and of short sums; the choices
// against all others, in us: 4096 x 1024 x 4096 15.2, next 25.3; 8192 x 8192 x
// 16384 484, 631; 300 x 1000 x 16384 in 8 parts 17, 19 in 4, 38 in one.
inline double choose_tiles(int64_t m, int64_t n, int64_t k, Product* p) {
  struct Cost {
    Shape shape;
    int64_t size, slots;     // edge of a tile, tiles that run at once
    double unit, fixed;      // of a round: a unit's, and what comes before and after
  };
  static constexpr Cost kCosts[] = {{kTiles128, 128, 512, 1220.0, 3000.0},
                                    {kTiles256, 256, 256, 1810.0, 7000.0}};
  const int64_t units = (row_codes(k) + 127) / 128;
  double best = 0.0;
  for (const Cost& c : kCosts) {
    const int64_t tiles = up(m, c.size) / c.size * (up(n, c.size) / c.size);
    for (int splits = 1; splits <= 16; splits *= 2) {
      const int64_t per = up((units + splits - 1) / splits, splits > 1 ? 2 : 1);
      const int64_t real = (units + per - 1) / per;
      if (splits > 1 && (real < splits || tiles * splits > c.slots)) break;
      const double rounds = (double)((tiles * real + c.slots - 1) / c.slots);
      // a block that has its CU to itself is faster, and over a long sum faster
      // still with more units on their way
      const bool alone = c.slots == 512 && tiles * real <= 256, deep = alone && per >= kDeepUnits;
      double t = deep ? (double)per * 520.0 + 5000.0
                      : rounds * ((double)per * c.unit * (alone ? 0.55 : 1.0) + c.fixed);
      if (real > 1) t += 3000.0 + (double)(m * n) * (real * 8.0 + 2.0) / 4000.0;
      if (best == 0.0 || t < best) {
        best = t;
        p->shape = deep ? kTiles128Deep : c.shape;
        p->splits = (int)real;
        p->per_split = (int)per;
      }
    }
  }
  return best;
}
// What the narrow kernel takes: b's bytes at 4 TB/s, and more the more rows of a.
// One row of 16384 x 16384 36 us (tiles 26), 16 rows 58 (27); of 4096 x 4096 4.4
// (8.3) and 5.8 (9.5), 64 rows 11.1 (11.0).
inline double narrow_time(int64_t m, int64_t n, int64_t k) {
  return 2500.0 + (double)n * row_codes(k) * (0.246e-3 + 0.0124e-3 * m);
}

inline ob_status plan_product(const ob_mx4_matmul_args* a, Product* out) {
  if (a == nullptr || !dtype(a->out_dtype) || !flag(a->accumulate)) return OB_ERR_ARG;
  const bool packed = a->a_codes != nullptr || a->a_scales != nullptr;
  if (!packed && !dtype(a->a_dtype)) return OB_ERR_ARG;
  const int64_t m = a->m, n = a->n, k = a->k;
  if (k < 0 || k > kMaxK || !shape(m, k) || !shape(n, k) || !shape(m, n) || !shape(n, m))
    return OB_ERR_SHAPE;
  *out = Product{};
  out->empty = m == 0 || n == 0;
  if (out->empty || k == 0) return OB_OK;
  const double time = choose_tiles(m, n, k, out);
  if (m <= kNarrowRows && n <= kNarrowCols && narrow_time(m, n, k) <= time) {
    out->shape = kNarrow;
    out->splits = out->per_split = 0;
  }
  out->quantize = !packed && (out->shape != kNarrow || m * padded(k) > kNarrowElems);
  if (out->quantize) {
    out->a_scales = up(m * row_codes(k), 256);
    out->parts = out->a_scales + up(m * row_scales(k), 256);
  }
  out->ws_bytes = out->parts;
  if (out->splits > 1) out->ws_bytes += (uint64_t)out->splits * m * up(n, 4) * 4;
  return OB_OK;
}

inline ob_status check_product(const ob_mx4_matmul_args* a, const Product& p) {
  if (!stride(a->m, a->n, a->out_stride)) return OB_ERR_ARG;
  const bool packed = a->a_codes != nullptr || a->a_scales != nullptr;
  if (!packed && !stride(a->m, 0, a->a_stride)) return OB_ERR_ARG;
  if (p.empty) return OB_OK;
  if (a->out == nullptr || !aligned(a->out, size_of(a->out_dtype))) return OB_ERR_ARG;
  if (a->k > 0) {
    if (packed ? a->a != nullptr || a->a_codes == nullptr || a->a_scales == nullptr ||
                     !aligned(a->a_codes, 16) || !aligned(a->a_scales, 16)
               : a->a == nullptr || !aligned(a->a, size_of(a->a_dtype)))
      return OB_ERR_ARG;
    if (a->b_codes == nullptr || a->b_scales == nullptr || !aligned(a->b_codes, 16) ||
        !aligned(a->b_scales, 16))
      return OB_ERR_ARG;
  }
  if (p.ws_bytes > 0 &&
      (a->workspace == nullptr || !aligned(a->workspace, 256) || a->ws_bytes < p.ws_bytes))
    return OB_ERR_WORKSPACE;
  const Range r[] = {
      range(a->a_codes, (uint64_t)a->m * row_codes(a->k), false),
      range(a->a_scales, (uint64_t)a->m * row_scales(a->k), false),
      range(a->a, strided_bytes(a->m, a->k, a->a_stride, a->a_dtype), false),
      range(a->b_codes, (uint64_t)a->n * row_codes(a->k), false),
      range(a->b_scales, (uint64_t)a->n * row_scales(a->k), false),
      range(a->out, strided_bytes(a->m, a->n, a->out_stride, a->out_dtype), true),
      range(a->workspace, p.ws_bytes, true)};
  return disjoint(r) ? OB_OK : OB_ERR_ARG;
}

}  // namespace mx4
}  // namespace ob
