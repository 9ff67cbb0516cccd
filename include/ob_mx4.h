/*
 * ob_mx4: matrices in microscaled 4-bit floating point on one MI355X (gfx950):
 * quantising them (with error feedback, stochastically, and in both directions
 * from one read), averaging messages and reading them back, and the product
 * of two of them on the matrix cores.
 *
 * Format.  A quantised matrix of rows x cols holds, row by row, blocks of 32
 * consecutive elements: a 4-bit code for each element (sign, 2 exponent bits,
 * 1 mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and a byte E for
 * each block; an element's value is its code's times 2^(E - 127).  E = 255
 * makes the whole block NaN.  (The elements and scales of the OCP microscaling
 * formats, E2M1 and E8M0.)
 *  - codes: element 2i of a row is the low half of byte i.  A row takes
 *    row_codes = 64 * ceil(cols / 128) bytes, rows follow each other.
 *  - scales: row_scales = 16 * ceil(cols / 512) bytes a row.
 *  - codes and scales behind the last element are zero.
 *
 * Arithmetic contract (fp32 unless stated):
 *  - quantising: c = x widened, or with a residual e its sum x + e rounded
 *    once.  a = the block's largest |c|; E - 127 = the least k >= -127 with
 *    a < 7 * 2^k to nearest, a <= 6 * 2^k stochastically: nothing is cut off,
 *    what lies between 6 and 7 rounds to 6.  y = |c| / 2^k, g = 0.5 below 2, 1
 *    below 4 and 2 from there; the code's magnitude is y / g rounded to
 *    nearest even, or floor(y / g + u / 65536), times g; it keeps c's sign.
 *    New residual: c - value, rounded once.  A block that holds a c that is
 *    not finite gets E = 255 and codes of zero, its residuals become NaN and,
 *    being added to what comes next, stay so until the caller clears them.
 *  - u: 16 random bits.  Elements 4i .. 4i+3 of the padded matrix (rows of
 *    128 * ceil(cols / 128)) take the low and the high half of word 0, then of
 *    word 1, hashed from i and the seed.  Equal seeds and inputs give equal bits:
 *    matrices whose errors have to be independent need seeds of their own.
 *  - a transposed result is the same function of the transposed matrix.
 *  - average: the values are added in the order of the messages, starting from
 *    the first, and the sum is multiplied by (float)(1.0 / n); rounded to
 *    nearest even for bfloat16.  (A value of 2^128, to which c rounds from
 *    3.5 * 2^126 on, is infinite here, not where its residual is taken.)
 *  - product: out[i][j] = sum over k of a[i][k] * b[j][k], each product exact,
 *    summed in fp32 in an order that goes by the sizes alone (equal inputs give
 *    equal bits), plus the old out with `accumulate`, rounded once to out's
 *    type.
 *
 * Ownership, streams and errors: the caller owns all device memory, which has
 * to lie on the current device; the library allocates none and keeps nothing
 * between calls.  Every call is enqueued on `stream` and returns without
 * waiting; it enqueues kernel launches only, so it may be captured, and calls
 * with memory of their own may run on several streams at once.  Argument errors
 * return before anything is enqueued; a HIP error returns OB_ERR_HIP.  Memory
 * that is written may not overlap what else the call reads or writes
 * (OB_ERR_ARG), except where stated; memory is taken from its first element to its
 * last, what lies between strided rows included.  No C++ exception crosses this
 * interface.
 */
#ifndef OB_MX4_H
#define OB_MX4_H

#include "ob_adam.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { OB_MX4_F32 = OB_GRAD_F32, OB_MX4_BF16 = OB_GRAD_BF16 };

enum { OB_MX4_MAX_MESSAGES = 64 };

/* Bytes of a row of codes and of scales.  rows and cols may be 0; OB_ERR_SHAPE
 * for a negative one, and for more than 2^35 elements in padded rows, here and
 * for every matrix of the calls below. */
ob_status ob_mx4_layout(int64_t rows, int64_t cols, int64_t* row_codes, int64_t* row_scales);

typedef struct {
  const void* x;        /* element (r, c) at x[r * stride + c], aligned to its type */
  int32_t dtype;        /* of x: OB_MX4_F32 or OB_MX4_BF16 */
  int32_t stochastic;   /* 1: stochastic rounding */
  int64_t rows, cols;
  int64_t stride;       /* elements between rows, >= 0 */
  uint64_t seed;        /* of the random bits */
  const uint64_t* seed_device; /* device: read when the call runs, in place of seed; NULL = seed */
  float* residual;      /* fp32[rows][cols], added to x and replaced; NULL = none.  Not
                           with codes_t (OB_ERR_ARG). */
  void* codes;          /* 16-byte aligned, with scales; both NULL: not wanted */
  void* scales;
  void* codes_t;        /* of the transposed matrix, cols x rows; both NULL: not wanted */
  void* scales_t;
} ob_mx4_quantize_args;

ob_status ob_mx4_quantize(const ob_mx4_quantize_args* args, void* stream);

/* Mean of n messages (1 .. OB_MX4_MAX_MESSAGES, OB_ERR_SHAPE otherwise; 1 reads a
 * matrix back) of rows x cols.  codes, scales: host arrays of n device pointers,
 * 16-byte aligned; they may repeat.  Element (r, c) goes to out[r * stride + c],
 * stride >= cols, of type dtype. */
ob_status ob_mx4_average(const void* const* codes, const void* const* scales, int32_t n,
                         int64_t rows, int64_t cols, int32_t dtype, void* out, int64_t stride,
                         void* stream);

typedef struct {
  int64_t m, n, k;      /* out is m x n, a m x k, b n x k; k <= 2^24, and the limit of elements
                           in padded rows holds for n x m too */
  const void* a_codes;  /* 16-byte aligned; NULL with a_scales: a is given in a */
  const void* a_scales;
  const void* a;        /* element (i, k) at a[i * a_stride + k]: quantised to nearest on the way */
  int32_t a_dtype;      /* of a: OB_MX4_F32 or OB_MX4_BF16 */
  int32_t out_dtype;
  int64_t a_stride;     /* >= 0 */
  const void* b_codes;
  const void* b_scales;
  void* out;            /* element (i, j) at out[i * out_stride + j] */
  int64_t out_stride;   /* >= n */
  int32_t accumulate;   /* 1: added to out */
  void* workspace;      /* 256-byte aligned device memory, ob_mx4_matmul_workspace bytes; NULL
                           where that is 0 */
  uint64_t ws_bytes;
} ob_mx4_matmul_args;

/* Bytes of workspace for these sizes and types (pointers are only tested for
 * NULL). */
ob_status ob_mx4_matmul_workspace(const ob_mx4_matmul_args* args, uint64_t* bytes);

ob_status ob_mx4_matmul(const ob_mx4_matmul_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif
