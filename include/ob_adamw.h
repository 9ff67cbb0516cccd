/*
 * ob_adamw: AdamW's step over many tensors at once, with its states in 32
 * bits or in 8, and the global gradient norm that clips it, on one MI355X
 * (gfx950).
 *
 * A plan (the handle) is made for a list of tensors; a step reads every
 * tensor's gradient and updates its parameters where they lie, in a few
 * launches however many tensors there are.
 *
 * Arithmetic contract (fp32 unless stated, one rounding per operation, in
 * this order; b = beta, ob = 1 - b in fp32):
 *  - norm: S = fp64 sum of g*g over all tensors with a gradient, in an order
 *    fixed by their sizes; norm = sqrt(S) * grad_scale in fp64.
 *  - clipping: coef = 1 if norm <= max_norm, else max_norm / norm (fp64; a
 *    NaN norm gives a NaN coef, an infinite one 0); gs = (float)(grad_scale *
 *    coef).  Without clipping gs = grad_scale.
 *  - step t (1-based, counted on the device): g' = g*gs (g widened to fp32);
 *    m = (b1*m) + (ob1*g'); v = (b2*v) + (ob2*(g'*g'));
 *    x = (x*decay) - (rate*(m / ((sqrtf(v)*rbc2) + eps))), with, in fp64 and
 *    rounded once, decay = 1 - lr*weight_decay, rate = lr / (1 - b1^t),
 *    rbc2 = 1 / sqrt(1 - b2^t), b^t formed by t fp64 multiplications.
 *    m and v here are the new values before any rounding to 8 bits.
 *    (Adam with decoupled weight decay; bias correction, eps outside the
 *    root.)
 *  - bfloat16 parameters: with `master`, x is an fp32 copy in the workspace
 *    and the parameter is it rounded to nearest even; without, x is the
 *    widened parameter, and the result is rounded to nearest even or, with
 *    `stochastic`, by adding 16 random bits below the kept ones and cutting.
 *  - 8-bit states are kept in blocks of 256 consecutive elements of one
 *    tensor.  First moment: OCP e4m3 codes of m * 2^(7 - E), rounded to
 *    nearest even, E = the exponent of the block's largest finite |m| (at
 *    least -119), stored as the byte E + 127.  Second moment: q = (bits(v) +
 *    16*r + 8) >> 20 with 16 random bits r, i.e. v rounded stochastically to
 *    3 mantissa bits; e = the block's largest q >> 3 (at least 32), stored as
 *    a byte; the code is q - ((e - 31)*8 + 1) clamped to 1..254, and 0 for v
 *    = 0.  A v below the block's 2^-31 is thus held as that floor, never as
 *    zero under the root.  A state element that is not finite is held as NaN
 *    (m: 0x7f or 0xff, v: 255) and leaves its block's exponents alone.
 *    Rounding v to nearest would freeze it: a step moves v by about 1 - b2 of
 *    itself, the codes are 6 to 12 % apart.
 *    Beside 8-bit states the square root and the quotient are formed from
 *    one-ulp approximations, so that m / (...) is within 7 * 2^-24 of its exact
 *    value, relatively; everything else rounds as stated.  They are rounded
 *    correctly there too for eps < 2^-30, for beta2 < 2^-10, for 0 < beta1 <
 *    2^-8, among a tensor's last 1023 elements where they do not fill a wave's
 *    share, and in blocks of 256 that held a v of 0 or hold a moment that is
 *    not finite or near the ends of fp32's range.
 *  - random bits: 32-bit words hashed from k/4 (k = the element's index in
 *    the state), the seed and the step count; elements 4i .. 4i+3 take the
 *    low and the high half of word 0, then of word 1, for v, and of words 2
 *    and 3 for a parameter.  The same seed, steps and inputs give the same
 *    bits.
 *
 * State layout: every tensor starts at a multiple of 1024 elements
 * (ob_adamw_layout); the elements between tensors are zero.
 *
 * Ownership, streams and errors as in ob_adam.h: the caller owns all device
 * memory, the library allocates none; every call is enqueued on the stream
 * given to ob_adamw_init (or ob_adamw_set_stream) and returns without waiting,
 * except where stated;
 * argument errors return before anything is enqueued and leave the state
 * untouched; a HIP error returns OB_ERR_HIP and poisons the handle.  The
 * handle's device (the one the workspace lies on) has to be the current one,
 * OB_ERR_ARG otherwise.  A handle is not thread-safe.  Calls of one handle
 * that are replayed from graphs share its workspace: order them.  No C++
 * exception crosses this interface.
 */
#ifndef OB_ADAMW_H
#define OB_ADAMW_H

#include "ob_adam.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ob_adamw_handle* ob_adamw_t;

/* Element types. */
enum { OB_ADAMW_F32 = OB_GRAD_F32, OB_ADAMW_BF16 = OB_GRAD_BF16 };

enum { OB_ADAMW_MAX_GROUPS = 32 };

typedef struct {
  int32_t n_tensors;   /* 1 .. 2^20 */
  int32_t n_groups;    /* hyperparameter groups, 1 .. OB_ADAMW_MAX_GROUPS (OB_ERR_ARG) */
  int32_t param_dtype; /* OB_ADAMW_F32 or OB_ADAMW_BF16 */
  int32_t grad_dtype;  /* OB_ADAMW_F32 or OB_ADAMW_BF16 */
  int32_t state_bits;  /* 32, 8, or 0: a plan for gradient norms only */
  int32_t master;      /* 1: fp32 copies of bfloat16 parameters in the workspace */
  int32_t stochastic;  /* 1: bfloat16 parameters without copies are rounded stochastically */
  float beta1, beta2, eps; /* 0 <= beta < 1, eps > 0 */
  uint64_t seed;       /* of the random bits */
} ob_adamw_config;

/* Where the state of each tensor lies and what it takes: offsets[i] = index
 * of tensor i's first element in every state array (a multiple of 1024;
 * offsets may be NULL), *length = elements of a state array, *bytes = bytes
 * of device workspace (256-byte aligned start).  numel: host array of the
 * n_tensors element counts, 0 allowed.  OB_ERR_SHAPE for a negative count or
 * a length past 2^40. */
ob_status ob_adamw_layout(const ob_adamw_config* cfg, const int64_t* numel, int64_t* offsets,
                          int64_t* length, uint64_t* bytes);

/* A plan over `workspace` with zero moments and step count 0.  group: host
 * array, tensor i's hyperparameter group (NULL: all 0).  params: host array
 * of device pointers as for ob_adamw_step, read for the master copies; NULL =
 * zeros, and ignored without `master`.  Waits for the stream: when it returns,
 * the plan's tables are uploaded, the parameters have been read and the whole
 * workspace is written, so either may be written on any stream; OB_ERR_PHASE
 * on a capturing stream. */
ob_status ob_adamw_init(const ob_adamw_config* cfg, const int64_t* numel, const int32_t* group,
                        void* workspace, uint64_t ws_bytes, const void* const* params,
                        void* stream, ob_adamw_t* out);

/* Like ob_adamw_init, but adopts the state of a copy of a workspace of the
 * same configuration and sizes: the workspace bytes are the whole state, the
 * step count among them, and later steps are bit-identical to those of an
 * uninterrupted run.  (The plan's own tables are written again, and the stream
 * is waited for.) */
ob_status ob_adamw_attach(const ob_adamw_config* cfg, const int64_t* numel, const int32_t* group,
                          void* workspace, uint64_t ws_bytes, void* stream, ob_adamw_t* out);

/* S and the norm of the gradients.  grads: host array of n_tensors device
 * pointers (NULL: no gradient, counts as zeros), contiguous, aligned to their
 * element size.  sumsq (fp64) and norm (fp32): device memory, one element,
 * either may be NULL.  The order of the sum goes by the tensors' sizes and by
 * which of them have a gradient alone, so equal inputs give equal bits. */
ob_status ob_adamw_grad_norm(ob_adamw_t h, const void* const* grads, float grad_scale,
                             double* sumsq, float* norm);

typedef struct {
  const float* lr;           /* host, [n_groups] */
  const float* weight_decay; /* host, [n_groups]; NULL = 0 */
  const float* lr_device;    /* device fp32[n_groups], read when the step runs, in place of
                                lr (for captured steps under a schedule); NULL = lr */
  float grad_scale;          /* > 0: 1, 1/loss scale, 1/workers */
  float max_norm;            /* > 0: clip by the global norm; 0: no clipping */
  int32_t skip_nonfinite;    /* 1: a step whose S is not finite changes nothing and is
                                counted as skipped */
  const double* sumsq;       /* device: S to clip and skip by (a sum over ranks, say);
                                NULL: S of these gradients, computed if needed */
  float* norm;               /* device: receives the norm; NULL = not wanted */
} ob_adamw_step_args;

/* One step.  params, grads: host arrays of n_tensors device pointers,
 * contiguous, aligned to their element size.  A tensor without a gradient
 * (NULL) is left as it is, state included, and its parameter pointer may be
 * NULL.  Parameters may overlap neither each other nor a gradient nor
 * the workspace (OB_ERR_ARG); gradients may overlap each other.  The step
 * count is kept on the device and the call enqueues kernel launches only, so
 * a captured step may be replayed: each replay is one more step on the
 * captured addresses.  OB_ERR_PHASE for a plan with state_bits 0. */
ob_status ob_adamw_step(ob_adamw_t h, const void* const* params, const void* const* grads,
                        const ob_adamw_step_args* args);

/* Fields of the state. */
enum {
  OB_ADAMW_M = 0,      /* first moment */
  OB_ADAMW_V = 1,      /* second moment */
  OB_ADAMW_MASTER = 2, /* fp32 master copies */
  OB_ADAMW_M_EXP = 3,  /* 8-bit states: exponent bytes, one per block of 256 */
  OB_ADAMW_V_EXP = 4
};

/* Elements [offset, offset + count) of OB_ADAMW_M, OB_ADAMW_V or
 * OB_ADAMW_MASTER, in the state layout, as `dtype` into device memory aligned
 * to its elements (8-bit states are decoded, which is exact in either type down to
 * 2^-126; 32-bit ones are rounded to nearest even for bfloat16). */
ob_status ob_adamw_get_state(ob_adamw_t h, int32_t field, int64_t offset, int64_t count,
                             int32_t dtype, void* dst);

/* The same elements from device fp32 memory.  8-bit states are encoded, both
 * rounded to nearest, so offset and count are multiples of 256.  Negative
 * second moments become 0.  Elements between tensors have to stay zero. */
ob_status ob_adamw_set_state(ob_adamw_t h, int32_t field, int64_t offset, int64_t count,
                             const float* src);

/* Device address and bytes of a field as it is stored: fp32, or for 8-bit
 * states the codes.  OB_ERR_ARG for a field the plan does not hold. */
ob_status ob_adamw_state(ob_adamw_t h, int32_t field, void** device, uint64_t* bytes);

/* Set the count of steps taken (0 .. 2^31 - 1), as when moments are brought
 * from elsewhere; skipped steps become 0.  Enqueued. */
ob_status ob_adamw_set_steps(ob_adamw_t h, int64_t steps);

/* Steps taken and steps skipped, replays among them.  Waits for the stream. */
ob_status ob_adamw_get_steps(ob_adamw_t h, int64_t* steps, int64_t* skipped);

/* As ob_adam_check_guards: -1, or the first guard found changed (in workspace
 * order: control block, chunk records, partial sums, m, v, m exponents, v
 * exponents, master copies).  Waits for the stream. */
ob_status ob_adamw_check_guards(ob_adamw_t h, int32_t* first_bad);

/* Enqueue later calls on `stream` (of the plan's device), as to record one on a
 * stream under capture.  The caller orders them after the earlier ones. */
ob_status ob_adamw_set_stream(ob_adamw_t h, void* stream);

/* Release the handle (the caller frees the workspace afterwards). */
ob_status ob_adamw_destroy(ob_adamw_t h);

#ifdef __cplusplus
}
#endif
#endif
