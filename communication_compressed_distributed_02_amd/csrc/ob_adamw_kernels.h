// Launchers of the gfx950 kernels behind the ob_adamw C interface.
// Internal to the library; every launcher enqueues on `stream` and returns
// hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_adamw_plan.h"

namespace ob {
namespace adamw {

constexpr int kMinExpM = 8;         // smallest exponent byte of a block of m
constexpr int kMinExpV = 32;        // smallest exponent byte of a block of v
struct StepPtrs {
  const void* g[kPtrsPerStep];
  void* p[kPtrsPerStep];
};
struct NormPtrs {
  const void* g[kPtrsPerNorm];
};

// The step count and the scalars of the step that follows, on the device.
struct Control {
  int64_t steps, skipped;
  double p1, p2;             // b1^steps, b2^steps
  float gscale, rbc2;
  uint32_t skip, k0, k1;
  uint32_t root;             // tickets of small launches: leaves that are done
  uint32_t leaf[kLeaves][16];  // and tickets taken, 64 bytes apart
  float decay[kMaxGroups], rate[kMaxGroups];
};

struct ControlArgs {
  float lr[kMaxGroups], wd[kMaxGroups];
  const float* lr_device;
  const double* partials;    // null: S from sumsq, or not needed
  const double* sumsq;
  int64_t n_partials;
  float* norm;
  uint64_t seed;
  float beta1, beta2, grad_scale, max_norm;
  int32_t n_groups, skip_nonfinite;
};

struct State {
  Control* control;
  const ChunkRec* recs;
  double* partials;
  void* m;                   // fp32 or codes
  void* v;
  uint8_t* m_exp;
  uint8_t* v_exp;
  float* master;
  float beta1, beta2, eps;
  int32_t param_bf16, grad_bf16, state_bits, has_master, stochastic;
};

// The launches over few chunks.
struct SmallStep {
  State s;
  ControlArgs a;
  const void* g[kSmallTensors];
  void* p[kSmallTensors];
};
struct SmallNorm {
  const ChunkRec* recs;
  Control* control;
  double* partials;
  double* sumsq;
  float* norm;
  float grad_scale;
  const void* g[kSmallTensors];
};
static_assert(sizeof(SmallStep) <= 4096 && sizeof(StepPtrs) + sizeof(State) + 16 <= 4096 &&
                  sizeof(NormPtrs) + 48 <= 4096,
              "kernel arguments");

// A step of n <= kSmallChunks chunks: control and update in one launch.
hipError_t launch_small(const SmallStep& k, int64_t n, hipStream_t stream);
// S and the norm of n <= kSmallChunks chunks in one launch.
hipError_t launch_small_norm(const SmallNorm& k, bool grad_bf16, int64_t n, hipStream_t stream);
// Chunks [c0, c0 + n) of tensors t0, t0 + 1, ... whose pointers `ptrs` holds.
hipError_t launch_step(const State& s, const StepPtrs& ptrs, uint32_t t0, int64_t c0, int64_t n,
                       hipStream_t stream);
// The same for the norm, leaving norm_partials(n) values from partials[at].
// backwards: a step follows; the chunks go from the last to the first, through
// the caches.
hipError_t launch_norm(const State& s, const NormPtrs& ptrs, uint32_t t0, int64_t c0, int64_t n,
                       int64_t at, bool backwards, hipStream_t stream);
// Folds the partials (or reads sumsq) and advances the step.
hipError_t launch_control(const State& s, const ControlArgs& a, hipStream_t stream);
// Folds the partials into the caller's sumsq and norm.
hipError_t launch_norm_finish(const State& s, int64_t n_partials, float grad_scale, double* sumsq,
                              float* norm, hipStream_t stream);
hipError_t launch_set_steps(const State& s, int64_t steps, double p1, double p2,
                            hipStream_t stream);
hipError_t launch_fill(void* dst, uint32_t word, uint64_t words, hipStream_t stream);
hipError_t launch_master(const State& s, const StepPtrs& ptrs, uint32_t t0, int64_t c0, int64_t n,
                         hipStream_t stream);
hipError_t launch_get(const State& s, int field, int64_t offset, int64_t count, bool bf16,
                      void* dst, hipStream_t stream);
hipError_t launch_set(const State& s, int field, int64_t offset, int64_t count, const float* src,
                      hipStream_t stream);

}  // namespace adamw
}  // namespace ob
