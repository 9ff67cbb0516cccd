// Host side of the ob_adamw C interface: validation, workspace layout, the
// list of chunks and the launch sequence of a step.  See include/ob_adamw.h
// for the contract; the kernels are in ob_adamw_kernels.hip.
#include "ob_adamw.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "ob_adamw_kernels.h"
#include "ob_kernels.h"

namespace {

namespace aw = ob::adamw;

constexpr int64_t kMaxSteps = (int64_t(1) << 31) - 1;
// Chunks of one launch of the step, 2 to 4 GB of traffic.  32-bit states,
// 2^14, 2^15 and 2^17 chunks: 1458, 1487 and 1507 us on 334M parameters, 7.62,
// 7.70 and 7.91 ms on 1.56B; 2^13 as 2^14.  8-bit ones, 2^14, 2^15, 2^16 and
// 2^18: 1072, 1074, 1078 and 1079 us, 3.11, 3.05, 3.01 and 3.02 ms.
constexpr int64_t kChunks32 = int64_t(1) << 14, kChunks8 = int64_t(1) << 16;
static_assert(aw::kGuardGap == ob::kGuardBytes, "the guards are those of ob_adam workspaces");

}  // namespace

struct ob_adamw_handle {
  aw::Plan plan;
  aw::State st{};
  aw::Places at{};
  char* base = nullptr;
  int device = -1;
  hipStream_t stream = nullptr;
  bool poisoned = false;
};

namespace {

ob_status fail(ob_adamw_t h, hipError_t e) {
  if (e == hipSuccess) return OB_OK;
  h->poisoned = true;
  return OB_ERR_HIP;
}

// The handle may be used, and its device is the current one.
ob_status usable(ob_adamw_t h) {
  if (h == nullptr) return OB_ERR_ARG;
  if (h->poisoned) return OB_ERR_HIP;
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess) return fail(h, hipErrorNoDevice);
  return cur == h->device ? OB_OK : OB_ERR_ARG;
}

// hipSuccess where the stream may be waited for; *capturing where it is
// being captured.
hipError_t capturing(hipStream_t stream, bool* out) {
  hipStreamCaptureStatus s = hipStreamCaptureStatusNone;
  const hipError_t e = hipStreamIsCapturing(stream, &s);
  if (e != hipSuccess) (void)hipGetLastError();
  *out = s != hipStreamCaptureStatusNone;
  return e;
}

hipError_t upload(ob_adamw_handle* h, const std::vector<aw::ChunkRec>& recs) {
  if (recs.empty()) return hipSuccess;
  return hipMemcpyAsync(h->base + h->at.recs, recs.data(), recs.size() * sizeof(aw::ChunkRec),
                        hipMemcpyHostToDevice, h->stream);
}

// Waits for what was enqueued, whether all of it was (e): the uploaded list goes
// with the caller, who may write the parameters and the workspace on any stream
// from then on.
hipError_t settle(ob_adamw_handle* h, hipError_t e) {
  const hipError_t w = hipStreamSynchronize(h->stream);
  return e != hipSuccess ? e : w;
}

// Validation common to init and attach, then a handle over the workspace.
ob_status make(const ob_adamw_config* cfg, const int64_t* numel, const int32_t* group,
               void* workspace, uint64_t ws_bytes, void* stream,
               std::vector<aw::ChunkRec>* recs, ob_adamw_handle** out) {
  const ob_status st = aw::check_config(cfg);
  if (st != OB_OK) return st;
  if (numel == nullptr) return OB_ERR_ARG;
  const int64_t length = aw::length_of(cfg, numel, nullptr);
  if (length < 0) return OB_ERR_SHAPE;
  for (int32_t i = 0; group != nullptr && i < cfg->n_tensors; ++i)
    if (group[i] < 0 || group[i] >= cfg->n_groups) return OB_ERR_ARG;
  const aw::Places at = aw::places_of(cfg, numel, length, sizeof(aw::Control));
  if (workspace == nullptr || !aw::aligned(workspace, 256) || ws_bytes < at.total)
    return OB_ERR_WORKSPACE;
  bool busy = false;
  if (capturing((hipStream_t)stream, &busy) != hipSuccess) return OB_ERR_HIP;
  if (busy) return OB_ERR_PHASE;
  hipPointerAttribute_t attr{};
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess || hipPointerGetAttributes(&attr, workspace) != hipSuccess) {
    (void)hipGetLastError();  // reported here, not by the caller's next launch
    return OB_ERR_HIP;
  }
  if (attr.device != cur || attr.type != hipMemoryTypeDevice) return OB_ERR_ARG;
  ob_adamw_handle* h = new ob_adamw_handle();
  *out = h;
  h->plan.make(*cfg, numel, group, recs);
  h->at = at;
  h->base = (char*)workspace;
  h->device = cur;
  h->stream = (hipStream_t)stream;
  aw::State& s = h->st;
  s.control = (aw::Control*)(h->base + at.control);
  s.recs = (const aw::ChunkRec*)(h->base + at.recs);
  s.partials = (double*)(h->base + at.partials);
  s.m = h->base + at.m;
  s.v = h->base + at.v;
  s.m_exp = (uint8_t*)(h->base + at.m_exp);
  s.v_exp = (uint8_t*)(h->base + at.v_exp);
  s.master = (float*)(h->base + at.master);
  s.beta1 = cfg->beta1;
  s.beta2 = cfg->beta2;
  s.eps = cfg->eps;
  s.param_bf16 = cfg->param_dtype == OB_ADAMW_BF16;
  s.grad_bf16 = cfg->grad_dtype == OB_ADAMW_BF16;
  s.state_bits = cfg->state_bits;
  s.has_master = cfg->master;
  s.stochastic = cfg->stochastic;
  return OB_OK;
}

void fill_ptrs(const aw::Span& s, const void* const* params, const void* const* grads,
               aw::StepPtrs* p) {
  for (int32_t i = 0; i < s.n; ++i) {
    p->g[i] = grads != nullptr ? grads[s.t0 + i] : nullptr;
    p->p[i] = const_cast<void*>(params[s.t0 + i]);
  }
}

// `fn(first chunk, chunks)` over a span, in equal launches of at most that size.
template <typename F>
hipError_t launches(ob_adamw_t h, const aw::Span& s, F fn) {
  const int64_t most = h->plan.cfg.state_bits == 32 ? kChunks32 : kChunks8;
  const int64_t parts = (s.chunks + most - 1) / most, per = (s.chunks + parts - 1) / parts;
  hipError_t e = hipSuccess;
  for (int64_t c = 0; c < s.chunks && e == hipSuccess; c += per)
    e = fn(s.c0 + c, std::min(per, s.chunks - c));
  return e;
}

// The partial sums of squares of every span; in front of a step (backwards)
// the first span last, with which the step begins.
hipError_t norm_pass(ob_adamw_t h, const void* const* grads, bool backwards) {
  const size_t spans = h->plan.norm_spans.size();
  int64_t at = 0;
  for (size_t i = 0; i < spans; ++i) {
    const aw::Span& s = h->plan.norm_spans[backwards ? spans - 1 - i : i];
    aw::NormPtrs p;
    for (int32_t k = 0; k < s.n; ++k) p.g[k] = grads[s.t0 + k];
    const hipError_t e =
        aw::launch_norm(h->st, p, (uint32_t)s.t0, s.c0, s.chunks, at, backwards, h->stream);
    if (e != hipSuccess) return e;
    at += aw::norm_partials(s.chunks);
  }
  return hipSuccess;
}

void* address_of(ob_adamw_t h, int32_t field) {
  switch (field) {
    case OB_ADAMW_M: return h->st.m;
    case OB_ADAMW_V: return h->st.v;
    case OB_ADAMW_MASTER: return h->st.master;
    case OB_ADAMW_M_EXP: return h->st.m_exp;
    default: return h->st.v_exp;
  }
}

constexpr uint32_t kGuardBase = 64;  // guard words apart from those of ob_adam workspaces

// beta^steps by as many products.  A power of a beta above a half ends among
// the smallest denormals, which a product with it leaves as they are, so no
// beta up to 0.9999 takes more than 7.4 million products (27 ms).
double power_of(float beta, int64_t steps) {
  double p = 1.0;
  for (int64_t i = 0; i < steps; ++i) {
    const double next = p * (double)beta;
    if (next == p) break;
    p = next;
  }
  return p;
}

hipError_t set_steps(ob_adamw_t h, int64_t steps) {
  return aw::launch_set_steps(h->st, steps, power_of(h->plan.cfg.beta1, steps),
                              power_of(h->plan.cfg.beta2, steps), h->stream);
}

// `fn()` with every C++ exception (the host lists' memory) turned into a status.
template <typename F>
ob_status guarded(F fn) {
  try {
    return fn();
  } catch (...) {
    return OB_ERR_ARG;
  }
}

// Clear the state and write the guards and the first control block.
hipError_t first_state(ob_adamw_t h) {
  const aw::Places& l = h->at;
  hipError_t e = aw::launch_fill(h->base, 0, l.total / 4, h->stream);
  for (int i = 0; i < aw::kNumGuards && e == hipSuccess; ++i)
    e = aw::launch_fill(h->base + l.guard[i], ob::guard_word(kGuardBase + i), ob::kGuardBytes / 4,
                        h->stream);
  const uint64_t exps = h->plan.cfg.state_bits == 8 ? (uint64_t)h->plan.length / aw::kScaleElems : 0;
  if (e == hipSuccess)
    e = aw::launch_fill(h->st.m_exp, aw::kMinExpM * 0x01010101u, exps / 4, h->stream);
  if (e == hipSuccess)
    e = aw::launch_fill(h->st.v_exp, aw::kMinExpV * 0x01010101u, exps / 4, h->stream);
  if (e == hipSuccess) e = set_steps(h, 0);
  return e;
}

}  // namespace

extern "C" {

ob_status ob_adamw_layout(const ob_adamw_config* cfg, const int64_t* numel, int64_t* offsets,
                          int64_t* length, uint64_t* bytes) {
  const ob_status st = aw::check_config(cfg);
  if (st != OB_OK) return st;
  if (numel == nullptr || length == nullptr || bytes == nullptr) return OB_ERR_ARG;
  if (aw::length_of(cfg, numel, nullptr) < 0) return OB_ERR_SHAPE;
  *length = aw::length_of(cfg, numel, offsets);
  *bytes = aw::places_of(cfg, numel, *length, sizeof(aw::Control)).total;
  return OB_OK;
}

ob_status ob_adamw_init(const ob_adamw_config* cfg, const int64_t* numel, const int32_t* group,
                        void* workspace, uint64_t ws_bytes, const void* const* params,
                        void* stream, ob_adamw_t* out) {
  if (out == nullptr) return OB_ERR_ARG;
  ob_adamw_handle* h = nullptr;
  const ob_status st = guarded([&]() -> ob_status {
    std::vector<aw::ChunkRec> recs;
    ob_status r = make(cfg, numel, group, workspace, ws_bytes, stream, &recs, &h);
    if (r != OB_OK) return r;
    const bool copies = cfg->master && params != nullptr;
    for (int32_t i = 0; copies && i < cfg->n_tensors; ++i)
      if (numel[i] > 0 && (params[i] == nullptr || !aw::aligned(params[i], 2))) return OB_ERR_ARG;
    hipError_t e = first_state(h);
    if (e == hipSuccess) e = upload(h, recs);
    for (size_t i = 0; copies && i < h->plan.step_spans.size() && e == hipSuccess; ++i) {
      const aw::Span& s = h->plan.step_spans[i];
      aw::StepPtrs p;
      fill_ptrs(s, params, nullptr, &p);
      e = launches(h, s, [&](int64_t c, int64_t n) {
        return aw::launch_master(h->st, p, (uint32_t)s.t0, c, n, h->stream);
      });
    }
    return settle(h, e) == hipSuccess ? OB_OK : OB_ERR_HIP;
  });
  if (st != OB_OK) {
    delete h;
    return st;
  }
  *out = h;
  return OB_OK;
}

ob_status ob_adamw_attach(const ob_adamw_config* cfg, const int64_t* numel, const int32_t* group,
                          void* workspace, uint64_t ws_bytes, void* stream, ob_adamw_t* out) {
  if (out == nullptr) return OB_ERR_ARG;
  ob_adamw_handle* h = nullptr;
  const ob_status st = guarded([&]() -> ob_status {
    std::vector<aw::ChunkRec> recs;
    const ob_status r = make(cfg, numel, group, workspace, ws_bytes, stream, &recs, &h);
    if (r != OB_OK) return r;
    return settle(h, upload(h, recs)) == hipSuccess ? OB_OK : OB_ERR_HIP;
  });
  if (st != OB_OK) {
    delete h;
    return st;
  }
  *out = h;
  return OB_OK;
}

ob_status ob_adamw_grad_norm(ob_adamw_t h, const void* const* grads, float grad_scale,
                             double* sumsq, float* norm) {
  ob_status st = usable(h);
  if (st != OB_OK) return st;
  if (!aw::valid_scale(grad_scale) || !aw::aligned(sumsq, 8) || !aw::aligned(norm, 4))
    return OB_ERR_ARG;
  st = h->plan.check_grads(grads);
  if (st != OB_OK) return st;
  if (h->plan.small) {
    aw::SmallNorm k{h->st.recs, h->st.control, h->st.partials, sumsq, norm, grad_scale, {}};
    for (int32_t i = 0; i < h->plan.cfg.n_tensors; ++i) k.g[i] = grads[i];
    return fail(h, aw::launch_small_norm(k, h->st.grad_bf16, h->plan.chunks, h->stream));
  }
  hipError_t e = norm_pass(h, grads, false);
  if (e == hipSuccess)
    e = aw::launch_norm_finish(h->st, h->plan.n_partials, grad_scale, sumsq, norm, h->stream);
  return fail(h, e);
}

ob_status ob_adamw_step(ob_adamw_t h, const void* const* params, const void* const* grads,
                        const ob_adamw_step_args* a) {
  ob_status st = usable(h);
  if (st != OB_OK) return st;
  st = h->plan.check_step(a);
  if (st == OB_OK) st = h->plan.check_ptrs(params, grads, h->base, h->at.total);
  if (st != OB_OK) return st;
  aw::ControlArgs c{};
  for (int32_t i = 0; i < h->plan.cfg.n_groups; ++i) {
    c.lr[i] = a->lr_device == nullptr ? a->lr[i] : 0.0f;
    c.wd[i] = a->weight_decay != nullptr ? a->weight_decay[i] : 0.0f;
  }
  c.lr_device = a->lr_device;
  c.norm = a->norm;
  c.seed = h->plan.cfg.seed;
  c.beta1 = h->plan.cfg.beta1;
  c.beta2 = h->plan.cfg.beta2;
  c.grad_scale = a->grad_scale;
  c.max_norm = a->max_norm;
  c.n_groups = h->plan.cfg.n_groups;
  c.skip_nonfinite = a->skip_nonfinite;
  c.sumsq = a->sumsq;
  hipError_t e = hipSuccess;
  if (a->sumsq == nullptr && (a->max_norm > 0.0f || a->skip_nonfinite || a->norm != nullptr)) {
    e = norm_pass(h, grads, true);
    c.partials = h->st.partials;
    c.n_partials = h->plan.n_partials;
  }
  if (e == hipSuccess && h->plan.small) {
    aw::SmallStep k;
    k.s = h->st;
    k.a = c;
    for (int32_t i = 0; i < h->plan.cfg.n_tensors; ++i) {
      k.g[i] = grads[i];
      k.p[i] = const_cast<void*>(params[i]);
    }
    return fail(h, aw::launch_small(k, h->plan.chunks, h->stream));
  }
  if (e == hipSuccess) e = aw::launch_control(h->st, c, h->stream);
  for (size_t i = 0; i < h->plan.step_spans.size() && e == hipSuccess; ++i) {
    const aw::Span& s = h->plan.step_spans[i];
    aw::StepPtrs p;
    fill_ptrs(s, params, grads, &p);
    e = launches(h, s, [&](int64_t c0, int64_t n) {
      return aw::launch_step(h->st, p, (uint32_t)s.t0, c0, n, h->stream);
    });
  }
  return fail(h, e);
}

ob_status ob_adamw_get_state(ob_adamw_t h, int32_t field, int64_t offset, int64_t count,
                             int32_t type, void* dst) {
  ob_status st = usable(h);
  if (st != OB_OK) return st;
  st = h->plan.check_range(field, offset, count, false);
  if (st != OB_OK) return st;
  if (!aw::dtype(type)) return OB_ERR_ARG;
  if (count == 0) return OB_OK;
  if (dst == nullptr || !aw::aligned(dst, aw::size_of(type))) return OB_ERR_ARG;
  return fail(h, aw::launch_get(h->st, field, offset, count, type == OB_ADAMW_BF16, dst,
                                h->stream));
}

ob_status ob_adamw_set_state(ob_adamw_t h, int32_t field, int64_t offset, int64_t count,
                             const float* src) {
  ob_status st = usable(h);
  if (st != OB_OK) return st;
  st = h->plan.check_range(field, offset, count, true);
  if (st != OB_OK) return st;
  if (count == 0) return OB_OK;
  if (src == nullptr || !aw::aligned(src, 4)) return OB_ERR_ARG;
  return fail(h, aw::launch_set(h->st, field, offset, count, src, h->stream));
}

ob_status ob_adamw_state(ob_adamw_t h, int32_t field, void** device, uint64_t* bytes) {
  if (h == nullptr || device == nullptr || bytes == nullptr) return OB_ERR_ARG;
  uint64_t elem, count;
  if (!h->plan.field(field, &elem, &count)) return OB_ERR_ARG;
  *device = address_of(h, field);
  *bytes = elem * count;
  return OB_OK;
}

ob_status ob_adamw_set_steps(ob_adamw_t h, int64_t steps) {
  const ob_status st = usable(h);
  if (st != OB_OK) return st;
  if (steps < 0 || steps > kMaxSteps) return OB_ERR_ARG;
  return fail(h, set_steps(h, steps));
}

ob_status ob_adamw_get_steps(ob_adamw_t h, int64_t* steps, int64_t* skipped) {
  const ob_status st = usable(h);
  if (st != OB_OK) return st;
  if (steps == nullptr || skipped == nullptr) return OB_ERR_ARG;
  bool busy = false;
  if (capturing(h->stream, &busy) != hipSuccess) return fail(h, hipErrorUnknown);
  if (busy) return OB_ERR_PHASE;
  if (hipStreamSynchronize(h->stream) != hipSuccess) return fail(h, hipErrorUnknown);
  int64_t both[2];
  static_assert(offsetof(aw::Control, steps) == 0 && offsetof(aw::Control, skipped) == 8,
                "the counts lead the control block");
  if (hipMemcpy(both, h->st.control, sizeof both, hipMemcpyDeviceToHost) != hipSuccess)
    return fail(h, hipErrorUnknown);
  *steps = both[0];
  *skipped = both[1];
  return OB_OK;
}

ob_status ob_adamw_check_guards(ob_adamw_t h, int32_t* first_bad) {
  const ob_status st = usable(h);
  if (st != OB_OK) return st;
  if (first_bad == nullptr) return OB_ERR_ARG;
  bool busy = false;
  if (capturing(h->stream, &busy) != hipSuccess) return fail(h, hipErrorUnknown);
  if (busy) return OB_ERR_PHASE;
  if (hipStreamSynchronize(h->stream) != hipSuccess) return fail(h, hipErrorUnknown);
  uint32_t words[ob::kGuardBytes / 4];
  *first_bad = -1;
  for (int i = 0; i < aw::kNumGuards && *first_bad < 0; ++i) {
    if (hipMemcpy(words, h->base + h->at.guard[i], sizeof words, hipMemcpyDeviceToHost) !=
        hipSuccess)
      return fail(h, hipErrorUnknown);
    for (uint32_t w : words)
      if (w != ob::guard_word(kGuardBase + i)) *first_bad = i;
  }
  return OB_OK;
}

ob_status ob_adamw_set_stream(ob_adamw_t h, void* stream) {
  if (h == nullptr) return OB_ERR_ARG;
  h->stream = (hipStream_t)stream;
  return OB_OK;
}

ob_status ob_adamw_destroy(ob_adamw_t h) {
  if (h == nullptr) return OB_ERR_ARG;
  delete h;
  return OB_OK;
}

}  // extern "C"
