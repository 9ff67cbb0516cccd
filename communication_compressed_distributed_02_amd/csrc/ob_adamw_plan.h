// The host side's arithmetic behind the ob_adamw C interface: validation, the
// workspace's layout, the list of chunks and the pointer checks.  No HIP in
// it, so that it is tested on its own.
#pragma once

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "ob_adamw.h"

namespace ob {
namespace adamw {

constexpr int kBlock = 256;         // threads of a block: 4 waves
constexpr int kRowElems = 1024;     // a tensor's state starts at a multiple of it
constexpr int kChunkElems = 4 * kRowElems;  // a record's share of one tensor
constexpr int kScaleElems = 256;    // elements that share the exponents of an 8-bit state
constexpr int kMaxGroups = OB_ADAMW_MAX_GROUPS;
// Pointers travel by value in the kernel arguments (4 KB of them), so a
// captured launch holds its own and no table in memory is shared.
constexpr int kPtrsPerStep = 240;
constexpr int kPtrsPerNorm = 480;
constexpr int kNormBlocks = 2048;   // partial sums of one launch of the norm, at most
// A step over at most so many chunks (2^20 elements) and tensors is one launch
// without a control kernel in front, and a norm over them one without a
// kernel behind (a partial sum a thread of the block that folds them).  The
// step in one launch and in two, 32-bit states: 4.2 and 6.0 us at 4 chunks, 7.4
// and 8.5 at 256, 10.5 and 13.3 at 512, 21.9 and 22.8 at 1024; 8-bit ones: 4.3
// and 6.1 at 4, 7.5 and 7.2 at 256, 9.3 and 9.2 at 512, 15.2 and 14.6 at 1024.
// Clipped, 32-bit: 11.3 and 13.0 at 256, 15.6 and 16.9 at 512, 30.5 and 27.0 at
// 1024; 8-bit: 11.4 and 12.5, 14.6 and 13.3, 24.1 and 20.0.  So 256 is the limit
// for 8-bit states; with 32-bit ones one launch would win at 512 as well.
constexpr int kSmallChunks = 256;
constexpr int kSmallTensors = 96;
constexpr int kLeaves = 16;  // counters that the tickets of a small launch go over
constexpr int32_t kMaxTensors = 1 << 20;
constexpr int64_t kMaxLength = int64_t(1) << 40;  // of a state array; no size below can overflow
constexpr int kNumGuards = 8;
constexpr uint64_t kGuardGap = 256;

// One chunk of work: `count` elements of tensor `tensor` from its element
// 1024*row, whose state starts at element 1024*state_row.
struct ChunkRec {
  uint32_t tensor;
  uint32_t row;
  uint32_t state_row;
  uint16_t count;
  uint16_t group;
};
static_assert(sizeof(ChunkRec) == 16, "one scalar load");

// Tensors whose pointers go with one launch, and their chunks.
struct Span {
  int32_t t0, n;
  int64_t c0, chunks;
};

// Byte offsets of the workspace's buffers, each followed by a guard.
struct Places {
  uint64_t control, recs, partials, m, v, m_exp, v_exp, master, total;
  uint64_t guard[kNumGuards];
};

// Memory that a step reads or writes, for the overlap check.
struct Range {
  uintptr_t begin, end;
  bool written;
};

inline bool aligned(const void* p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
inline uint64_t up256(uint64_t x) { return (x + 255u) & ~uint64_t(255); }
inline bool valid_beta(float b) { return isfinite(b) && b >= 0.0f && b < 1.0f; }
inline bool valid_scale(float s) { return isfinite(s) && s > 0.0f; }
inline bool flag(int32_t v) { return v == 0 || v == 1; }
inline bool dtype(int32_t v) { return v == OB_ADAMW_F32 || v == OB_ADAMW_BF16; }
inline uint64_t size_of(int32_t dtype) { return dtype == OB_ADAMW_BF16 ? 2 : 4; }
inline int64_t rows_of(int64_t numel) { return (numel + kRowElems - 1) / kRowElems; }
inline int64_t chunks_of(int64_t numel) { return (numel + kChunkElems - 1) / kChunkElems; }
// Partial sums that a norm over n chunks leaves.
inline int64_t norm_partials(int64_t n) { return n < kNormBlocks ? n : kNormBlocks; }

inline ob_status check_config(const ob_adamw_config* c) {
  if (c == nullptr) return OB_ERR_ARG;
  if (!dtype(c->param_dtype) || !dtype(c->grad_dtype)) return OB_ERR_ARG;
  if (c->state_bits != 0 && c->state_bits != 8 && c->state_bits != 32) return OB_ERR_ARG;
  if (!flag(c->master) || !flag(c->stochastic)) return OB_ERR_ARG;
  if ((c->master || c->stochastic) && c->param_dtype != OB_ADAMW_BF16) return OB_ERR_ARG;
  if (c->master && (c->stochastic || c->state_bits == 0)) return OB_ERR_ARG;
  if (!valid_beta(c->beta1) || !valid_beta(c->beta2) || !isfinite(c->eps) || !(c->eps > 0.0f))
    return OB_ERR_ARG;
  if (c->n_groups < 1 || c->n_groups > OB_ADAMW_MAX_GROUPS) return OB_ERR_ARG;
  if (c->n_tensors < 1 || c->n_tensors > kMaxTensors) return OB_ERR_SHAPE;
  return OB_OK;
}

// Elements of a state array, or -1 where the counts are not allowed.
inline int64_t length_of(const ob_adamw_config* c, const int64_t* numel, int64_t* offsets) {
  int64_t at = 0;
  for (int32_t i = 0; i < c->n_tensors; ++i) {
    if (numel[i] < 0 || numel[i] > kMaxLength) return -1;
    if (offsets != nullptr) offsets[i] = at;
    at += rows_of(numel[i]) * kRowElems;
    if (at > kMaxLength) return -1;
  }
  return at;
}

// Chunks of tensors [t, t + per), as far as there are any.
inline int64_t chunks_from(const ob_adamw_config* c, const int64_t* numel, int32_t t, int32_t per) {
  int64_t n = 0;
  for (int32_t i = t; i < c->n_tensors && i < t + per; ++i) n += chunks_of(numel[i]);
  return n;
}

inline Places places_of(const ob_adamw_config* c, const int64_t* numel, int64_t length,
                        uint64_t control_bytes) {
  const uint64_t chunks = (uint64_t)chunks_from(c, numel, 0, c->n_tensors);
  int64_t partials = 0;
  for (int32_t t = 0; t < c->n_tensors; t += kPtrsPerNorm)
    partials += norm_partials(chunks_from(c, numel, t, kPtrsPerNorm));
  const uint64_t n = (uint64_t)length, state = n * (uint64_t)(c->state_bits / 8);
  const uint64_t exps = c->state_bits == 8 ? n / kScaleElems : 0;
  Places l{};
  uint64_t at = 0;
  int i = 0;
  auto place = [&](uint64_t bytes) {
    const uint64_t start = at;
    l.guard[i++] = up256(start + bytes);
    at = up256(start + bytes) + kGuardGap;
    return start;
  };
  l.control = place(control_bytes);
  l.recs = place(chunks * sizeof(ChunkRec));
  l.partials = place((uint64_t)partials * sizeof(double));
  l.m = place(state);
  l.v = place(state);
  l.m_exp = place(exps);
  l.v_exp = place(exps);
  l.master = place(c->master ? 4 * n : 0);
  l.total = at;
  return l;
}

// The tensors, their chunks and the spans of both kinds of launch.
struct Plan {
  ob_adamw_config cfg{};
  int64_t length = 0;      // elements of a state array
  int64_t n_partials = 0;
  std::vector<int64_t> numel;
  std::vector<Span> step_spans, norm_spans;
  int64_t chunks = 0;
  bool small = false;      // few enough chunks and tensors for the launches of small steps
  // the pointers that passed the checks last, and room for the check
  std::vector<const void*> seen_p, seen_g;
  std::vector<Range> ranges;

  // May throw std::bad_alloc.  group may be null.
  void make(const ob_adamw_config& c, const int64_t* sizes, const int32_t* group,
            std::vector<ChunkRec>* recs) {
    cfg = c;
    length = length_of(&c, sizes, nullptr);
    numel.assign(sizes, sizes + c.n_tensors);
    seen_p.assign(c.n_tensors, nullptr);
    seen_g.assign(c.n_tensors, nullptr);
    ranges.reserve(2 * (size_t)c.n_tensors + 1);
    recs->reserve((size_t)chunks_from(&c, sizes, 0, c.n_tensors));
    int64_t row = 0;
    for (int32_t i = 0; i < c.n_tensors; ++i) {
      for (int64_t at = 0; at < numel[i]; at += kChunkElems) {
        ChunkRec r{};
        r.tensor = (uint32_t)i;
        r.row = (uint32_t)(at / kRowElems);
        r.state_row = (uint32_t)(row + at / kRowElems);
        r.count = (uint16_t)std::min<int64_t>(kChunkElems, numel[i] - at);
        r.group = (uint16_t)(group != nullptr ? group[i] : 0);
        recs->push_back(r);
      }
      row += rows_of(numel[i]);
    }
    chunks = (int64_t)recs->size();
    small = chunks > 0 && chunks <= kSmallChunks && c.n_tensors <= kSmallTensors;
    list_spans(kPtrsPerStep, &step_spans);
    list_spans(kPtrsPerNorm, &norm_spans);
    for (const Span& s : norm_spans) n_partials += norm_partials(s.chunks);
  }

  void list_spans(int32_t per, std::vector<Span>* out) const {
    int64_t c0 = 0;
    for (int32_t t = 0; t < cfg.n_tensors; t += per) {
      const int64_t chunks = chunks_from(&cfg, numel.data(), t, per);
      if (chunks > 0) out->push_back({t, std::min(per, cfg.n_tensors - t), c0, chunks});
      c0 += chunks;
    }
  }

  // Pointers at element alignment, none missing that is needed, and nothing
  // that is written ([base, base + ws_bytes) among it) overlapping anything
  // else.  What passed last passes again without the sort.
  ob_status check_ptrs(const void* const* params, const void* const* grads, const void* base,
                       uint64_t ws_bytes) {
    const size_t n = (size_t)cfg.n_tensors, bytes = n * sizeof(void*);
    if (params == nullptr || grads == nullptr) return OB_ERR_ARG;
    if (memcmp(params, seen_p.data(), bytes) == 0 && memcmp(grads, seen_g.data(), bytes) == 0)
      return OB_OK;
    const uint64_t pb = size_of(cfg.param_dtype), gb = size_of(cfg.grad_dtype);
    std::vector<Range>& r = ranges;  // its memory is reserved: nothing here allocates
    r.clear();
    r.push_back({(uintptr_t)base, (uintptr_t)base + ws_bytes, true});
    for (size_t i = 0; i < n; ++i) {
      if (numel[i] == 0 || grads[i] == nullptr) continue;
      if (params[i] == nullptr || !aligned(params[i], pb) || !aligned(grads[i], gb))
        return OB_ERR_ARG;
      const uintptr_t p = (uintptr_t)params[i], g = (uintptr_t)grads[i];
      r.push_back({p, p + pb * (uint64_t)numel[i], true});
      r.push_back({g, g + gb * (uint64_t)numel[i], false});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
    uintptr_t any = 0, written = 0;  // furthest ends so far
    for (const Range& x : r) {
      if (x.begin < (x.written ? any : written)) return OB_ERR_ARG;
      any = std::max(any, x.end);
      if (x.written) written = std::max(written, x.end);
    }
    memcpy(seen_p.data(), params, bytes);
    memcpy(seen_g.data(), grads, bytes);
    return OB_OK;
  }

  ob_status check_grads(const void* const* grads) const {
    if (grads == nullptr) return OB_ERR_ARG;
    for (int32_t i = 0; i < cfg.n_tensors; ++i)
      if (!aligned(grads[i], size_of(cfg.grad_dtype))) return OB_ERR_ARG;
    return OB_OK;
  }

  ob_status check_step(const ob_adamw_step_args* a) const {
    if (cfg.state_bits == 0) return OB_ERR_PHASE;
    if (a == nullptr || (a->lr == nullptr && a->lr_device == nullptr) ||
        !flag(a->skip_nonfinite) || !valid_scale(a->grad_scale) || !(a->max_norm >= 0.0f) ||
        !aligned(a->lr_device, 4) || !aligned(a->sumsq, 8) || !aligned(a->norm, 4))
      return OB_ERR_ARG;
    for (int32_t i = 0; i < cfg.n_groups; ++i) {
      if (a->lr_device == nullptr && !isfinite(a->lr[i])) return OB_ERR_ARG;
      if (a->weight_decay != nullptr && !isfinite(a->weight_decay[i])) return OB_ERR_ARG;
    }
    return OB_OK;
  }

  // A field's stored element bytes and elements; false for one the plan lacks.
  bool field(int32_t f, uint64_t* elem, uint64_t* count) const {
    const bool exp = f == OB_ADAMW_M_EXP || f == OB_ADAMW_V_EXP;
    *elem = exp ? 1 : (f == OB_ADAMW_MASTER ? 4 : (uint64_t)cfg.state_bits / 8);
    *count = (uint64_t)length / (exp ? kScaleElems : 1);
    if (exp) return cfg.state_bits == 8;
    if (f == OB_ADAMW_MASTER) return cfg.master != 0;
    return (f == OB_ADAMW_M || f == OB_ADAMW_V) && cfg.state_bits != 0;
  }

  ob_status check_range(int32_t f, int64_t offset, int64_t count, bool whole_groups) const {
    uint64_t elem, size;
    if (f == OB_ADAMW_M_EXP || f == OB_ADAMW_V_EXP || !field(f, &elem, &size)) return OB_ERR_ARG;
    if (offset < 0 || count < 0 || offset > (int64_t)size || count > (int64_t)size - offset)
      return OB_ERR_ARG;
    if (whole_groups && elem == 1 && (offset % kScaleElems != 0 || count % kScaleElems != 0))
      return OB_ERR_ARG;
    return OB_OK;
  }
};

}  // namespace adamw
}  // namespace ob
