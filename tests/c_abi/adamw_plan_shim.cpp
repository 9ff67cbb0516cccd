// Test access to the host arithmetic behind ob_adamw (ob_adamw_plan.h), which
// has no HIP in it: built with g++ and the sanitizers, called through ctypes.
#include "ob_adamw_plan.h"

using namespace ob::adamw;

extern "C" {

int shim_config(const ob_adamw_config* c) { return check_config(c); }

int64_t shim_length(const ob_adamw_config* c, const int64_t* numel, int64_t* offsets) {
  return length_of(c, numel, offsets);
}

// recs: room for `room` records; returns how many there are.
int64_t shim_recs(const ob_adamw_config* c, const int64_t* numel, const int32_t* group,
                  ChunkRec* recs, int64_t room, int64_t* n_partials) {
  Plan p;
  std::vector<ChunkRec> r;
  p.make(*c, numel, group, &r);
  *n_partials = p.n_partials;
  for (int64_t i = 0; i < room && i < (int64_t)r.size(); ++i) recs[i] = r[(size_t)i];
  return (int64_t)r.size();
}

// spans of the step (which = 0) or of the norm, four numbers each.
int64_t shim_spans(const ob_adamw_config* c, const int64_t* numel, int which, int64_t* out,
                   int64_t room) {
  Plan p;
  std::vector<ChunkRec> r;
  p.make(*c, numel, nullptr, &r);
  const std::vector<Span>& s = which ? p.norm_spans : p.step_spans;
  for (int64_t i = 0; i < room && i < (int64_t)s.size(); ++i) {
    const Span& x = s[(size_t)i];
    const int64_t four[4] = {x.t0, x.n, x.c0, x.chunks};
    memcpy(out + 4 * i, four, sizeof four);
  }
  return (int64_t)s.size();
}

void shim_places(const ob_adamw_config* c, const int64_t* numel, uint64_t control, Places* out) {
  *out = places_of(c, numel, length_of(c, numel, nullptr), control);
}

// The pointer check `times` times over (the later ones take the short way).
int shim_ptrs(const ob_adamw_config* c, const int64_t* numel, const void* const* params,
              const void* const* grads, const void* base, uint64_t ws_bytes, int times) {
  Plan p;
  std::vector<ChunkRec> r;
  p.make(*c, numel, nullptr, &r);
  int st = OB_OK;
  for (int i = 0; i < times; ++i) st = p.check_ptrs(params, grads, base, ws_bytes);
  return st;
}

int shim_step(const ob_adamw_config* c, const int64_t* numel, const ob_adamw_step_args* a) {
  Plan p;
  std::vector<ChunkRec> r;
  p.make(*c, numel, nullptr, &r);
  return p.check_step(a);
}

int shim_range(const ob_adamw_config* c, const int64_t* numel, int32_t field, int64_t offset,
               int64_t count, int whole) {
  Plan p;
  std::vector<ChunkRec> r;
  p.make(*c, numel, nullptr, &r);
  return p.check_range(field, offset, count, whole != 0);
}

}  // extern "C"
