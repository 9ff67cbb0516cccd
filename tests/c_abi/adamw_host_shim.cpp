// ob_adamw.hip, the host side behind the ob_adamw C interface, built with g++
// over a HIP runtime and launchers that do nothing but write down in which
// order they were called: one letter each, see the functions below.
#include "ob_adamw.hip"

#include <string>

namespace {
std::string calls;
double powers[2];
hipError_t note(char c) {
  calls += c;
  return hipSuccess;
}
}  // namespace

extern "C" {

const char* shim_calls() { return calls.c_str(); }
void shim_forget() { calls.clear(); }
// b1^t and b2^t as they were last set.
void shim_powers(double* out) { memcpy(out, powers, sizeof powers); }

hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  return *s = hipStreamCaptureStatusNone, hipSuccess;
}
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void*) {
  a->device = 0;
  a->type = hipMemoryTypeDevice;
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) {
  return note('u');  // an upload
}
hipError_t hipMemcpy(void*, const void*, size_t, hipMemcpyKind) { return note('r'); }  // a read-back
hipError_t hipStreamSynchronize(hipStream_t) { return note('w'); }  // a wait

}  // extern "C"

namespace ob {
namespace adamw {
hipError_t launch_small(const SmallStep&, int64_t, hipStream_t) { return note('s'); }
hipError_t launch_small_norm(const SmallNorm&, bool, int64_t, hipStream_t) { return note('n'); }
hipError_t launch_step(const State&, const StepPtrs&, uint32_t, int64_t, int64_t, hipStream_t) {
  return note('s');
}
hipError_t launch_norm(const State&, const NormPtrs&, uint32_t, int64_t, int64_t, int64_t, bool,
                       hipStream_t) {
  return note('n');
}
hipError_t launch_control(const State&, const ControlArgs&, hipStream_t) { return note('c'); }
hipError_t launch_norm_finish(const State&, int64_t, float, double*, float*, hipStream_t) {
  return note('n');
}
hipError_t launch_set_steps(const State&, int64_t, double p1, double p2, hipStream_t) {
  powers[0] = p1;
  powers[1] = p2;
  return note('t');
}
hipError_t launch_fill(void*, uint32_t, uint64_t, hipStream_t) { return note('f'); }
hipError_t launch_master(const State&, const StepPtrs&, uint32_t, int64_t, int64_t, hipStream_t) {
  return note('m');  // reads the parameters
}
hipError_t launch_get(const State&, int, int64_t, int64_t, bool, void*, hipStream_t) {
  return note('g');
}
hipError_t launch_set(const State&, int, int64_t, int64_t, const float*, hipStream_t) {
  return note('p');
}
}  // namespace adamw
}  // namespace ob
