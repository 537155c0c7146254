// Host-only stand-ins for the launchers of the block operators: linked with
// block_api.cpp into a shared object built with a host compiler and the
// sanitizers. Each records the call, touches no pointer and reports success.
#include <atomic>

#include "block.h"

namespace {
std::atomic<int> g_launches{0};
hipError_t record() {
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return hipSuccess;
}
}  // namespace

extern "C" int retention_shim_launches(void) { return g_launches.load(std::memory_order_relaxed); }

namespace ret {

hipError_t launch_gated_recurrence(int, int, const View&, const View&, const View&, const Sequences&, const float*,
                                   float*, void*, hipStream_t) {
  return record();
}
hipError_t launch_gated_recurrence_backward(int, int, const View&, const View&, const View&, const View&, const View&,
                                            const View&, const Sequences&, const float*, const float*, float*, void*,
                                            hipStream_t) {
  return record();
}
hipError_t launch_gated_recurrence_step(int, int, const View&, const View&, const View&, int, int, int, float*, int,
                                        const int*, hipStream_t) {
  return record();
}
hipError_t launch_gated_norm(int, const View&, const View&, const View&, int, int, int, int, const NormArgs&,
                             hipStream_t) {
  return record();
}
hipError_t launch_gated_norm_backward(int, const View&, const View&, const View&, const View&, const View&, int, int,
                                      int, int, const NormArgs&, float*, float*, void*, hipStream_t) {
  return record();
}
hipError_t launch_residual_norm(int, int, const View&, const View&, const View&, const View&, int, int, int,
                                const NormArgs&, const float*, float, hipStream_t) {
  return record();
}
hipError_t launch_residual_norm_backward(int, int, const View&, const View&, const View&, const View&, const View&,
                                         const View&, const View&, int, int, int, const NormArgs&, const float*,
                                         float, float*, float*, float*, void*, hipStream_t) {
  return record();
}

}  // namespace ret
