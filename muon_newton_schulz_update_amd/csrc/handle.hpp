// What the entry points beside the matrix step (train_api.cpp, norm_api.cpp) use
// of a handle whose definition is api.cpp's.
#pragma once
#include <hip/hip_runtime.h>

#include <new>
#include <string>
#include <vector>

#include "../../include/libmuon.h"

namespace muon {

// A device buffer that grows on demand and is freed with the handle. Each
// user has its own: the Newton-Schulz workspace keeps zero padding that no
// other kernel may write. What it outgrows is freed, unless a call on it was
// captured: then a graph may still replay on it, and it is kept until the
// handle goes. It grows at least by half, but by no more than kGrowMost past
// what is asked for.
constexpr size_t kGrowMost = size_t(256) << 20;
struct GrowBuffer {
  void* ptr = nullptr;
  size_t bytes = 0;
  bool captured = false;         // a captured call uses it
  std::vector<void*> outgrown;
  void release() {
    if (ptr) (void)hipFree(ptr);
    for (void* p : outgrown) (void)hipFree(p);
    outgrown.clear();
    ptr = nullptr;
    bytes = 0;
    captured = false;
  }
};
struct TrainState {
  GrowBuffer head;            // cross entropy pieces
  GrowBuffer norm;            // NormState
  GrowBuffer rows;            // sums of the norms' gradients
  bool norm_clean = false;    // the norm kernel's ticket is 0
};

TrainState& train_state(muon_handle* h);
hipStream_t handle_stream(const muon_handle* h);
int handle_device(const muon_handle* h);
muon_status handle_error(muon_handle* h, muon_status code, const std::string& msg);
void handle_clear_error(muon_handle* h);
bool handle_capturing(const muon_handle* h);     // whether the handle's stream is being captured
// At least `bytes` of b for a call that is about to be enqueued (to be called
// for every use: it notes the captured ones).
muon_status grow(muon_handle* h, GrowBuffer& b, size_t bytes, const char* what);

#define HIP_DO(h, expr)                                                                                     \
  do {                                                                                                      \
    hipError_t e_ = (expr);                                                                                 \
    if (e_ != hipSuccess)                                                                                   \
      return handle_error((h), MUON_ERR_HIP, std::string(#expr) + ": " + hipGetErrorString(e_));            \
  } while (0)

// Runs an entry point's body with the handle's device current and keeps
// exceptions (allocation failure in the host-side checks) from the caller.
template <typename F>
muon_status guarded(muon_handle* h, F body) noexcept {
  if (!h) return MUON_ERR_INVALID_ARG;
  int before = -1;
  const int want = handle_device(h);
  if (hipGetDevice(&before) != hipSuccess) before = want;
  if (before != want && hipSetDevice(want) != hipSuccess) {
    (void)hipGetLastError();
    return MUON_ERR_HIP;
  }
  muon_status r;
  try {
    r = body();
  } catch (const std::bad_alloc&) {
    r = MUON_ERR_ALLOC;
  } catch (...) {
    r = MUON_ERR_INVALID_ARG;
  }
  if (before != want) (void)hipSetDevice(before);
  return r;
}

}  // namespace muon
