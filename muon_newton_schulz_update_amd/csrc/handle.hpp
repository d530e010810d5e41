// What the training-step entry points (train_api.cpp) use of a handle whose
// definition is api.cpp's.
#pragma once
#include <hip/hip_runtime.h>

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

}  // namespace muon
