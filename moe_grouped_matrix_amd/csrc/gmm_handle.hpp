// gmm_handle.hpp -- the library handle and the host helpers that every C entry
// point uses.
#pragma once

#include <hip/hip_runtime.h>

#include <map>
#include <string>

#include "gmm.h"

struct gmm_handle {
  int device = 0;
  int cu_count = 0;
  uint32_t* flags = nullptr;  // device word of data-error flags (kDeviceBlock bytes)
  // the transposed product's work-queue counters (kQueueWords int32, zero
  // between calls), one block per stream: calls on one stream run in order,
  // so each call finds its stream's counters reset by the previous one;
  // calls on different streams never share counters
  std::map<void*, int32_t*> queues;
  int tile_policy = 0;        // 0 auto, 1 small tiles, 2 big tiles
  int grid_limit = 0;         // > 0: at most this many workgroups per launch
  void* scratch = nullptr;    // device address of the device's static scratch
  std::string err;
};

namespace gmmh {

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) prev = -1;
    if (prev != dev) (void)hipSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

inline gmm_status fail(gmm_handle* h, gmm_status st, const std::string& msg) {
  if (h) h->err = msg;
  return st;
}

}  // namespace gmmh
