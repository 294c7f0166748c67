// gmm_handle.hpp -- the library handle and the host helpers that every C entry
// point uses.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <map>
#include <mutex>
#include <string>
#include <thread>

#include "gmm.h"

namespace gmmh {

// The text of the last failure of every thread that used the handle.  A
// thread's text is written by that thread alone, so the pointer that it gets
// stays good until its own next call.
class ErrorTexts {
 public:
  void clear() {
    if (!any_.load(std::memory_order_relaxed)) return;  // (a thread sees its own set())
    std::lock_guard<std::mutex> lk(mu_);
    const auto it = text_.find(std::this_thread::get_id());
    if (it != text_.end()) it->second.clear();
  }
  void set(const std::string& text) {
    std::lock_guard<std::mutex> lk(mu_);
    text_[std::this_thread::get_id()] = text;
    any_.store(true, std::memory_order_relaxed);
  }
  const char* get() const {
    std::lock_guard<std::mutex> lk(mu_);
    const auto it = text_.find(std::this_thread::get_id());
    return it != text_.end() ? it->second.c_str() : "";
  }

 private:
  mutable std::mutex mu_;
  std::map<std::thread::id, std::string> text_;
  std::atomic<bool> any_{false};
};

}  // namespace gmmh

struct gmm_handle {
  int device = 0;
  int cu_count = 0;
  uint32_t* flags = nullptr;  // device word of data-error flags (kDeviceBlock bytes)
  // the transposed product's work-queue counters (kQueueWords int32, zero
  // between calls), one block per stream: calls on one stream run in order,
  // so each call finds its stream's counters reset by the previous one;
  // calls on different streams never share counters
  std::map<void*, int32_t*> queues;
  std::mutex queues_mu;                // held while queues is looked at or added to
  std::atomic<int> tile_policy{0};     // 0 auto, 1 small tiles, 2 big tiles
  std::atomic<int> grid_limit{0};      // > 0: at most this many workgroups per launch
  void* scratch = nullptr;             // device address of the device's static scratch
  gmmh::ErrorTexts err;
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
  if (h) h->err.set(msg);
  return st;
}

}  // namespace gmmh
