// What is set up once for each device of a process.  Plain C++, so that it can be
// tested without a GPU.
#pragma once
#include <atomic>
#include <mutex>

class PerDevice {
 public:
  // Calls set_up() the first time that it is asked for on `device`, and again after a
  // failure; returns what it returned (0: success).
  template <class F>
  auto operator()(int device, F &&set_up) -> decltype(set_up()) {
    using E = decltype(set_up());
    if (device < 0 || device >= kDevices) return set_up();
    if (done_[device].load(std::memory_order_acquire)) return E(0);
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[device].load(std::memory_order_relaxed)) return E(0);
    const E e = set_up();
    if (e == E(0)) done_[device].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::mutex mu_;
  std::atomic<bool> done_[kDevices] = {};
};
