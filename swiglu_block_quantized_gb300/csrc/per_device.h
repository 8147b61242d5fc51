// per_device.h -- facts that are found out once a device and then read by any thread
// without a lock.  Host code only.
#pragma once
#include <atomic>
#include <mutex>

namespace m4q {

template <typename T, int N>
class PerDevice {
 public:
  // The facts of device `id` in [0, N), after `make(T*)` has succeeded (returned 0) once for
  // it, in `*out`.  A thread that waited while another made them looks again before it makes
  // them itself: once they are known they are never written.  Returns make's error, or 0.
  template <typename F>
  int get(int id, T* out, F make) {
    Slot& k = slots_[id];
    if (!k.known.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!k.known.load(std::memory_order_relaxed)) {
        const int rc = make(&k.facts);
        if (rc != 0) return rc;
        k.known.store(true, std::memory_order_release);
      }
    }
    *out = k.facts;
    return 0;
  }

 private:
  struct Slot {
    std::atomic<bool> known{false};
    T facts{};
  };
  Slot slots_[N];
  std::mutex mu_;
};

}  // namespace m4q
