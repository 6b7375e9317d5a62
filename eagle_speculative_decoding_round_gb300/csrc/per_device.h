// per_device.h -- host state that belongs to a device, not to the process: kernel attributes
// (set on the device that is current) and what a device answers about itself.
#pragma once
#include <stdint.h>

#include <atomic>

namespace e3 {

constexpr int kMaxDevices = 64;  // (a device beyond them is asked every time)

// Runs f once on each device; a run that fails is not remembered.  E(0) means success.  f may
// run on two threads at the same time, so it has to be a thing that can be done twice.
template <typename E>
class OncePerDevice {
 public:
  template <typename F>
  E run(int device, F&& f) {
    const bool held = device >= 0 && device < kMaxDevices;
    const uint64_t bit = held ? uint64_t{1} << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return static_cast<E>(0);
    const E e = f();
    if (e == static_cast<E>(0) && held) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// A positive number that each device answers by itself; 0 (no answer) is not remembered.
class NumberPerDevice {
 public:
  template <typename F>
  int get(int device, F&& f) {
    const bool held = device >= 0 && device < kMaxDevices;
    int n = held ? known_[device].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    n = f();
    if (n > 0 && held) known_[device].store(n, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<int> known_[kMaxDevices] = {};
};

}  // namespace e3
