// What each kernel's dynamic shared memory limit has been set to, by device.
// Host code only, without CUDA: the caller passes the setter.
#pragma once

#include <stddef.h>

#include <mutex>

namespace sd {

// The limit is an attribute that outlives the call, and setting it on every
// launch costs host time on the decode loop, so it is set where it has to
// grow. It never shrinks: another thread may have raised it and not launched yet.
class SmemLimits {
 public:
  static constexpr int kDevices = 64, kKernels = 128;  // the library has some 50 kernels that need it
  static constexpr int kNoRoom = -1;

  // set(bytes) -> 0 or an error, called under the lock where `bytes` is above
  // what the kernel has. Returns its error, or kNoRoom without having called it.
  template <class Set>
  int raise(const void* kern, int dev, size_t bytes, Set set) {
    if (dev < 0 || dev >= kDevices) return kNoRoom;
    std::lock_guard<std::mutex> lock(mu_);
    Entry* e = done_[dev];
    int i = 0;
    while (i < n_[dev] && e[i].kern != kern) ++i;
    if (i == kKernels) return kNoRoom;
    if (i < n_[dev] && e[i].bytes >= bytes) return 0;
    const int err = set(bytes);
    if (err != 0) return err;
    e[i] = Entry{kern, bytes};
    if (i == n_[dev]) ++n_[dev];
    return 0;
  }

 private:
  struct Entry { const void* kern; size_t bytes; };
  std::mutex mu_;
  Entry done_[kDevices][kKernels];
  int n_[kDevices] = {};
};

}  // namespace sd
