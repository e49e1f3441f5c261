// wq_once.h -- host-side work that is to be done once per device, as setting a kernel's attributes is.
#pragma once
#include <stdint.h>

#include <atomic>

namespace wq {

// Runs set() (true: it worked) unless it worked on this device before.  A failure is not remembered: the next call tries
// again.  Devices from 64 on are not remembered either.  Two threads may both run set().
template <class Set>
inline bool once_per_device(std::atomic<uint64_t>& done, int device, Set&& set) {
  const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (!set()) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

}  // namespace wq
