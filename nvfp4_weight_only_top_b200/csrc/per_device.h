// A number that each device is asked for once.  Host code only.
#pragma once

#include <atomic>

namespace moe {

// get(dev, query): query()'s answer for device dev, kept once it is above 0 (a query that fails answers 0 and is made
// again the next time).  Devices past the table's end are asked every time.  Static objects; any thread.
struct PerDevice {
  static constexpr int kDevices = 64;
  std::atomic<int> n[kDevices] = {};                    // 0: not known
  template <typename Query>
  int get(int dev, Query query) {
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept) {
      const int known = n[dev].load(std::memory_order_relaxed);
      if (known > 0) return known;
    }
    const int v = query();
    if (kept && v > 0) n[dev].store(v, std::memory_order_relaxed);
    return v;
  }
};

}  // namespace moe
