// A number that depends on the device only, asked for once per device (host code).
#pragma once

#include <atomic>

namespace ssd {

class PerDevice {
  public:
    // ask(dev), kept from the first time that it is positive; `otherwise`, which is not kept, until then.
    // Threads may ask at the same time.  (Devices from kDevices on are asked every time.)
    template <typename F> int get(int dev, int otherwise, F ask) {
        const bool keep = dev >= 0 && dev < kDevices;
        int n = keep ? known_[dev].load(std::memory_order_relaxed) : 0;
        if (n > 0) return n;
        n = dev >= 0 ? ask(dev) : 0;
        if (n <= 0) return otherwise;
        if (keep) known_[dev].store(n, std::memory_order_relaxed);
        return n;
    }

  private:
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices]{};
};

}  // namespace ssd
