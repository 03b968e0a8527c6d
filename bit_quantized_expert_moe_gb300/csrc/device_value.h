// A number that belongs to a device, looked up once for each.
#pragma once

#include <atomic>

namespace moe {

class DeviceValue {
    static constexpr int DEVICES = 64;
    std::atomic<int> of_[DEVICES] = {};  // 0: not looked up yet

public:
    // The number of device `dev`; find() returns it, or one below 1 where it cannot be
    // had now.  Threads that call together may look it up twice, to the same end.
    template <class F>
    int get(int dev, F find) {
        if (dev < 0 || dev >= DEVICES) return find();
        int v = of_[dev].load(std::memory_order_relaxed);
        if (v < 1) {
            v = find();
            if (v >= 1) of_[dev].store(v, std::memory_order_relaxed);
        }
        return v;
    }
};

}  // namespace moe
