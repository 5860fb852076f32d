// lm_device_once.h -- work done once for each device, by whichever thread comes first.
#pragma once

#include <atomic>

namespace lm {

constexpr int kMaxDevices = 64;

// Remembers for which devices `set` has succeeded.  Two threads that come first together may
// both call it, so it has to be one that can be called again; nobody returns true before a
// call of it has.
class DeviceOnce {
public:
    template <typename F>
    bool run(int device, F set) {
        if (device < 0 || device >= kMaxDevices) return false;
        if (done_[device].load(std::memory_order_acquire)) return true;
        if (!set()) return false;
        done_[device].store(true, std::memory_order_release);
        return true;
    }

private:
    std::atomic<bool> done_[kMaxDevices] = {};
};

}  // namespace lm
