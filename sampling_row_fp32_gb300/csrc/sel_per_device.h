// sel_per_device.h -- what the library asks of the driver once for each device.
// (No CUDA in here: a host program can test it.)
#pragma once

#include <atomic>
#include <cstdint>
#include <mutex>

namespace sel {

// A value of a trivially copyable type for each device ordinal. Only what a
// query that succeeded gave is kept: after a failure the next call asks again.
template <typename V>
class PerDevice {
    static constexpr int kMax = 64;
    std::atomic<uint64_t> known_{0};  // a bit a device
    std::mutex lock_;
    V value_[kMax] = {};

public:
    // query(V&) -> whether it succeeded. Devices past the last ordinal are asked
    // every time. Any number of threads may call this.
    template <typename Query>
    bool get(int device, V& out, Query query) {
        const bool kept = device >= 0 && device < kMax;
        const uint64_t bit = kept ? 1ull << device : 0;
        if (known_.load(std::memory_order_acquire) & bit) {
            out = value_[device];
            return true;
        }
        if (!query(out)) return false;
        if (kept) {
            const std::lock_guard<std::mutex> guard(lock_);
            if (!(known_.load(std::memory_order_relaxed) & bit)) {
                value_[device] = out;
                known_.fetch_or(bit, std::memory_order_release);
            }
        }
        return true;
    }
};

}  // namespace sel
