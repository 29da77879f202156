// Settings that CUDA keeps for each device, made once per device.
#pragma once

#include <atomic>
#include <cstdint>

namespace tern {

// Calls a setter until it has succeeded for a device; a failure is not kept.
class OncePerDevice {
public:
    // Result of `set` (0: success), or success without a call.  Devices outside
    // [0, 64) are set every time.
    template <typename Set>
    auto operator()(int device, Set&& set) -> decltype(set()) {
        using Status = decltype(set());
        const bool known = device >= 0 && device < 64;
        const uint64_t bit = known ? uint64_t(1) << device : 0;
        if (done_.load(std::memory_order_acquire) & bit) return static_cast<Status>(0);
        const Status status = set();
        if (status == static_cast<Status>(0)) done_.fetch_or(bit, std::memory_order_release);
        return status;
    }

private:
    std::atomic<uint64_t> done_{0};
};

}  // namespace tern
