// Something that is set once a device (a kernel's attribute), by whichever
// call comes first.
#pragma once

#include <stdint.h>

#include <atomic>

namespace moeq {

// `done`: devices 0 .. 127 on which it has been set; on a device beyond, and
// after a failure, it is set again each time.
struct OncePerDevice {
    std::atomic<uint64_t> done[2]{};
    template <typename Set>
    auto on(int dev, Set set) -> decltype(set()) {
        const bool known = dev >= 0 && dev < 128;
        const uint64_t bit = uint64_t(1) << (dev & 63);
        if (known && (done[dev >> 6].load(std::memory_order_acquire) & bit)) return {};
        using E = decltype(set());
        const E e = set();
        if (e == E{} && known) done[dev >> 6].fetch_or(bit, std::memory_order_release);
        return e;
    }
};

}  // namespace moeq
