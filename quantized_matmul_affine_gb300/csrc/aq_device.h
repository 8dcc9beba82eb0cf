// What is done or asked once on every device a process uses.
#pragma once

#include <stdint.h>

#include <atomic>

namespace aq {

// An answer a device: ask() is called for a device until it has answered, and
// the answer kept for that device alone.  (Two threads may ask at once; both get
// the same answer.)  Devices past 63 are asked every time.
class PerDevice {
    std::atomic<uint64_t> asked_{0}, yes_{0};

public:
    template <class Ask>
    bool operator()(int device, Ask ask) {
        const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0u;
        if (asked_.load(std::memory_order_acquire) & bit) return yes_.load(std::memory_order_relaxed) & bit;
        const bool yes = ask();
        if (yes) yes_.fetch_or(bit, std::memory_order_relaxed);
        asked_.fetch_or(bit, std::memory_order_release);
        return yes;
    }
};

}  // namespace aq
