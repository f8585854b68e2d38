// timeouts.cuh -- how a device-wide count of timeouts is reported, each once.
//
// Kernels on any stream add to the count while a status call reads it, so the
// count is never cleared: a clear ordered behind the read on the caller's stream
// would erase what other streams add in between.  The host remembers up to where
// it has reported instead.  (Plain C++: no CUDA in here.)
#pragma once

#include <atomic>
#include <cstdint>

namespace sqz {

class ReportedTimeouts {
public:
    // Whether `count`, just read from the device, holds timeouts that no call has
    // reported yet; they count as reported from here on.  (A call that read the
    // count earlier than another and comes later reports nothing: the other
    // has.  Differences are signed, so the count may wrap.)
    bool take(uint32_t count) {
        uint32_t upto = upto_.load(std::memory_order_relaxed);
        while ((int32_t)(count - upto) > 0)
            if (upto_.compare_exchange_weak(upto, count, std::memory_order_relaxed)) return true;
        return false;
    }

private:
    std::atomic<uint32_t> upto_{0};
};

}  // namespace sqz
