// What each device answers to a question about a kernel (how many of its blocks
// or clusters it holds).  Host code only, without CUDA.
#pragma once

#include <atomic>

namespace fibatt {

// The answer is asked for once a device and kept; 0 stands for "not asked yet", so
// no answer is 0.  What `ask` sets on the way (a kernel's attributes belong to the
// device that is current) is thereby set on every device before its first answer is
// used.  A device that could not be told (dev < 0), or one beyond those kept, is
// asked each time.  Calls of several threads may ask twice.
class PerDevice {
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices] = {};

public:
    template <typename Ask>
    int get(int dev, Ask ask) {
        if (dev < 0 || dev >= kDevices) return ask();
        int answer = known_[dev].load(std::memory_order_acquire);
        if (answer) return answer;
        answer = ask();
        known_[dev].store(answer, std::memory_order_release);
        return answer;
    }
};

}  // namespace fibatt
