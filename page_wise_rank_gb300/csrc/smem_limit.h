// How much dynamic shared memory a kernel has been allowed, per device (host code).
#pragma once
#include <atomic>
#include <mutex>

namespace pkv {

// The largest value that has been set for each device, beside a setter with no
// memory of its own (the driver keeps whatever it was given last).  Threads
// that ask for different sizes set them one after another, so that the value in
// force is never below the one recorded here.
class SmemLimit {
  public:
    static constexpr int kDevices = 64;
    // Calls set(bytes) if less than that was set before; 0 is its success.
    template <typename Set>
    int raise(int dev, int bytes, Set set) {
        if (allowed_[dev].load(std::memory_order_acquire) >= bytes) return 0;
        std::lock_guard<std::mutex> lock(mu_);
        if (allowed_[dev].load(std::memory_order_relaxed) >= bytes) return 0;
        const int e = set(bytes);
        if (e == 0) allowed_[dev].store(bytes, std::memory_order_release);
        return e;
    }

  private:
    std::mutex mu_;
    std::atomic<int> allowed_[kDevices] = {};
};

}  // namespace pkv
