// Preparations that are made once for each device and kept (plain C++, so that a test can fail them).
#pragma once
#include <atomic>
#include <cstdint>
#include <mutex>

namespace sdv2 {

class PerDevice {
public:
    // Runs `prepare`, whose status 0 means success, until it has succeeded once for `device`; a failure is returned
    // and tried again by the next call.  What it wrote is visible to every thread that was told of success.
    template <typename F>
    auto run(int device, F&& prepare) -> decltype(prepare())
    {
        const uint64_t bit = uint64_t(1) << (device & 63);
        if (done_.load(std::memory_order_acquire) & bit) return {};
        std::lock_guard<std::mutex> lock(one_);
        if (done_.load(std::memory_order_relaxed) & bit) return {};
        const auto status = prepare();
        if (status == decltype(prepare()){}) done_.fetch_or(bit, std::memory_order_release);
        return status;
    }

private:
    std::atomic<uint64_t> done_{0};
    std::mutex one_;
};

}  // namespace sdv2
