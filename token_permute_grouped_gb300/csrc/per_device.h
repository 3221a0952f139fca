// What a launch needs to know of the device it runs on (SMs, clusters resident
// at once), asked for once a device.
#pragma once

#include <atomic>
#include <mutex>

namespace a2av {

template <typename T>
class PerDevice {
public:
    // The value of device `dev`, or nullptr where query(T &) says that it failed
    // (the next call asks again).  Threads that come at once wait for the first.
    template <typename Query>
    const T *get(int dev, Query query) {
        if (dev < 0 || dev >= kDevices) return nullptr;
        Entry &e = entries_[dev];
        if (!e.ready.load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> lock(mutex_);
            if (!e.ready.load(std::memory_order_relaxed)) {
                if (!query(e.value)) return nullptr;
                e.ready.store(true, std::memory_order_release);
            }
        }
        return &e.value;
    }

private:
    static constexpr int kDevices = 64;
    struct Entry {
        std::atomic<bool> ready{false};
        T value{};
    };
    Entry entries_[kDevices];
    std::mutex mutex_;
};

}  // namespace a2av
