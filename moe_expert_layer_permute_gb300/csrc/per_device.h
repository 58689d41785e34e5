// per_device.h - what a launch has to set or ask once for each GPU of the process (function attributes, resident
// blocks); plain C++, checked on the host (tests/test_per_device.py).
#pragma once
#include <mutex>

namespace moe {

template <typename V>
class PerDevice {
public:
    // `out` from `make(&value)` on `device`'s first call; an error that it returns is not kept, so that the next call
    // tries again.
    template <typename Make>
    auto get(int device, V* out, Make make) -> decltype(make(out)) {
        using Err = decltype(make(out));
        if (device < 0 || device >= kMost) return make(out);
        std::lock_guard<std::mutex> lock(mutex_);
        if (!have_[device]) {
            const Err err = make(value_ + device);
            if (err != Err(0)) return err;
            have_[device] = true;
        }
        *out = value_[device];
        return Err(0);
    }

private:
    static constexpr int kMost = 64;
    std::mutex mutex_;
    bool have_[kMost] = {};
    V value_[kMost] = {};
};

}  // namespace moe
