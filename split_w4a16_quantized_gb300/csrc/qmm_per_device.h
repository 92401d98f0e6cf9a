// A value made once per device: a kernel's shared-memory opt-in and the address of
// a __device__ variable belong to the device that was current when they were asked
// for.  Host code without CUDA, so that it compiles alone.
#pragma once

#include <mutex>

namespace qmm {

template <class T>
class PerDevice {
public:
    // make()'s result for `device`; make runs once for each of the first 64.
    template <class F>
    T get(int device, F&& make) {
        if (device < 0 || device >= kDevices) return make();
        std::call_once(once_[device], [&] { value_[device] = make(); });
        return value_[device];
    }

private:
    static constexpr int kDevices = 64;
    std::once_flag once_[kDevices];
    T value_[kDevices] = {};
};

}  // namespace qmm
