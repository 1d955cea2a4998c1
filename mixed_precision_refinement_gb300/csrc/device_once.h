// What has to be set once on each device of a process.  Host code without CUDA.
#pragma once

#include <atomic>
#include <cstdint>

namespace zs {

class OncePerDevice {
  public:
    // set() on the first call for device `dev` and again after every call that failed (a
    // result other than its type's zero); its result, or zero.  Threads may meet here: both
    // then call it.
    template <typename F>
    auto run(int dev, F set) -> decltype(set()) {
        using R = decltype(set());
        const bool known = dev >= 0 && dev < kDevices;
        const uint64_t bit = known ? uint64_t(1) << dev % 64 : 0;
        if (known && (done_[dev / 64].load(std::memory_order_acquire) & bit)) return R{};
        const R r = set();
        if (r == R{} && known) done_[dev / 64].fetch_or(bit, std::memory_order_release);
        return r;
    }

  private:
    static constexpr int kDevices = 256;  // of those beyond, every call sets it
    std::atomic<uint64_t> done_[kDevices / 64] = {};
};

}  // namespace zs
