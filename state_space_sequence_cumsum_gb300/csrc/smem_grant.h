// Dynamic shared memory beyond what a kernel may take by default, asked for
// per kernel and device (no CUDA headers: the order of the steps is tested on
// the host).
#pragma once
#include <atomic>
#include <cstddef>
#include <mutex>

namespace ssd {

constexpr int kSmemDevices = 64;

// What a kernel has been given, per device; one static object per kernel.
struct SmemGrant {
    std::atomic<int> bytes[kSmemDevices];
    std::mutex mu;
};

// set(bytes) puts the kernel's limit on device `dev` at `bytes` and returns 0
// or an error, which is passed on.  The limit replaces the one before it, so
// it is set and noted under a lock and only ever raised: a call that found its
// bytes granted may launch while others ask for less or more.  (Past
// kSmemDevices devices nothing is noted and every call sets its own.)
template <typename Set> auto raise_smem(SmemGrant &g, int dev, size_t bytes, Set set) -> decltype(set(0))
{
    if (dev >= kSmemDevices)
        return set((int)bytes);
    if (g.bytes[dev].load(std::memory_order_acquire) >= (int)bytes)
        return {};
    std::lock_guard<std::mutex> lk(g.mu);
    if (g.bytes[dev].load(std::memory_order_relaxed) >= (int)bytes)
        return {};
    const auto e = set((int)bytes);
    if (!e)
        g.bytes[dev].store((int)bytes, std::memory_order_release);
    return e;
}

}  // namespace ssd
