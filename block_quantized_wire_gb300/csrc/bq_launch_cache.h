// What a launch needs to know of a kernel, remembered: how many CTAs an SM holds. And the
// kernels' dynamic shared memory limits, which only ever rise.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

namespace bqk {

// Rt answers for the current device: limit(kernel, &bytes), raise_limit(kernel, bytes) and
// ctas_per_sm(kernel, block, smem, &ctas), each 0 or an error.
template <class Rt>
class LaunchCache {
public:
    // CTAs of `block` threads and `smem` bytes of dynamic shared memory that an SM of the
    // current device (number `device`) holds, at least 1. Afterwards the kernel may be launched
    // with `smem` bytes, and stays so: a limit is read back from the runtime before it is
    // raised, so that neither a call with less nor an entry that has been replaced lowers it
    // under another thread's launch.
    int ctas_per_sm(Rt &rt, const void *kernel, size_t smem, int block, int device, int *ctas)
    {
        std::lock_guard<std::mutex> lock(mu_);
        const Entry want = {kernel, smem, block, device, 0};
        const size_t home = hash(want);
        size_t at = kWays;
        for (size_t i = 0; i < kWays; i++) {
            const Entry &e = entries_[(home + i) % kEntries];
            if (e.ctas == 0) {
                at = i;
                break;
            }
            if (e.kernel == kernel && e.smem == smem && e.block == block && e.device == device) {
                *ctas = e.ctas;
                return 0;
            }
        }
        size_t limit = 0;
        if (int err = rt.limit(kernel, &limit)) return err;
        if (smem > limit)
            if (int err = rt.raise_limit(kernel, smem)) return err;
        if (int err = rt.ctas_per_sm(kernel, block, smem, ctas)) return err;
        if (*ctas < 1) *ctas = 1;
        if (at == kWays) at = next_++ % kWays;  // all taken: one of them goes
        Entry &slot = entries_[(home + at) % kEntries];
        slot = want;
        slot.ctas = *ctas;
        return 0;
    }

private:
    static constexpr size_t kEntries = 1024, kWays = 8;
    struct Entry {
        const void *kernel;
        size_t smem;
        int block, device;
        int ctas;  // 0: free
    };
    static size_t hash(const Entry &e)
    {
        uint64_t h = reinterpret_cast<uintptr_t>(e.kernel);
        for (uint64_t v : {(uint64_t)e.smem, (uint64_t)e.block, (uint64_t)e.device})
            h = (h ^ (h >> 29) ^ v) * 0x9e3779b97f4a7c15ull;
        return static_cast<size_t>(h >> 40) % kEntries;
    }
    std::mutex mu_;
    Entry entries_[kEntries] = {};
    size_t next_ = 0;
};

}  // namespace bqk
