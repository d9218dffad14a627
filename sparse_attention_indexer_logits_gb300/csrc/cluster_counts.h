// How many clusters of a size a device runs at a time, looked up once for each.
#pragma once

#include <atomic>

namespace pml {

// Calls come from several threads and for several devices at once.  Each count is
// one word that is written whole, so that it is known or not: a thread that does
// not find it asks for itself, and gets what the others get.
class ClusterCounts {
public:
    static constexpr int kDevices = 64, kMaxSize = 8;

    // Of clusters of `size` CTAs, a power of two up to kMaxSize; ask(size) says it.
    template <class Ask>
    int get(int device, int size, Ask ask)
    {
        if (device < 0 || device >= kDevices) return ask(size);
        std::atomic<int>& known = plus_one_[device][size];
        int n = known.load(std::memory_order_relaxed);
        if (n == 0) {
            n = ask(size) + 1;
            known.store(n, std::memory_order_relaxed);
        }
        return n - 1;
    }

private:
    std::atomic<int> plus_one_[kDevices][kMaxSize + 1] = {};    // 0: not asked yet
};

}  // namespace pml
