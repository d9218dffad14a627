// Counts of clusters asked for by several threads at once.
#include <atomic>
#include <initializer_list>
#include <thread>

#include "cluster_counts.h"

static pml::ClusterCounts counts;

// What `ask` says of a size on a device.
static int said(int device, int size) { return 1000 * device + size; }

// Thread 0 asks first and is in the middle of it when thread 1 asks for `size` on
// `device`: out[0] and out[1] are what they get, out[2] what a later call gets,
// out[3] how often that asked.
extern "C" void two_first_calls(int device, int size, int* out)
{
    std::atomic<bool> entered{false}, go{false};
    std::thread first([&] {
        out[0] = counts.get(0, 8, [&](int s) {
            entered = true;
            while (!go) std::this_thread::yield();
            return said(0, s);
        });
    });
    while (!entered) std::this_thread::yield();
    std::thread second([&] { out[1] = counts.get(device, size, [&](int s) { return said(device, s); }); });
    second.join();
    go = true;
    first.join();
    out[3] = 0;
    out[2] = counts.get(device, size, [&](int) { return ++out[3]; });
}

// Devices in turn, and one that a table has no place for: each its own.
extern "C" int in_turn()
{
    for (int round = 0; round < 3; ++round)
        for (int device : {1, 2, 63, 64, 1000})
            for (int size : {2, 4, 8})
                if (counts.get(device, size, [&](int s) { return said(device, s); }) != said(device, size)) return 0;
    return 1;
}

// A device that runs none is asked once.
extern "C" int none(int* asked)
{
    *asked = 0;
    int n = 0;
    for (int i = 0; i < 3; ++i) n += counts.get(5, 4, [&](int) { ++*asked; return 0; });
    return n;
}
