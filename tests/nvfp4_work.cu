// How work over caches held in 4 bits is counted and shared out, for tests on the
// CPU.
#include "common.cuh"
#include "nvfp4_cache.h"

using namespace pml;

extern "C" int blocks(int len) { return blocks_of(len); }

extern "C" long long items(long long tokens, long long batch, int group, int rows)
{
    return nvfp4_items(tokens, batch, group, rows);
}

extern "C" int large_items(long long tokens, long long batch, int group) { return nvfp4_large_items(tokens, batch, group); }

extern "C" int by_tiles(long long tokens, long long batch, int num_heads, int group)
{
    return nvfp4_by_tiles(tokens, batch, num_heads, group);
}

extern "C" int lists_by_tiles(long long tokens, int num_heads, int group, int k, int num_ctas)
{
    return nvfp4_lists_by_tiles(tokens, num_heads, group, k, num_ctas);
}
