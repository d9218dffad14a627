// How work over caches held in 4 bits is counted and shared out, for tests on the
// CPU.
#include "common.cuh"
#include "nvfp4_cache.h"

using namespace pml;

extern "C" int blocks(int len) { return blocks_of(len); }
