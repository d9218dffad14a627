// The arithmetic of csrc/attention_work.cuh for tests on the CPU.
#include "attention_work.cuh"

using namespace pml;
using namespace pml::attn;

static AttnArgs args(int group, int bt_width, int causal, int window)
{
    AttnArgs a = {};
    a.half_tokens = kAttnHalfRows / group;
    a.bt_width = bt_width;
    a.causal = causal;
    a.window = window;
    return a;
}

extern "C" long long request_units(int group, int bt_width, int causal, int window, int nq, int kv)
{
    return units_of_request(args(group, bt_width, causal, window), nq, kv);
}

extern "C" int request_tiles(int group, int nq) { return tiles_of(args(group, 1, 0, 0), nq); }

extern "C" void span(int group, int bt_width, int causal, int window, int nq, int kv, int tile, int* out)
{
    const Span s = tile_span(args(group, bt_width, causal, window), nq, kv, tile);
    const int v[7] = {s.t0, s.ntok, s.lo, s.hi, s.j0, s.n, s.cost};
    for (int i = 0; i < 7; ++i) out[i] = v[i];
}

extern "C" int item_units(int n, int cost)
{
    Span s = {};
    s.n = n;
    s.cost = cost;
    return units_of(s);
}

extern "C" int before(int n, int cost, int unit)
{
    Span s = {};
    s.n = n;
    s.cost = cost;
    return tiles_before(s, unit);
}
