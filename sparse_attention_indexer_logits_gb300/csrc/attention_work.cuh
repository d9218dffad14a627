// How attention's work is counted and cut: the tiles that a request's tokens
// look at, and the units that the CTAs' ranges share out.  (Plain arithmetic,
// also compiled for the host.)
#pragma once

#include "common.cuh"
#include "serving.h"

namespace pml {
namespace attn {

// The tokens and tiles of tile `tile` of a request with nq new tokens of kv.
struct Span {
    int t0, ntok;    // tokens of the request
    int lo, hi;      // keys that some row of the tile may see
    int j0, n;       // their tiles of 128 keys; at least one
    int cost;        // units of a tile
};

__host__ __device__ __forceinline__ Span tile_span(const AttnArgs& a, int nq, int kv, int tile)
{
    Span s;
    const int per = 2 * a.half_tokens;
    s.t0 = tile * per;
    s.ntok = min(per, nq - s.t0);
    const int there = (int)min((long long)kv, (long long)a.bt_width * kBlockKeys);
    const long long pos0 = (long long)kv - nq + s.t0;      // position of the tile's first token
    long long hi = there;
    if (a.causal) hi = min(hi, pos0 + s.ntok);
    long long lo = 0;
    if (a.window > 0) lo = max(lo, pos0 - a.window + 1);
    if (hi <= lo) { hi = 0; lo = 0; }
    s.lo = (int)lo;
    s.hi = (int)hi;
    s.j0 = s.lo / kAttnTileKeys;
    s.n = s.hi > 0 ? (s.hi - 1) / kAttnTileKeys + 1 - s.j0 : 1;     // (hi + 127 may pass an int)
    s.cost = s.ntok <= a.half_tokens ? 1 : 2;
    return s;
}

__host__ __device__ __forceinline__ int tiles_of(const AttnArgs& a, int nq)
{
    const int per = 2 * a.half_tokens;
    return (nq + per - 1) / per;
}

// Units of work.  A tile is one where the halves take the tiles in turn and two
// where both see it (1800 and 3600 cycles), and beginning and ending an item
// (Q's way in, the first copies, the output) is three.  A mixed batch of 24
// requests takes 54.9 us, with two, four or six units an item 58.0, 55.1 or
// 55.6; 64 tokens of 2048 listed positions 29.2 us, with two, four or six 29.2,
// 31.8 or 32.7.  A range has the tiles whose first unit lies in it.
constexpr int kItemUnits = 3;

__host__ __device__ __forceinline__ int units_of(const Span& s) { return s.n * s.cost + kItemUnits; }
__host__ __device__ __forceinline__ int tiles_before(const Span& s, int unit)
{
    const int u = max(0, unit - kItemUnits);
    return s.cost == 1 ? u : (u + 1) >> 1;
}

// Units of all of a request's tiles: 2^31 and more for a million tokens over
// as many keys.
__host__ __device__ __forceinline__ long long units_of_request(const AttnArgs& a, int nq, int kv)
{
    const int tiles = tiles_of(a, nq);
    long long units = 0;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) units += units_of(tile_span(a, nq, kv, i));
    return units;
}

}  // namespace attn
}  // namespace pml
