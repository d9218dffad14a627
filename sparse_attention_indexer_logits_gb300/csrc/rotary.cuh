// Rotary angles, shared by the kernels that rotate.
//
// The angle of pair j at position p is p * inv_freq[j].  In 32 bits that
// product loses everything at far positions (an ulp of 10^6 radians is 0.06),
// and 64-bit floating point is slow on this GPU, so the angle is kept as a
// 64-bit fixed-point fraction of a turn: step = inv_freq / 2 pi * 2^64, once
// per frequency, and step * p mod 2^64 is the exact fraction of a turn that
// step stands for, whatever p is (negative ones too).  Its top 32 bits, read
// as a signed number, are the turn in [-1/2, 1/2): sincospif takes twice that
// with no reduction left to do.  The error is that of step, 2^-53 of
// inv_freq, times p, plus the rounding of the turn to a float, at most 2^-26
// of a turn (1e-7 radians).
#pragma once

#include <stdint.h>

#include "serving.h"

namespace pml {

// mantissa * 2^exponent / 2 pi * 2^64, modulo 2^64, mantissa below 2^53.
__device__ __forceinline__ uint64_t turn_step(uint64_t mantissa, int exponent, bool negative)
{
    // 2^66 / 2 pi: the top 64 bits of the constant
    constexpr uint64_t kInvTwoPi = 0xa2f9836e4e44152aull;
    const uint64_t hi = __umul64hi(mantissa << 11, kInvTwoPi);   // m * 2^11 * c / 2^64
    const uint64_t lo = (mantissa << 11) * kInvTwoPi;
    const int s = exponent + 51;
    uint64_t step;
    if (s <= -64 || s >= 128) step = 0;
    else if (s < 0) step = hi >> -s;
    else if (s == 0) step = hi;
    else if (s < 64) step = (hi << s) | (lo >> (64 - s));
    else step = lo << (s - 64);
    return negative ? 0ull - step : step;
}

__device__ __forceinline__ uint64_t load_step(const RotaryArgs& r, int j)
{
    if (r.freq64) {
        const uint64_t b = __ldg(static_cast<const unsigned long long*>(r.inv_freq) + j);
        const int e = (int)(b >> 52) & 0x7ff;
        const uint64_t m = b & 0xfffffffffffffull;
        return e == 0 || e == 0x7ff ? 0 : turn_step(m | (1ull << 52), e - 1075, b >> 63);
    }
    const uint32_t b = __ldg(static_cast<const uint32_t*>(r.inv_freq) + j);
    const int e = (int)(b >> 23) & 0xff;
    const uint64_t m = b & 0x7fffffu;
    // the mantissa as a 53-bit one
    return e == 0 || e == 0xff ? 0 : turn_step((m | (1u << 23)) << 29, e - 150 - 29, b >> 31);
}

__device__ __forceinline__ long long load_position(const RotaryArgs& r, long long t)
{
    return r.pos64 ? __ldg(static_cast<const long long*>(r.positions) + t)
                   : (long long)__ldg(static_cast<const int32_t*>(r.positions) + t);
}

// (cosine, sine) of `step` at `position`, times mscale, the sine's sign set.
__device__ __forceinline__ float2 turned(uint64_t step, long long position, float mscale, float sign)
{
    const uint64_t phase = step * (uint64_t)position;
    const float turn2 = (float)(int32_t)(phase >> 32) * 0x1p-31f;
    float s, c;
    sincospif(turn2, &s, &c);
    return make_float2(c * mscale, s * mscale * sign);
}

// Where pair j lies in a token's part of the table below.  Neighbouring
// threads take neighbouring runs of `run` pairs and read them two at a time:
// the first two of every run, then the next two, so that these reads are
// contiguous.  With kTwin a thread takes two runs, whose first ones precede
// the second ones.
template <int kRun, bool kTwin>
__device__ __forceinline__ int turn_place(int half, int j)
{
    if constexpr (kRun < 2) {
        return j;
    } else {
        const int run = j / kRun, k = j % kRun;
        if constexpr (!kTwin) return 2 * ((k >> 1) * (half / kRun) + run) + (k & 1);
        const int runs = (half / kRun + 1) >> 1;
        return 2 * (((run & 1) * (kRun / 2) + (k >> 1)) * runs + (run >> 1)) + (k & 1);
    }
}

// Values of a token in the table: room for an odd run out, and an even number.
__host__ __device__ __forceinline__ int turn_stride(int half) { return (half + 5) & ~1; }

// Fills cs[t * turn_stride(half) + turn_place(j)] for the CTA's tokens; every
// thread of the CTA calls.
template <int kRun, bool kTwin>
__device__ __forceinline__ void fill_turns(const RotaryArgs& r, float2* cs, long long token0,
                                           int tokens)
{
    const int half = r.half;
    if (half == 0) return;
    // thread = (pair, token lane): one step per thread while pairs <= threads
    const int lanes = max(1, (int)blockDim.x / half);
    const int g = (int)threadIdx.x / half;
    if (g < lanes && g < tokens) {
        // (both loads on their way before either is used)
        const long long first = load_position(r, token0 + g);
        for (int j = (int)threadIdx.x - g * half; j < half; j += blockDim.x) {
            const uint64_t step = load_step(r, j);
            const int at = turn_place<kRun, kTwin>(half, j);
            for (int t = g; t < tokens; t += lanes)
                cs[t * turn_stride(half) + at] =
                    turned(step, t == g ? first : load_position(r, token0 + t), r.mscale, r.sign);
        }
    }
}

// A token's page and slot, found by one thread; false: nothing is written.
__device__ __forceinline__ bool find_slot(const SlotArgs& s, long long token, long long position,
                                          bool& padding, long long& page, int& slot)
{
    const int req = __ldg(s.requests + token);
    padding = req < 0 || position < 0;
    page = 0;
    slot = 0;
    if (padding) return false;
    if (req >= s.num_requests) {
        atomicOr(s.status, 4u);   // PML_STATUS_BAD_REQUEST
        return false;
    }
    const long long col = position >> 6;
    if (col >= s.bt_width) {
        atomicOr(s.status, 2u);   // PML_STATUS_BAD_BLOCK
        return false;
    }
    page = __ldg(s.block_table + (long long)req * s.bt_stride + col);
    slot = (int)(position & 63);
    if (page < 0 || page >= s.num_pages) {
        atomicOr(s.status, 2u);
        return false;
    }
    return true;
}

}  // namespace pml
