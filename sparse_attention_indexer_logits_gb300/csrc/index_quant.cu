// The indexer's inputs on sm_103a: q and key rows of 128 rotated, quantised
// to e4m3, the keys written into the fp8 cache with their scales.
//
//   r = rope(x);  s = max(max |r|, 1e-12) / 448;  code = e4m3(r / s)
//
// A q row's scale goes into its head weight (w * s * weight_scale), a key's
// next to it in its page (the s_p of the logits), so the logits are those of
// the unquantised rows up to the codes' rounding (half a step, 2^-4).
//
// Bound by memory: 256 bytes in, 128 out per row.  Four lanes hold a row,
// two units of sixteen elements each, a unit arranged so that both elements
// of a pair lie in it (where half of the row turns, every lane has one unit
// that does and one that does not); a CTA takes a few rows a lane of the
// flattened (token, head) list, a token's key after its heads, loads them
// all, computes its tokens' angles while they are on their way, and works.
// A row's maximum takes two shuffles; it keeps a NaN, so a row with one gets
// a NaN scale instead of a silent one.  The quotient is a product with
// 448 / max, one rounding more than a division (2^-23 against the code's
// 2^-4) and a tenth of its instructions.
//
// Measured (a plain copy reaches 6776 GB/s): 8192 tokens x 65 rows 47.2 us,
// 4.43 TB/s, 65 % of the copy: 256 bytes a lane quad are some 180 instructions
// (issue slots 51 % busy at 24 warps an SM), and the 80 registers that hold
// the rows allow no more warps.  Eight lanes a row took 51.7 us, sixteen 60.1.
// A decode step's 128 tokens: 4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dependent.cuh"
#include "rotary.cuh"
#include "serving.h"

namespace pml {

namespace {

constexpr int kThreads = kQuantThreads;
constexpr int kRowLanes = kQuantLanes;                       // lanes of a row
constexpr int kRows = kThreads / kRowLanes;        // rows of a CTA's step

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Eight values to eight e4m3 codes (round to nearest even, saturating; NaN
// stays NaN).
__device__ __forceinline__ uint2 pack_e4m3(const float (&x)[8], float inv)
{
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t p;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(p)
            : "f"(x[2 * i + 1] * inv), "f"(x[2 * i] * inv));
        h[i] = p;
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool INTER>
__global__ void __launch_bounds__(kThreads, 3) index_quant_kernel(const IndexQuantArgs a)
{
    extern __shared__ __align__(16) float2 cs[];
    __shared__ long long page_of[kQuantMaxTokens];
    __shared__ int slot_of[kQuantMaxTokens];
    __shared__ int state_of[kQuantMaxTokens];    // 0 padding, 1 q only, 2 q and key

    allow_dependent_launch();
    grid_dependency_wait();
    const int half = a.rot.half, off8 = a.rot.offset >> 3, half8 = half >> 3;
    const int rows = a.heads + (a.k != nullptr ? 1 : 0);          // of a token
    const long long row0 = (long long)blockIdx.x * a.rows_per_cta;
    const int count = (int)min((long long)a.rows_per_cta, (long long)a.tokens * rows - row0);
    const long long token0 = row0 / rows;
    const int first = (int)(row0 - token0 * rows);
    const int nt = (first + count - 1) / rows + 1;
    const float per_row = 1.0f / (float)rows;

    const int lane = threadIdx.x & (kRowLanes - 1);
    const unsigned mask = 0xfu << (threadIdx.x & 28);
    // the two 8-element chunks of each of this lane's units, lane and lane +
    // 4: the halves of eight pairs, or two chunks outside the rotated part,
    // or (interleaved) two neighbours
    int c0[2], c1[2];
    bool turn0[2], turn1[2];       // which of the chunks turn
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = lane + kRowLanes * i;
        if (INTER || u >= half8) {
            c0[i] = 2 * (INTER ? u : u - half8);
            c1[i] = c0[i] + 1;
            if (!INTER && c0[i] >= off8) c0[i] += 2 * half8;
            if (!INTER && c1[i] >= off8) c1[i] += 2 * half8;
            turn0[i] = INTER && c0[i] >= off8 && c0[i] < off8 + 2 * half8;
            turn1[i] = INTER && c1[i] >= off8 && c1[i] < off8 + 2 * half8;
        } else {
            c0[i] = off8 + u;
            c1[i] = c0[i] + half8;
            turn0[i] = turn1[i] = true;
        }
    }
    // token of the CTA and row of the token, of this group's next row
    const int i0 = (int)threadIdx.x / kRowLanes;
    const int t0 = (int)(((float)(first + i0) + 0.5f) * per_row);     // (first + i0) / rows: below 2^16
    const int h0 = first + i0 - t0 * rows;
    auto next = [&](int& t, int& h) {
        h += kRows;
        while (h >= rows) { h -= rows; ++t; }
    };
    uint4 v0[kQuantRows][2], v1[kQuantRows][2];
    float weight[kQuantRows];
    {
        int t = t0, h = h0;
#pragma unroll
        for (int b = 0; b < kQuantRows; ++b, next(t, h)) {
            if (i0 + b * kRows >= count) continue;
            const long long tok = token0 + t;
            const __nv_bfloat16* src =
                h == a.heads ? static_cast<const __nv_bfloat16*>(a.k) + tok * a.k_token
                             : static_cast<const __nv_bfloat16*>(a.q) + tok * a.q_token + h * a.q_head;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v0[b][i] = __ldg(reinterpret_cast<const uint4*>(src) + c0[i]);
                v1[b][i] = __ldg(reinterpret_cast<const uint4*>(src) + c1[i]);
            }
            weight[b] = lane == 0 && h < a.heads ? __ldg(a.weights + tok * a.heads + h) : 0.0f;
        }
    }

    fill_turns<INTER ? 4 : 8, INTER>(a.rot, cs, token0, nt);
    // (by the last warp: the first ones have the angles)
    if (const int t = (int)threadIdx.x - (kThreads - 32); t >= 0 && t < nt) {
        bool pad = false;
        long long page = 0;
        int slot = 0;
        bool ok = false;
        if (a.k != nullptr)
            ok = find_slot(a.slot, token0 + t, load_position(a.rot, token0 + t), pad, page, slot);
        else
            pad = load_position(a.rot, token0 + t) < 0;
        page_of[t] = page;
        slot_of[t] = slot;
        state_of[t] = pad ? 0 : ok ? 2 : 1;
    }
    __syncthreads();

    int t = t0, h = h0;
#pragma unroll
    for (int b = 0; b < kQuantRows; ++b, next(t, h)) {
        if (i0 + b * kRows >= count) continue;         // (the lanes of a row together)
        const bool is_k = h == a.heads;
        if (state_of[t] < (is_k ? 2 : 1)) continue;
        float x[2][8], y[2][8];
        const float2* c = cs + t * turn_stride(half);
        // two pairs' angles at a time
        auto turn2 = [](float& p0, float& q0, float& p1, float& q1, float4 w) {
            const float a0 = p0, b0 = q0, a1 = p1, b1 = q1;
            p0 = a0 * w.x - b0 * w.y;
            q0 = b0 * w.x + a0 * w.y;
            p1 = a1 * w.z - b1 * w.w;
            q1 = b1 * w.z + a1 * w.w;
        };
        float amax = 1e-12f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            unpack8(v0[b][i], x[i]);
            unpack8(v1[b][i], y[i]);
            if constexpr (INTER) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    if (turn0[i])
                        turn2(x[i][2 * e], x[i][2 * e + 1], x[i][2 * e + 2], x[i][2 * e + 3],
                              *reinterpret_cast<const float4*>(c + turn_place<4, true>(half, 4 * (c0[i] - off8) + e)));
                    if (turn1[i])
                        turn2(y[i][2 * e], y[i][2 * e + 1], y[i][2 * e + 2], y[i][2 * e + 3],
                              *reinterpret_cast<const float4*>(c + turn_place<4, true>(half, 4 * (c1[i] - off8) + e)));
                }
            } else if (turn0[i]) {
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    turn2(x[i][e], y[i][e], x[i][e + 1], y[i][e + 1],
                          *reinterpret_cast<const float4*>(
                              c + turn_place<8, false>(half, 8 * (lane + kRowLanes * i) + e)));
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = max_nan(amax, max_nan(fabsf(x[i][e]), fabsf(y[i][e])));
        }
#pragma unroll
        for (int o = kRowLanes / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(mask, amax, o));
        // (a quarter of both: the intrinsic gives 0 for divisors past 2^126)
        const float inv = __fdividef(112.0f, 0.25f * amax);
        const float scale = amax * (1.0f / 448.0f);
        uint8_t* dst = is_k ? a.kv_fused + page_of[t] * kFp8BlockBytes + slot_of[t] * kHeadDim
                            : a.q_out + ((token0 + t) * a.heads + h) * kHeadDim;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint2 p0 = pack_e4m3(x[i], inv), p1 = pack_e4m3(y[i], inv);
            if constexpr (INTER) {
                reinterpret_cast<uint4*>(dst)[lane + kRowLanes * i] = make_uint4(p0.x, p0.y, p1.x, p1.y);
            } else {
                reinterpret_cast<uint2*>(dst)[c0[i]] = p0;
                reinterpret_cast<uint2*>(dst)[c1[i]] = p1;
            }
        }
        if (lane == 0) {
            if (is_k)
                reinterpret_cast<float*>(a.kv_fused + page_of[t] * kFp8BlockBytes +
                                         kFp8BlockKeyBytes)[slot_of[t]] = scale;
            else
                a.w_out[(token0 + t) * a.heads + h] = weight[b] * scale * a.weight_scale;
        }
    }
}

}  // namespace

cudaError_t launch_index_quant(const IndexQuantArgs& a, cudaStream_t stream)
{
    const long long rows = (long long)a.tokens * (a.heads + (a.k != nullptr ? 1 : 0));
    const unsigned grid = (unsigned)((rows + a.rows_per_cta - 1) / a.rows_per_cta);
    const size_t smem = (size_t)kQuantMaxTokens * turn_stride(a.rot.half) * sizeof(float2);
    return a.rot.interleaved
               ? launch_dependent(index_quant_kernel<true>, dim3(grid), kThreads, smem, stream, a)
               : launch_dependent(index_quant_kernel<false>, dim3(grid), kThreads, smem, stream, a);
}

}  // namespace pml
