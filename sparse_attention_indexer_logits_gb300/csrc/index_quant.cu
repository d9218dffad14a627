// The indexer's inputs on sm_103a: q and key rows of 128 rotated, quantised
// to e4m3, the keys written into the fp8 cache with their scales.
//
//   r = rope(x);  s = max(max |r|, 1e-12) / 448;  code = e4m3(r / s)
//
// A q row's scale goes into its head weight (w * s * weight_scale), a key's
// next to it in its page (the s_p of the logits), so the logits are those of
// the unquantised rows up to the codes' rounding (half a step, 2^-4).
//
// Bound by memory: 256 bytes in, 128 out per row.  Eight lanes hold a row,
// sixteen elements each, arranged so that both elements of a pair lie in one
// lane; the row's maximum takes three shuffles.  The maximum is taken over
// the values' bits, which orders infinities above all numbers and NaNs above
// those, so a row with a NaN gets a NaN scale instead of a silent one.  The
// quotient is a product with 448 / max: one rounding more than a division
// (2^-24 against the code's 2^-4), a tenth of its instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "rotary.cuh"
#include "serving.h"

namespace pml {

namespace {

constexpr int kThreads = 256;
constexpr int kRowLanes = 8;                       // lanes of a row
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

template <bool INTER>
__global__ void __launch_bounds__(kThreads) index_quant_kernel(const IndexQuantArgs a)
{
    extern __shared__ float2 cs[];
    __shared__ long long page_of[8];
    __shared__ int slot_of[8];
    __shared__ int state_of[8];    // 0 padding, 1 q only, 2 q and key

    const long long token0 = (long long)blockIdx.x * a.tokens_per_cta;
    const int nt = (int)min((long long)a.tokens_per_cta, (long long)a.tokens - token0);
    const int half = a.rot.half, off8 = a.rot.offset >> 3, half8 = half >> 3;

    fill_turns(a.rot, cs, token0, nt);
    if ((int)threadIdx.x < nt) {
        const int t = threadIdx.x;
        bool pad = false;
        long long page = 0;
        int slot = 0;
        bool ok = false;
        if (a.k != nullptr)
            ok = find_slot(a.slot, token0 + t, load_position(a.rot, token0 + t), pad, page, slot);
        page_of[t] = page;
        slot_of[t] = slot;
        state_of[t] = pad ? 0 : ok ? 2 : 1;
    }
    __syncthreads();

    const int lane = threadIdx.x & (kRowLanes - 1);
    const unsigned mask = 0xffu << (threadIdx.x & 24);
    // the two 8-element chunks of this lane: the halves of eight pairs, or
    // two chunks outside the rotated part, or (interleaved) two neighbours
    int c0 = 2 * lane, c1 = 2 * lane + 1;
    bool turned_pair = false;
    if constexpr (!INTER) {
        if (lane < half8) {
            c0 = off8 + lane;
            c1 = c0 + half8;
            turned_pair = true;
        } else {
            c0 = 2 * (lane - half8);
            c1 = c0 + 1;
            if (c0 >= off8) c0 += 2 * half8;
            if (c1 >= off8) c1 += 2 * half8;
        }
    }
    const int rows_per_token = a.heads + (a.k != nullptr ? 1 : 0);
    for (int r = (int)threadIdx.x / kRowLanes; r < nt * rows_per_token; r += kRows) {
        const int t = r / rows_per_token;
        const int h = r - t * rows_per_token;
        const bool is_k = h == a.heads;
        const int st = state_of[t];
        if (st == 0 || (is_k && st == 1)) continue;     // whole rows together
        const long long tok = token0 + t;
        const __nv_bfloat16* src =
            is_k ? static_cast<const __nv_bfloat16*>(a.k) + tok * a.k_token
                 : static_cast<const __nv_bfloat16*>(a.q) + tok * a.q_token + h * a.q_head;
        const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(src) + c0);
        const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(src) + c1);
        float x[8], y[8];
        unpack8(v0, x);
        unpack8(v1, y);
        const float2* c = cs + t * half;
        if constexpr (INTER) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int ch = (b == 0 ? c0 : c1) - off8;
                if (ch >= 0 && ch < 2 * half8) {
                    float(&z)[8] = b == 0 ? x : y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 w = c[4 * ch + e];
                        const float p = z[2 * e], q = z[2 * e + 1];
                        z[2 * e] = p * w.x - q * w.y;
                        z[2 * e + 1] = q * w.x + p * w.y;
                    }
                }
            }
        } else if (turned_pair) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 w = c[8 * lane + e];
                const float p = x[e], q = y[e];
                x[e] = p * w.x - q * w.y;
                y[e] = q * w.x + p * w.y;
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
            top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
        // as bits: a NaN maximum stays one
        const float amax = __uint_as_float(max(top, __float_as_uint(1e-12f)));
        const float scale = amax / 448.0f;
        const float inv = 448.0f / amax;
        const uint2 p0 = pack_e4m3(x, inv), p1 = pack_e4m3(y, inv);
        uint8_t* dst = is_k ? a.kv_fused + page_of[t] * kFp8BlockBytes + slot_of[t] * kHeadDim
                            : a.q_out + (tok * a.heads + h) * kHeadDim;
        if constexpr (INTER) {
            reinterpret_cast<uint4*>(dst)[lane] = make_uint4(p0.x, p0.y, p1.x, p1.y);
        } else {
            reinterpret_cast<uint2*>(dst)[c0] = p0;
            reinterpret_cast<uint2*>(dst)[c1] = p1;
        }
        if (lane == 0) {
            if (is_k)
                reinterpret_cast<float*>(a.kv_fused + page_of[t] * kFp8BlockBytes +
                                         kFp8BlockKeyBytes)[slot_of[t]] = scale;
            else
                a.w_out[tok * a.heads + h] =
                    __ldg(a.weights + tok * a.heads + h) * scale * a.weight_scale;
        }
    }
}

}  // namespace

cudaError_t launch_index_quant(const IndexQuantArgs& a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((a.tokens + a.tokens_per_cta - 1) / a.tokens_per_cta);
    const size_t smem = (size_t)a.tokens_per_cta * a.rot.half * sizeof(float2);
    if (a.rot.interleaved) index_quant_kernel<true><<<grid, kThreads, smem, stream>>>(a);
    else index_quant_kernel<false><<<grid, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pml
