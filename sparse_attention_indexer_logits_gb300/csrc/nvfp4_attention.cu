// Attention of new tokens over K/V caches held in 4 bits.
//
//   out[t, h] = sum_p softmax_p(scale * q[t, h] . k_p) v_p
//
// over values code * s * g (codes E2M1, s the E4M3 scale of sixteen values, g
// the cache's power of two) and the positions p that token t may see.  One CTA
// per (token, head): each warp takes every fourth key, a lane the same few
// elements of each row, with a running maximum and sum; the warps' results are
// joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dependent.cuh"
#include "nvfp4_cache.h"
#include "ptx.cuh"

namespace pml {

namespace {

constexpr int kWarps = 4;

template <bool FP16>
__device__ __forceinline__ float load16(const void* p, long long at)
{
    if constexpr (FP16) return __half2float(static_cast<const __half*>(p)[at]);
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kWarps * 32) nvfp4_attention_kernel(const NvAttnArgs a)
{
    constexpr int E = D / 32;              // elements of a lane
    __shared__ float part[kWarps][D + 2];
    allow_dependent_launch();
    grid_dependency_wait();
    const long long t = blockIdx.x;
    const int head = blockIdx.y, kvh = head / a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int req, kv, lo = 0, hi;
    if (a.selected) {
        req = __ldg(a.requests + t);
        if (req >= a.batch && threadIdx.x == 0) atomicOr(a.status, kStatusBadRequest);
        const bool fine = req >= 0 && req < a.batch;
        kv = fine ? max(__ldg(a.kv_lens + req), 0) : 0;
        req = fine ? req : 0;
        hi = a.sel_k;
    } else {
        int start, end;
        if (a.cu_q) {
            int l = 0, r = a.batch;        // the last request that begins at or before t
            while (r - l > 1) {
                const int m = (l + r) >> 1;
                if (__ldg(a.cu_q + m) <= t) l = m;
                else r = m;
            }
            req = l;
            start = __ldg(a.cu_q + l);
            end = __ldg(a.cu_q + l + 1);
            if (t < start || t >= end) return;
        } else {
            req = (int)(t / a.q_per_request);
            start = req * a.q_per_request;
            end = start + a.q_per_request;
        }
        kv = max(__ldg(a.kv_lens + req), 0);
        const long long pos = (long long)kv - (end - t);
        hi = kv;
        if (a.causal) hi = (int)max(min((long long)hi, pos + 1), 0ll);
        if (a.window > 0) lo = (int)max(pos - a.window + 1, 0ll);
    }
    const long long there = (long long)a.bt_width * kBlockKeys;
    kv = (int)min((long long)kv, there);
    if (!a.selected) hi = min(hi, kv);
    float q[E], acc[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load16<FP16>(a.q, t * a.q_token + head * a.q_head + lane * E + e);
        acc[e] = 0.0f;
    }
    for (int i = lo + warp; i < hi; i += kWarps) {
        int p = i;
        if (a.selected) {
            p = __ldg(a.selected + t * a.sel_stride + i);
            if (p < 0 || p >= kv) continue;
        }
        long long page = __ldg(a.block_table + req * a.bt_stride + (p >> 6));
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.status, kStatusBadBlock);
            page = 0;
        }
        auto row = [&](const NvCache& c, float (&x)[E]) {
            const uint8_t* codes = c.codes + page * c.page + (p & 63) * c.slot + kvh * c.head + lane * (E / 2);
            const uint32_t s = e4m3_to_f16x2_dup(__ldg(c.scales + page * c.s_page + (p & 63) * c.s_slot +
                                                       kvh * c.s_head + lane * E / kNvGroup));
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t h = mul_f16x2(e2m1x2_to_f16x2(__ldg(codes + e / 2)), s);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                x[e] = f.x;
                x[e + 1] = f.y;
            }
        };
        float k[E], v[E], dot = 0.0f;
        row(a.kc, k);
        row(a.vc, v);
#pragma unroll
        for (int e = 0; e < E; ++e) dot = fmaf(q[e], k[e], dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float z = dot * a.scale, next = fmaxf(m, z);
        const float f = m == -INFINITY ? 0.0f : expf(m - next), w = z == -INFINITY ? 0.0f : expf(z - next);
        m = next;
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * v[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
    if (lane == 0) {
        part[warp][D] = m;
        part[warp][D + 1] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][D]);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
        const float f = part[w][D] == -INFINITY ? 0.0f : expf(part[w][D] - top);
        sum += part[w][D + 1] * f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += part[w][lane * E + e] * f;
    }
    const float inv = sum > 0.0f || sum != sum ? a.vc.scale / sum : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const long long at = t * a.out_token + head * a.out_head + lane * E + e;
        if constexpr (FP16) static_cast<__half*>(a.out)[at] = __float2half_rn(acc[e] * inv);
        else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(acc[e] * inv);
    }
    if (lane == 0 && a.lse) a.lse[t * a.kv_heads * a.group + head] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_nvfp4_attention(int head_dim, bool fp16, const NvAttnArgs& a, cudaStream_t stream)
{
    const dim3 grid((unsigned)a.tokens, (unsigned)(a.kv_heads * a.group));
    if (head_dim == 128)
        return fp16 ? launch_dependent(nvfp4_attention_kernel<128, true>, grid, kWarps * 32, 0, stream, a)
                    : launch_dependent(nvfp4_attention_kernel<128, false>, grid, kWarps * 32, 0, stream, a);
    return fp16 ? launch_dependent(nvfp4_attention_kernel<64, true>, grid, kWarps * 32, 0, stream, a)
                : launch_dependent(nvfp4_attention_kernel<64, false>, grid, kWarps * 32, 0, stream, a);
}

}  // namespace pml
