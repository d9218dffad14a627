// Rotary positions on sm_103a, alone or on the way into a paged cache.
//
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = position * inv_freq[j]
//
// for the `half` pairs of each head that start at `offset`: (i, half + i), or
// (2i, 2i + 1) when interleaved; the head's other elements pass through.  The
// gradient is the transposed rotation: the sine's sign turns.  In the paged
// form the launch rotates q into its own tensor, rotates k into the pages of
// the key cache and copies v into those of the value cache.
//
// Bound by memory: every element is read once and written once, about three
// operations each.  A CTA takes a few tokens: their cosines and sines are
// computed once into shared memory (an angle serves every head), then the
// threads walk the tokens' (head, unit) pairs, a unit being one 16-byte
// access that holds whole pairs, or two accesses that hold the two halves of
// eight (four in fp32) pairs.  Narrower accesses serve sizes and strides that
// 16 bytes do not divide.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rotary.cuh"
#include "serving.h"

namespace pml {

namespace {

constexpr int kThreads = 256;

template <int BYTES>
struct Raw;
template <>
struct Raw<2> { using type = uint16_t; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<16> { using type = uint4; };

template <typename T>
__device__ __forceinline__ float to_float(T x) { return static_cast<float>(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x) { return static_cast<T>(x); }

template <typename T, int VEC>
union Vec {
    typename Raw<VEC * sizeof(T)>::type raw;
    T e[VEC];
    __device__ Vec() {}
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(Vec<T, VEC>& v, const T* p)
{
    using R = typename Raw<VEC * sizeof(T)>::type;
    v.raw = __ldg(reinterpret_cast<const R*>(p));
}
// in place the other threads' stores may share this launch's memory: no
// read-only path
template <typename T, int VEC>
__device__ __forceinline__ void load_vec_rw(Vec<T, VEC>& v, const T* p)
{
    using R = typename Raw<VEC * sizeof(T)>::type;
    v.raw = *reinterpret_cast<const R*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, VEC>& v)
{
    using R = typename Raw<VEC * sizeof(T)>::type;
    *reinterpret_cast<R*>(p) = v.raw;
}

// MODE 0: pairs in two halves, VEC pairs per unit; 1: interleaved pairs, VEC
// elements (VEC / 2 pairs) per unit; 2: interleaved pairs read element by
// element (VEC 1).
template <typename T, int VEC, int MODE, bool PAGED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a)
{
    extern __shared__ float2 cs[];
    __shared__ long long page_of[8];
    __shared__ int slot_of[8];
    __shared__ int state_of[8];    // 0 padding, 1 q only, 2 q, k and v

    const long long token0 = (long long)blockIdx.x * a.tokens_per_cta;
    const int nt = (int)min((long long)a.tokens_per_cta, (long long)a.tokens - token0);
    const int half = a.rot.half, rot = 2 * half, off = a.rot.offset;

    fill_turns(a.rot, cs, token0, nt);
    if constexpr (PAGED) {
        if ((int)threadIdx.x < nt) {
            const int t = threadIdx.x;
            bool pad;
            long long page;
            int slot;
            const bool ok = find_slot(a.slot, token0 + t, load_position(a.rot, token0 + t), pad,
                                      page, slot);
            page_of[t] = page;
            slot_of[t] = slot;
            state_of[t] = pad ? 0 : ok ? 2 : 1;
        }
    }
    __syncthreads();

    // units of a rotated row, and those that only pass through
    const int turn_units = MODE == 1 ? rot / VEC : half / VEC;
    const int rest_units = a.skip_rest ? 0 : (a.dim - rot) / VEC;
    const int q_row = turn_units + rest_units;
    const int k_row = turn_units + (a.dim - rot) / VEC;
    const int v_row = a.dim / VEC;
    const int q_units = a.q.heads * q_row;
    const int k_units = PAGED ? a.k.heads * k_row : 0;
    const int units = q_units + k_units + (PAGED ? a.v.heads * v_row : 0);

    for (int i = threadIdx.x; i < nt * units; i += kThreads) {
        const int t = i / units;
        int u = i - t * units;
        const T* src;
        T* dst;
        bool rotated = true;
        if constexpr (PAGED) {
            const int st = state_of[t];
            if (st == 0 || (st == 1 && u >= q_units)) continue;
        }
        if (!PAGED || u < q_units) {
            const int h = u / q_row;
            u -= h * q_row;
            src = static_cast<const T*>(a.q.src) + (token0 + t) * a.q.src_token + h * a.q.src_head;
            dst = static_cast<T*>(a.q.dst) + (token0 + t) * a.q.dst_token + h * a.q.dst_head;
        } else {
            const bool is_k = u < q_units + k_units;
            u -= is_k ? q_units : q_units + k_units;
            const int row = is_k ? k_row : v_row;
            const RopeRows& r = is_k ? a.k : a.v;
            const int h = u / row;
            u -= h * row;
            rotated = is_k;
            src = static_cast<const T*>(r.src) + (token0 + t) * r.src_token + h * r.src_head;
            dst = static_cast<T*>(r.dst) + page_of[t] * r.dst_page + slot_of[t] * r.dst_token +
                  h * r.dst_head;
        }
        if (rotated && u < turn_units) {
            const float2* c = cs + t * half;
            if constexpr (MODE == 0) {
                const int j = u * VEC;
                Vec<T, VEC> x, y;
                load_vec_rw(x, src + off + j);
                load_vec_rw(y, src + off + half + j);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 w = c[j + e];
                    const float p = to_float(x.e[e]), q = to_float(y.e[e]);
                    x.e[e] = from_float<T>(p * w.x - q * w.y);
                    y.e[e] = from_float<T>(q * w.x + p * w.y);
                }
                store_vec(dst + off + j, x);
                store_vec(dst + off + half + j, y);
            } else if constexpr (MODE == 1) {
                const int j = u * VEC;
                Vec<T, VEC> x;
                load_vec_rw(x, src + off + j);
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float2 w = c[(j + e) >> 1];
                    const float p = to_float(x.e[e]), q = to_float(x.e[e + 1]);
                    x.e[e] = from_float<T>(p * w.x - q * w.y);
                    x.e[e + 1] = from_float<T>(q * w.x + p * w.y);
                }
                store_vec(dst + off + j, x);
            } else {
                const float2 w = c[u];
                const float p = to_float(src[off + 2 * u]), q = to_float(src[off + 2 * u + 1]);
                dst[off + 2 * u] = from_float<T>(p * w.x - q * w.y);
                dst[off + 2 * u + 1] = from_float<T>(q * w.x + p * w.y);
            }
        } else {
            // an element outside the rotated part, or of v
            int e = rotated ? (u - turn_units) * VEC : u * VEC;
            if (rotated && e >= off) e += rot;
            Vec<T, VEC> x;
            load_vec_rw(x, src + e);
            store_vec(dst + e, x);
        }
    }
}

template <typename T, int VEC, int MODE>
cudaError_t launch_mode(const RopeArgs& a, cudaStream_t stream)
{
    const unsigned grid = (unsigned)((a.tokens + a.tokens_per_cta - 1) / a.tokens_per_cta);
    const size_t smem = (size_t)a.tokens_per_cta * a.rot.half * sizeof(float2);
    if (a.paged) rope_kernel<T, VEC, MODE, true><<<grid, kThreads, smem, stream>>>(a);
    else rope_kernel<T, VEC, MODE, false><<<grid, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RopeArgs& a, cudaStream_t stream)
{
    constexpr int kWide = 16 / (int)sizeof(T);
    const bool il = a.rot.interleaved != 0;
    if (a.vec == kWide)
        return il ? launch_mode<T, kWide, 1>(a, stream) : launch_mode<T, kWide, 0>(a, stream);
    if (a.vec == 2) return il ? launch_mode<T, 2, 1>(a, stream) : launch_mode<T, 2, 0>(a, stream);
    return il ? launch_mode<T, 1, 2>(a, stream) : launch_mode<T, 1, 0>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream)
{
    if (a.elem == 4) return launch_type<float>(a, stream);
    return a.fp16 ? launch_type<__half>(a, stream) : launch_type<__nv_bfloat16>(a, stream);
}

}  // namespace pml
