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
// operations each.  A row (one head of one token) is cut into units of two
// 16-byte accesses: the two halves of eight (four in fp32) pairs, two
// neighbours of whole pairs, or two that only pass through.  A power of two
// of neighbouring threads takes a row, a thread a unit of up to four rows, and
// a CTA that many rows of the flattened (token, head) list: it loads all it
// will ever load, computes its tokens' cosines and sines into shared memory
// while that is on its way (an angle serves every head), turns and stores.
// Sixteen-bit values are unpacked and packed two to a word: converted one by
// one they take a quarter-rate instruction each, and the kernel's time was
// its instructions'.  Narrower accesses serve sizes and strides that 16 bytes
// do not divide.
//
// Measured (a plain copy reaches 6776 GB/s): 16384 tokens x 32 heads of 128 in
// bf16 40.9 us, 6.56 TB/s, 97 % of the copy; 8190 tokens x 80 heads of 128 in
// fp16 into pages 56.5 us, 5.95 TB/s, 88 % (issue slots 69 % busy); 4099 x 24
// heads of 96 in fp32 14.4 us, 5.2 TB/s, 78 % (short: 75 MB).  Four CTAs an
// SM (64 registers) instead of three took the pages from 64.0 to 56.5 us, the
// fp32 rows from 16.0 to 14.4.  A decode step's 64 tokens x 48 rows: 3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dependent.cuh"
#include "rotary.cuh"
#include "serving.h"

namespace pml {

namespace {

constexpr int kThreads = kRopeThreads;

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
    uint32_t w[(VEC * sizeof(T) + 3) / 4];
    __device__ Vec() {}
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(Vec<T, VEC>& v, const T* p)
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

// Two neighbouring 16-bit values of a word.
__device__ __forceinline__ float2 unpack(uint32_t w, __half)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 unpack(uint32_t w, __nv_bfloat16)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __half)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (p, q) turned by the angle of c = (cosine, sine)
__device__ __forceinline__ float2 turn(float p, float q, float cosine, float sine)
{
    return make_float2(p * cosine - q * sine, q * cosine + p * sine);
}

// Pair i is (x[i], y[i]); c: the token's angles, this unit's the u-th run.
template <typename T, int VEC>
__device__ __forceinline__ void turn_across(Vec<T, VEC>& x, Vec<T, VEC>& y, const float2* c, int half, int u)
{
    if constexpr (VEC == 1) {
        const float2 v = turn(to_float(x.e[0]), to_float(y.e[0]), c[u].x, c[u].y);
        x.e[0] = from_float<T>(v.x);
        y.e[0] = from_float<T>(v.y);
    } else {
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
            const float4 w = *reinterpret_cast<const float4*>(c + turn_place<VEC, false>(half, u * VEC + 2 * k));
            if constexpr (sizeof(T) == 2) {
                const float2 a = unpack(x.w[k], T()), b = unpack(y.w[k], T());
                const float2 p = turn(a.x, b.x, w.x, w.y), q = turn(a.y, b.y, w.z, w.w);
                x.w[k] = pack(p.x, q.x, T());
                y.w[k] = pack(p.y, q.y, T());
            } else {
                const float2 p = turn(x.e[2 * k], y.e[2 * k], w.x, w.y);
                const float2 q = turn(x.e[2 * k + 1], y.e[2 * k + 1], w.z, w.w);
                x.e[2 * k] = p.x;
                y.e[2 * k] = p.y;
                x.e[2 * k + 1] = q.x;
                y.e[2 * k + 1] = q.y;
            }
        }
    }
}

// Pair i is (v[2i], v[2i + 1]); its angles are the run-th run of the token's.
template <typename T, int VEC>
__device__ __forceinline__ void turn_along(Vec<T, VEC>& v, const float2* c, int half, int run)
{
    constexpr int kPairs = VEC / 2;
    if constexpr (kPairs == 1) {
        const float2 w = c[run];
        if constexpr (sizeof(T) == 2) {
            const float2 a = unpack(v.w[0], T()), p = turn(a.x, a.y, w.x, w.y);
            v.w[0] = pack(p.x, p.y, T());
        } else {
            const float2 p = turn(v.e[0], v.e[1], w.x, w.y);
            v.e[0] = p.x;
            v.e[1] = p.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPairs; k += 2) {
            const float4 w = *reinterpret_cast<const float4*>(c + turn_place<kPairs, true>(half, run * kPairs + k));
            if constexpr (sizeof(T) == 2) {
                const float2 a = unpack(v.w[k], T()), b = unpack(v.w[k + 1], T());
                const float2 p = turn(a.x, a.y, w.x, w.y), q = turn(b.x, b.y, w.z, w.w);
                v.w[k] = pack(p.x, p.y, T());
                v.w[k + 1] = pack(q.x, q.y, T());
            } else {
                const float2 p = turn(v.e[2 * k], v.e[2 * k + 1], w.x, w.y);
                const float2 q = turn(v.e[2 * k + 2], v.e[2 * k + 3], w.z, w.w);
                v.e[2 * k] = p.x;
                v.e[2 * k + 1] = p.y;
                v.e[2 * k + 2] = q.x;
                v.e[2 * k + 3] = q.y;
            }
        }
    }
}

// MODE 0: pairs in two halves, VEC pairs per unit; 1: interleaved pairs, two
// neighbouring accesses per unit; 2: interleaved pairs, two elements per unit
// (VEC 1).
template <typename T, int VEC, int MODE, bool PAGED>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeArgs a)
{
    extern __shared__ __align__(16) float2 cs[];
    __shared__ long long page_of[kRopeMaxTokens];
    __shared__ int slot_of[kRopeMaxTokens];
    __shared__ int state_of[kRopeMaxTokens];    // 0 padding, 1 q only, 2 q, k and v

    allow_dependent_launch();
    grid_dependency_wait();
    const int half = a.rot.half, rot = 2 * half, off = a.rot.offset;
    const int rows = a.q.heads + (PAGED ? a.k.heads + a.v.heads : 0);    // of a token
    // the CTA's rows of all tokens' rows, and its tokens
    const long long row0 = (long long)blockIdx.x * a.rows_per_cta;
    const int count = (int)min((long long)a.rows_per_cta, (long long)a.tokens * rows - row0);
    const long long token0 = row0 / rows;
    const int first = (int)(row0 - token0 * rows);         // row of the first token
    const int nt = (first + count - 1) / rows + 1;
    const int u = threadIdx.x & ((1 << a.row_lanes_log2) - 1);
    const int rows_step = kThreads >> a.row_lanes_log2;
    const float per_row = 1.0f / (float)rows;

    // this thread's unit: two accesses of a row, at e0 and e1 (< 0: none); of
    // a row that turns, and of one that does not (v)
    const int turn_units = MODE != 1 ? half / VEC : 0;
    const bool turns = u < turn_units;
    int e0, e1, v0 = -1, v1 = -1;
    if (turns) {
        e0 = MODE == 2 ? off + 2 * u : off + u * VEC;
        e1 = MODE == 2 ? e0 + 1 : e0 + half;
    } else {
        const int k = 2 * (u - turn_units), rest = (a.dim - (MODE == 1 ? 0 : rot)) / VEC;
        e0 = k < rest ? k * VEC : -1;
        e1 = k + 1 < rest ? (k + 1) * VEC : -1;
        if (MODE != 1) {
            if (e0 >= off) e0 += rot;
            if (e1 >= off) e1 += rot;
        }
    }
    if constexpr (PAGED) {
        if (2 * u < a.dim / VEC) v0 = 2 * u * VEC;
        if (2 * u + 1 < a.dim / VEC) v1 = (2 * u + 1) * VEC;
    }
    // (MODE 1) an access turns if it lies in the rotated part
    const bool in0 = MODE == 1 && e0 >= off && e0 < off + rot;
    const bool in1 = MODE == 1 && e1 >= off && e1 < off + rot;
    // q in place: what does not turn stays
    const int q0 = a.skip_rest && !turns && !in0 ? -1 : e0, q1 = a.skip_rest && !turns && !in1 ? -1 : e1;

    Vec<T, VEC> x[kRopeUnits], y[kRopeUnits];
    // token of the CTA and row of the token, of unit b
    auto place = [&](int b, int& t, int& r) {
        const int i = (int)(threadIdx.x >> a.row_lanes_log2) + b * rows_step;
        r = first + i;
        t = (int)(((float)r + 0.5f) * per_row);      // r / rows: r is below 2^16
        r -= t * rows;
        return i < count;
    };
#pragma unroll
    for (int b = 0; b < kRopeUnits; ++b) {
        int t, r;
        if (!place(b, t, r)) continue;
        const bool is_q = !PAGED || r < a.q.heads, is_v = PAGED && r >= a.q.heads + a.k.heads;
        const RopeRows& set = is_q ? a.q : is_v ? a.v : a.k;
        const int head = is_q ? r : is_v ? r - a.q.heads - a.k.heads : r - a.q.heads;
        const T* src = static_cast<const T*>(set.src) + (token0 + t) * set.src_token + head * set.src_head;
        const int f0 = is_q ? q0 : is_v ? v0 : e0, f1 = is_q ? q1 : is_v ? v1 : e1;
        if (f0 >= 0) load_vec(x[b], src + f0);
        if (f1 >= 0) load_vec(y[b], src + f1);
    }

    fill_turns<MODE == 1 ? VEC / 2 : VEC, MODE == 1>(a.rot, cs, token0, nt);
    if constexpr (PAGED) {
        // (by the last warp: the first ones have the angles)
        const int t = (int)threadIdx.x - (kThreads - 32);
        if (t >= 0 && t < nt) {
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

#pragma unroll
    for (int b = 0; b < kRopeUnits; ++b) {
        int t, r;
        if (!place(b, t, r)) continue;
        const bool is_q = !PAGED || r < a.q.heads, is_v = PAGED && r >= a.q.heads + a.k.heads;
        const RopeRows& set = is_q ? a.q : is_v ? a.v : a.k;
        const int head = is_q ? r : is_v ? r - a.q.heads - a.k.heads : r - a.q.heads;
        T* dst = static_cast<T*>(set.dst) + head * set.dst_head;
        if constexpr (PAGED) {
            if (state_of[t] < (is_q ? 1 : 2)) continue;
            dst += is_q ? (token0 + t) * set.dst_token : page_of[t] * set.dst_page + slot_of[t] * set.dst_token;
        } else {
            dst += (token0 + t) * set.dst_token;
        }
        const int f0 = is_q ? q0 : is_v ? v0 : e0, f1 = is_q ? q1 : is_v ? v1 : e1;
        if (!is_v) {
            const float2* c = cs + t * turn_stride(half);
            if constexpr (MODE == 1) {
                if (in0) turn_along(x[b], c, half, (e0 - off) / VEC);
                if (in1) turn_along(y[b], c, half, (e1 - off) / VEC);
            } else {
                if (turns) turn_across(x[b], y[b], c, half, u);
            }
        }
        if (f0 >= 0) store_vec(dst + f0, x[b]);
        if (f1 >= 0) store_vec(dst + f1, y[b]);
    }
}

template <typename T, int VEC, int MODE>
cudaError_t launch_mode(const RopeArgs& a, cudaStream_t stream)
{
    const long long rows = (long long)a.tokens * (a.q.heads + a.k.heads + a.v.heads);
    const dim3 grid((unsigned)((rows + a.rows_per_cta - 1) / a.rows_per_cta));
    const size_t smem = (size_t)kRopeMaxTokens * turn_stride(a.rot.half) * sizeof(float2);
    return a.paged ? launch_dependent(rope_kernel<T, VEC, MODE, true>, grid, kThreads, smem, stream, a)
                   : launch_dependent(rope_kernel<T, VEC, MODE, false>, grid, kThreads, smem, stream, a);
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
