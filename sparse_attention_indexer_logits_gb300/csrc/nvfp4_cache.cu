// K/V caches held in 4 bits on sm_103a: rows quantised into their pages as they
// are written, and pages read back in 16 bits.
//
// A row is E2M1 codes, two to a byte, and one E4M3 scale s for sixteen values
// x; with the cache's power of two g
//
//   s = e4m3(max |x| / (6 g)),   code = e2m1(x / (s g)),   value = code s g.
//
// The codes are those of the exact quotient, ties to the even one: x has at
// most 11 significant bits and s g four, so a quotient that is not on a border
// between two codes is 2^-12 or more away from it, and one that is comes out
// exact from a product with 1 / (s g) and one step of Newton's.  A value read
// has at most six significant bits: exact in both types within their range.
//
// Both are bound by memory: 2 bytes of a value on one side, 9/16 on the other.
// Measured (a copy reaches 6794 GB/s; inputs that are not in L2):
//   7 contexts of 9000 .. 32768 keys read, 4 heads of 64, bf16
//       29.6 us, 138 MB: 69 % of the copy; about 5 us of it are a launch and the
//       lookups before the first codes.  (A strip's codes loaded while the one
//       before is turned: no faster; three CTAs an SM 30.9, five 30.1; stores that
//       stay in L2 30.7 against 26.9 where the pages read are there)
//   8190 tokens written, 8 heads of 128, fp16, and their contexts read
//       22.0 us, 86 MB in two launches: a floor of 12.7
//   64 tokens written and contexts of up to 160 read: 11.7 us, a floor of 3.9: two
//       launches, each a chain of three loads
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dependent.cuh"
#include "nvfp4_cache.h"
#include "rotary.cuh"

namespace pml {

namespace {

constexpr uint32_t kNanScale = 0x7f;

template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t w)
{
    if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    uint32_t r;
    if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_of(float x)
{
    uint16_t p;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(0.0f), "f"(x));
    return p & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code)
{
    const uint32_t h = e4m3_to_f16x2_dup(code);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// Eight values to eight codes, four bytes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&x)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Eight values' codes under the scale d, rc = 1 / d.
template <bool FP16>
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[4], float d, float rc)
{
    const uint64_t nd = pack2(-d, -d), rr = pack2(rc, rc);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<FP16>(w[i]);
        const uint64_t v = pack2(f.x, f.y), p = mul2(v, rr), q = fma2(fma2(p, nd, v), rr, p);
        asm("mov.b64 {%0, %1}, %2;" : "=f"(x[2 * i]), "=f"(x[2 * i + 1]) : "l"(q));
    }
    return e2m1x8_of(x);
}

// The same past the largest scale, where a quotient might be infinite.
template <bool FP16>
__device__ __noinline__ uint32_t codes_beyond(uint32_t a, uint32_t b, uint32_t c, uint32_t e, float d, float rc)
{
    const uint32_t w[4] = {a, b, c, e};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<FP16>(w[i]);
        const float u = fminf(fmaxf(f.x, -8.0f * d), 8.0f * d), v = fminf(fmaxf(f.y, -8.0f * d), 8.0f * d);
        x[2 * i] = fmaf(fmaf(-u * rc, d, u), rc, u * rc);
        x[2 * i + 1] = fmaf(fmaf(-v * rc, d, v), rc, v * rc);
    }
    return e2m1x8_of(x);
}

// Sixteen values to their codes and scale.
template <bool FP16>
__device__ __forceinline__ uint2 quantise16(const uint4 (&v)[2], float g, uint32_t& scale)
{
    const uint32_t w[2][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w}};
    // magnitudes compare like their bits, infinities and NaN above all others
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, w[i / 4][i % 4] & 0x7fff7fffu);
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    if (top >= (FP16 ? 0x7c00u : 0x7f80u)) {
        scale = kNanScale;
        return make_uint2(0u, 0u);
    }
    const float amax = unpack16<FP16>(top).x;
    scale = e4m3_of(__fdiv_rn(amax, 6.0f * g));
    const float d = e4m3_value(scale) * g;
    if (d == 0.0f) return make_uint2(0u, 0u);
    const float rc = __frcp_rn(d);
    if (amax > 8.0f * d)
        return make_uint2(codes_beyond<FP16>(w[0][0], w[0][1], w[0][2], w[0][3], d, rc),
                          codes_beyond<FP16>(w[1][0], w[1][1], w[1][2], w[1][3], d, rc));
    return make_uint2(codes_of<FP16>(w[0], d, rc), codes_of<FP16>(w[1], d, rc));
}

// A thread takes a group of sixteen, eight (four) threads a row; a CTA sixteen
// tokens and two (four) of their rows (k's heads, then v's).  Neighbouring rows of
// threads are neighbouring tokens of one head: what a warp writes is 256 bytes
// of codes and a whole sector of scales in a page that holds its heads one after
// another.  Every thread looks up its token's slot, while its values are on their
// way.  (Four groups a thread, a token's slot looked up once and shared: 25.8 us
// for a chunk of 8190 tokens written and read back, 23.5 with the lookup beside the
// quantising, 22.0 so: the full number of threads an SM, and no barrier.)
template <int D, bool FP16>
__global__ void __launch_bounds__(kNvAppendThreads, 8) nvfp4_append_kernel(const NvAppendArgs a)
{
    constexpr int kLanes = D / kNvGroup;
    allow_dependent_launch();
    grid_dependency_wait();
    const int i = threadIdx.x / kLanes, g = threadIdx.x % kLanes;
    const long long token = (long long)blockIdx.x * kNvAppendTokens + i % kNvAppendTokens;
    const int head = blockIdx.y * (kNvAppendThreads / kLanes / kNvAppendTokens) + i / kNvAppendTokens;
    if (token >= a.tokens || head >= 2 * a.heads) return;
    const bool is_v = head >= a.heads;
    const int h = is_v ? head - a.heads : head;
    const uint16_t* row = is_v ? static_cast<const uint16_t*>(a.v) + token * a.v_token + h * a.v_head
                               : static_cast<const uint16_t*>(a.k) + token * a.k_token + h * a.k_head;
    const uint4* src = reinterpret_cast<const uint4*>(row) + 2 * g;
    const uint4 v[2] = {__ldg(src), __ldg(src + 1)};
    const long long pos = a.pos64 ? __ldg(static_cast<const long long*>(a.positions) + token)
                                  : (long long)__ldg(static_cast<const int32_t*>(a.positions) + token);
    bool pad;
    long long page;
    int slot;
    const bool ok = find_slot(a.slot, token, pos, pad, page, slot);
    const NvCache& c = is_v ? a.vc : a.kc;
    uint32_t scale;
    const uint2 codes = quantise16<FP16>(v, c.scale, scale);
    if (!ok) return;
    *reinterpret_cast<uint2*>(c.codes + page * c.page + slot * c.slot + h * c.head + g * 8) = codes;
    c.scales[page * c.s_page + slot * c.s_slot + h * c.s_head + g] = (uint8_t)scale;
}

constexpr int kReadThreads = 256, kReadCtas = 4;

// Blocks of request b that are there.
__device__ __forceinline__ int blocks_there(const NvReadArgs& a, int b)
{
    return min(blocks_of(__ldg(a.kv_lens + b)), a.width);
}

// The pages of all requests, each in strips (a head's keys and values), in order,
// cut into one contiguous range per CTA.  A thread turns eight values, four bytes
// of codes, into sixteen bytes, several rows at a time.
template <int D, bool FP16>
__global__ void __launch_bounds__(kReadThreads, kReadCtas) nvfp4_read_kernel(const NvReadArgs a)
{
    __shared__ int start[2];               // request, block
    __shared__ long long first_left[2];    // strip within the block, strips of the range
    allow_dependent_launch();
    grid_dependency_wait();
    const int strips = a.heads;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        long long total = 0;
        for (int b = lane; b < a.batch; b += 32) total += blocks_there(a, b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const long long s0 = range_start(total * strips, gridDim.x, blockIdx.x);
        const long long s1 = range_start(total * strips, gridDim.x, blockIdx.x + 1);
        if (lane == 0) {
            first_left[0] = s0 % strips;
            first_left[1] = s1 - s0;
        }
        long long rem = s0 / strips;
        if (s0 < s1) {
            for (int c = 0; c < a.batch; c += 32) {
                const long long n = c + lane < a.batch ? blocks_there(a, c + lane) : 0;
                long long incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += u;
                }
                if (incl - n <= rem && rem < incl) {
                    start[0] = c + lane;
                    start[1] = (int)(rem - (incl - n));
                }
                const long long all = __shfl_sync(0xffffffffu, incl, 31);
                if (rem < all) break;
                rem -= all;
            }
        }
    }
    __syncthreads();
    long long left = first_left[1];
    if (left == 0) return;
    int b = start[0], j = start[1], strip = (int)first_left[0];
    const int unit = threadIdx.x % (D / 8), row0 = threadIdx.x / (D / 8);
    constexpr int kStep = kReadThreads / (D / 8), kUnits = kBlockKeys / kStep;
    // the caches' scales, where fp16 holds them
    const bool plain[2] = {a.kc.scale >= 0x1p-14f && a.kc.scale <= 0x1p15f, a.vc.scale >= 0x1p-14f && a.vc.scale <= 0x1p15f};
    const uint32_t g16[2] = {pack16<true>(a.kc.scale, a.kc.scale), pack16<true>(a.vc.scale, a.vc.scale)};
    for (; left > 0; --left) {
        const int rows = min(__ldg(a.kv_lens + b) - j * kBlockKeys, kBlockKeys);
        const long long page = __ldg(a.block_table + b * a.bt_stride + j);
        const long long to = __ldg(a.out_table + b * a.ot_stride + j);
        if (page < 0 || page >= a.num_pages || to < 0 || to >= a.out_pages) {
            if (threadIdx.x == 0) atomicOr(a.status, kStatusBadBlock);
        } else {
            const long long slots[2] = {a.k_slot, a.v_slot};
            uint16_t* const out[2] = {static_cast<uint16_t*>(a.k_out) + to * a.k_page + strip * a.k_head + unit * 8,
                                      static_cast<uint16_t*>(a.v_out) + to * a.v_page + strip * a.v_head + unit * 8};
            uint32_t w[2][kUnits], s[2][kUnits];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const NvCache& c = x ? a.vc : a.kc;
                const uint8_t* codes = c.codes + page * c.page + strip * c.head + unit * 4;
                const uint8_t* scales = c.scales + page * c.s_page + strip * c.s_head + unit / 2;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    const int r = row0 + i * kStep;
                    if (r >= rows) continue;
                    w[x][i] = __ldg(reinterpret_cast<const uint32_t*>(codes + r * c.slot));
                    s[x][i] = __ldg(scales + r * c.s_slot);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float g = x ? a.vc.scale : a.kc.scale;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    const int r = row0 + i * kStep;
                    if (r >= rows) continue;
                    uint32_t v[4], y[4];
                    e2m1x8_to_f16x2x4(w[x][i], v);
                    const uint32_t sc = e4m3_to_f16x2_dup(s[x][i]);
                    // (in fp16 a product with a power of two rounds as one in fp32 would)
                    if (FP16 && plain[x]) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = mul_f16x2(mul_f16x2(v[e], sc), g16[x]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = unpack16<true>(mul_f16x2(v[e], sc));
                            float lo, hi;
                            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(mul2(pack2(f.x, f.y), pack2(g, g))));
                            y[e] = pack16<FP16>(lo, hi);
                        }
                    }
                    uint4* to_row = reinterpret_cast<uint4*>(out[x] + r * slots[x]);
                    __stcs(to_row, make_uint4(y[0], y[1], y[2], y[3]));    // (written once, four fifths of the traffic)
                }
            }
        }
        if (++strip == strips) {
            strip = 0;
            if (++j >= blocks_there(a, b)) {
                j = 0;
                ++b;
                while (b < a.batch && blocks_there(a, b) == 0) ++b;
                if (b >= a.batch) return;
            }
        }
    }
}

}  // namespace

cudaError_t launch_nvfp4_append(const NvAppendArgs& a, cudaStream_t stream)
{
    const int heads_per_cta = kNvAppendThreads / (a.dim / kNvGroup) / kNvAppendTokens;
    const dim3 grid((unsigned)((a.tokens + kNvAppendTokens - 1) / kNvAppendTokens),
                    (unsigned)((2 * a.heads + heads_per_cta - 1) / heads_per_cta));
    if (a.dim == 128)
        return a.fp16 ? launch_dependent(nvfp4_append_kernel<128, true>, grid, kNvAppendThreads, 0, stream, a)
                      : launch_dependent(nvfp4_append_kernel<128, false>, grid, kNvAppendThreads, 0, stream, a);
    return a.fp16 ? launch_dependent(nvfp4_append_kernel<64, true>, grid, kNvAppendThreads, 0, stream, a)
                  : launch_dependent(nvfp4_append_kernel<64, false>, grid, kNvAppendThreads, 0, stream, a);
}

cudaError_t launch_nvfp4_read(const NvReadArgs& a, int sm_count, cudaStream_t stream)
{
    const dim3 grid((unsigned)(sm_count * kReadCtas));
    if (a.dim == 128)
        return a.fp16 ? launch_dependent(nvfp4_read_kernel<128, true>, grid, kReadThreads, 0, stream, a)
                      : launch_dependent(nvfp4_read_kernel<128, false>, grid, kReadThreads, 0, stream, a);
    return a.fp16 ? launch_dependent(nvfp4_read_kernel<64, true>, grid, kReadThreads, 0, stream, a)
                  : launch_dependent(nvfp4_read_kernel<64, false>, grid, kReadThreads, 0, stream, a);
}

}  // namespace pml
