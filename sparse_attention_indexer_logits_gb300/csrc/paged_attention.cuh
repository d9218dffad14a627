// Attention of new tokens over a paged cache on sm_103a.
//
//   out[t, h] = sum_p softmax_p(scale * q[t, h] . k_p) v_p
//
// over the positions p that token t may see: those of its request up to its
// own (causal), past position - window (window > 0), or the ones a list
// names.  One pass over the keys with a running maximum m and sum l of
// exponentials: a tile of 128 keys gives S = Q K^T, P = 2^(c S - c m), O += P V
// (fp16: 2^7 times as much, see PScale);
// at the end out = O / l and lse = scale * m + ln l.
//
// Work.  The rows of an item are up to 256 (token, head) pairs that share a kv
// head; a tile of 128 keys is one or two units of work, the item itself three.
// The units of all items, in order, are cut into one contiguous range per CTA,
// so a long request's keys are split over many CTAs and short requests share
// one, whatever the mix.  A range that ends inside an item leaves its (m, l, O)
// in the workspace and a second kernel joins the pieces.
//
// A CTA holds two 128-row accumulator pairs (S and O, 512 TMEM columns).  An
// item of more than 128 rows gives each its own half of the rows and both see
// every tile; an item of at most 128 rows gives both the same rows and the
// tiles in turn, and their two results are joined at its end.  Either way the
// tensor core works on one half while the other half's softmax runs:
//
//   load warp        walks the range; per item a descriptor and the Q rows,
//                    per tile the K and V pages (TMA, 128-byte swizzle) into
//                    a ring of stages; listed rows are gathered by it and the
//                    gather warp, 16 bytes a lane (cp.async).  TMA's gather4
//                    took 6800 cycles for the 512 row pieces of a tile's K
//                    and V, twice the time of everything else
//   land warp        counts the stages whose copies have landed into a plain
//                    word, which the MMA warp polls for less than an mbarrier
//   MMA warp         S_h = Q_h K^T (both operands in shared memory), then
//                    O_h += P_h V with P_h read from TMEM, where it replaced
//                    S_h, and V as the transposed operand
//   2 softmax groups 128 threads each, a row per thread: S from TMEM, maximum,
//                    exponentials, sum, P back to TMEM.  O is rescaled only
//                    when a row's maximum has grown by more than 2^8 in P's
//                    scale (exact: l and O share the reference), which is
//                    rare after the first tiles
//
// Masked places never reach a result, whatever they hold: scores are replaced
// by -inf before the maximum; V rows that no row of the item may see are
// zeroed in shared memory; and where a tile's V rows are visible to some rows
// and hidden from others (the causal diagonal, a window's edge) and hold an
// infinity or NaN, the group adds that tile's product row by row itself.
//
// Measured (a plain copy reaches 6776 GB/s, a library bf16 product 1909
// TFLOP/s):
//   64 single tokens over U[1024, 32768] keys, 8 kv heads of 128, bf16
//       687 us, 4.71 GB: bound by HBM, 101 % of the copy
//   4096 tokens that end 32768 keys, 32 heads over 4, bf16
//       1500-1555 us, 2.06 TFLOP: 1.33-1.37 PFLOP/s, 69-72 % of the
//       product's.  One half's chain (scores, softmax, P V) is hidden behind
//       the other's except for its hand-overs, and the board is at its power
//       limit
//   24 requests of 1 .. 500 tokens over up to 8000 keys, window 1500, fp16, 64
//       55 us: a floor of 7; a tile's chain of 3600 cycles, 17 tiles a CTA,
//       and the way into and out of two or three items
//   64 tokens x 2048 listed positions, 64 heads over 1, bf16
//       29 us: a floor of 10; a fixed part of 12 us (prologue, first lookups,
//       join), then the row copies.  (Sixteen lanes a row took 36 us: an
//       offset to shuffle for every copy)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention_work.cuh"
#include "common.cuh"
#include "dependent.cuh"
#include "ptx.cuh"
#include "serving.h"

namespace pml {
namespace attn {

constexpr int kThreads = 384;      // three warpgroups: softmax, softmax, MMA and copies
// Registers per thread: the block is launched with 168, the third warpgroup
// gives some back and the softmax groups, which hold a row of S, take them
// (2 * 208 + 88 = 3 * 168).
constexpr int kLaunchRegs = 168, kHighRegs = 208, kLowRegs = 88;
// (a scheduler serves warps w, w + 4, w + 8: the issuer, which polls, is not
// with the warps that hold the first 32 rows, all the rows of a small call)
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 11;
constexpr int kLoadWarp = 9;
constexpr int kGatherWarp = 8;     // selected: the second half of each tile's rows
constexpr int kLandWarp = 10;
constexpr int kItemSlots = 4;
constexpr int kItemInts = 16;

// item descriptor
enum { kItN, kItJ0, kItFlags, kItTok0, kItNtok, kItHead, kItPos0, kItKvHi, kItLo, kItHi, kItSlot };
constexpr int kAlt = 1;      // both halves hold the same rows and take the tiles in turn
constexpr int kWhole = 2;    // the piece is a whole item: write the output
constexpr int kEnd = 8;      // no more items
// piece record in the workspace
enum { kPcUsed, kPcTok0, kPcNtok, kPcHead, kPcLast };

// A wait by a whole warp: one result for all lanes, so that a wait that ran
// out in some lanes only cannot part them before the next warp-wide step.
// (The slow path is inlined: a kernel that re-splits its registers contains no
// calls.)
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, volatile int* abort,
                                          unsigned int* status)
{
    return __all_sync(0xffffffffu, mbar_wait<false>(b, parity, abort, status));
}

__device__ __forceinline__ uint32_t ld_acquire_shared(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint4 ld_acquire_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.acquire.cta.shared::cta.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_release_shared(uint32_t addr, uint32_t v)
{
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Waits until `places` copies have landed and (words != 0) the four warps of
// a group have written their part of the group's P number `count`, each
// saying so in its word; skip: the group has added that tile's product itself
// (all four say the same).
__device__ __forceinline__ bool words_ready(uint32_t landed, uint32_t places, uint32_t words,
                                            uint32_t count, bool& skip, volatile int* abort,
                                            unsigned int* status)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        uint4 w = make_uint4(2 * count, 2 * count, 2 * count, 2 * count);
        if (words != 0) w = ld_acquire_shared_v4(words);
        const uint32_t there = ld_acquire_shared(landed);
        if (there >= places && (w.x >> 1) == count && (w.y >> 1) == count && (w.z >> 1) == count &&
            (w.w >> 1) == count) {
            skip = w.x & 1u;
            return true;
        }
        if ((it & 255u) == 0) {
            if (*abort) return false;
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                atomicOr(status, kStatusWaitTimeout);
                *abort = 1;
                return false;
            }
        }
    }
}

// P, and so l and O, are 2^kLog2 times the weights: fp16 has half steps of
// 2^-25 below 2^-14, and a long row's many small weights, each under half a
// step, would be lost beside one large one.  With 2^7, and a reference that may
// be too low by 2^8, P stays below 2^15, and weights from 2^-21 of the largest
// on keep fp16's 11 bits.
template <bool FP16>
struct PScale {
    static constexpr float kLog2 = FP16 ? 7.0f : 0.0f;
    static constexpr float kInverse = FP16 ? 0x1p-7f : 1.0f;     // of a sum, before its logarithm
};

// Where columns 4 * col .. 4 * col + 3 of a row of a workspace slot lie.
template <int D>
__device__ __forceinline__ long long partial_at(int cta, int slot, int col, int row)
{
    return ((((long long)cta * 2 + slot) * (D / 4) + col) * kAttnSlotRows + row) * 4;
}

template <int D>
struct Cfg {
    static constexpr int kBlocks = D / 64;                     // 128-byte column blocks
    static constexpr int kBlockBytes = 128 * 128;              // 128 rows of 128 bytes
    static constexpr int kStageBytes = kBlocks * kBlockBytes;  // a K or V tile
    static constexpr int kHalfBytes = kBlocks * kBlockBytes;   // a Q half
    static constexpr int kStages = D == 128 ? 5 : 11;
    static constexpr int kQ = 0;
    static constexpr int kRing = kQ + 2 * kHalfBytes;
    static constexpr int kStats = kRing + kStages * kStageBytes;      // float2 [2][128]
    static constexpr int kBars = kStats + 2 * 128 * 8;
    // barriers: full, empty per stage; q full, q empty per half; s full, pv done, group
    // sync per half; o empty, alt sync; item full, item empty; the issuer's
    // last commit
    static constexpr int kNumBars = 2 * kStages + 4 + 6 + 2 + 2 * kItemSlots + 1;
    static constexpr int kItems = (kBars + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kMisc = kItems + kItemSlots * kItemInts * 4;
    static constexpr int kTotal = kMisc + 192;
};

constexpr uint32_t kColS = 0;      // S_h at 128 h; P_h over its first 64 columns
constexpr uint32_t kColO = 256;    // O_h at 256 + 128 h

// MN-major operand (V: keys are the rows, 128 bytes of columns each, 128-byte
// swizzle): groups of 64 columns lie `lbo` bytes apart, groups of eight keys
// 1024 bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lbo)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Sixteen bytes, or zeros (bytes = 0: src is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr)
{
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r)
                 : "r"(taddr)
                 : "memory");
    return r;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// 2^x; -inf gives 0
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    uint32_t r;
    if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t w)
{
    if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Whether either 16-bit value of w is an infinity or NaN.
template <bool FP16>
__device__ __forceinline__ bool not_finite(uint32_t w)
{
    constexpr uint32_t kExp = FP16 ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t kOne = FP16 ? 0x04000400u : 0x00800080u;
    return (((w & kExp) + kOne) & 0x80008000u) != 0;
}

__device__ __forceinline__ void request_of(const AttnArgs& a, int b, int& tok0, int& nq, int& kv)
{
    if (a.cu_q != nullptr) {
        const int s = __ldg(a.cu_q + b), e = __ldg(a.cu_q + b + 1);
        tok0 = min(max(s, 0), a.tokens);
        nq = min(max(e, tok0), a.tokens) - tok0;
    } else {
        tok0 = b * a.q_per_request;
        nq = a.q_per_request;
    }
    kv = max(__ldg(a.kv_lens + b), 0);
}

// Where a CTA's range begins, and how many units it has.
struct Start {
    int b, head, tile;   // selected: b is the token
    int at;              // unit of the item
    long long left;
};

// Executed by one warp.  `units`: shared memory for one number per request.
__device__ __forceinline__ Start find_start(const AttnArgs& a, long long* units, int lane)
{
    Start s = {0, 0, 0, 0, 0};
    long long total = 0;
#pragma unroll 1
    for (int b = lane; b < a.batch; b += 32) {
        int tok0, nq, kv;
        request_of(a, b, tok0, nq, kv);
        units[b] = units_of_request(a, nq, kv);
        total += units[b];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= a.kv_heads;
    long long rem = range_start(total, gridDim.x, blockIdx.x);
    s.left = range_start(total, gridDim.x, blockIdx.x + 1) - rem;
    if (s.left == 0) return s;
    // the request that holds unit `rem`, 32 at a time
    long long per_head = 0;
#pragma unroll 1
    for (int c = 0; c < a.batch; c += 32) {
        const long long v = c + lane < a.batch ? units[c + lane] : 0;
        long long incl = v * a.kv_heads;
        const long long mine = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned who = __ballot_sync(0xffffffffu, incl - mine <= rem && rem < incl);
        if (who) {
            const int l = __ffs(who) - 1;
            s.b = c + l;
            per_head = __shfl_sync(0xffffffffu, v, l);
            rem -= __shfl_sync(0xffffffffu, incl - mine, l);
            break;
        }
        rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    if (per_head == 0) { s.left = 0; return s; }    // never
    s.head = (int)(rem / per_head);
    long long off = rem - s.head * per_head;
    // the tile of that request's head, 32 at a time
    int tok0, nq, kv;
    request_of(a, s.b, tok0, nq, kv);
    const int tiles = tiles_of(a, nq);
#pragma unroll 1
    for (int c = 0; c < tiles; c += 32) {
        const int v = c + lane < tiles ? units_of(tile_span(a, nq, kv, c + lane)) : 0;
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned who = __ballot_sync(0xffffffffu, incl - v <= off && off < incl);
        if (who) {
            const int l = __ffs(who) - 1;
            s.tile = c + l;
            s.at = (int)(off - __shfl_sync(0xffffffffu, incl - v, l));
            break;
        }
        off -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return s;
}

template <int D, bool FP16, bool SEL>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap qmap,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const AttnArgs a)
{
    using C = Cfg<D>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    if (base & 1023u) {                       // the swizzled tiles need it; never seen
        if (threadIdx.x == 0) atomicOr(a.status, kStatusWaitTimeout);
        return;
    }
    const uint32_t bar = base + C::kBars;
    auto full_bar = [&](int s) { return bar + 8u * s; };
    auto empty_bar = [&](int s) { return bar + 8u * (S + s); };
    const uint32_t qfull0 = bar + 8u * (2 * S), qempty0 = qfull0 + 16u;   // per Q half
    const uint32_t sfull0 = qempty0 + 16u, pvdone0 = sfull0 + 16u,
                   group0 = pvdone0 + 16u, oempty = group0 + 16u, altbar = oempty + 8u,
                   itfull0 = altbar + 8u, itempty0 = itfull0 + 8u * kItemSlots, drain = itempty0 + 8u * kItemSlots;
    int* items = reinterpret_cast<int*>(smem + C::kItems);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
    volatile int* votes = reinterpret_cast<volatile int*>(smem + C::kMisc + 16);      // [2][2][4]
    // P written by warp w of half h: 2 * tiles, + 1 if this tile's product with V
    // has been added already
    const uint32_t ready0 = base + C::kMisc + 128;
    volatile uint32_t* ready = reinterpret_cast<volatile uint32_t*>(smem + C::kMisc + 128);   // [2][4]
    // places of the ring whose copies have landed, and (the producer's last
    // word) how many there will be
    const uint32_t landed_word = base + C::kMisc + 160;
    volatile int* total_places = reinterpret_cast<volatile int*>(smem + C::kMisc + 164);
    float2* stats = reinterpret_cast<float2*>(smem + C::kStats);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *total_places = -1;
        st_release_shared(landed_word, 0);
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), SEL ? 2 : 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(drain, 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(qfull0 + 8u * h, 1);
            mbar_init(qempty0 + 8u * h, 1);
            mbar_init(sfull0 + 8u * h, 1);
            mbar_init(pvdone0 + 8u * h, 1);
            mbar_init(group0 + 8u * h, 4);
            for (int w = 0; w < 4; ++w) ready[4 * h + w] = 0;
        }
        mbar_init(oempty, 8);
        mbar_init(altbar, 8);
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(itfull0 + 8u * i, 1);
            mbar_init(itempty0 + 8u * i, 9);
        }
        fence_mbar_init();
        tma_prefetch_map(&qmap);
        if (!SEL) {
            tma_prefetch_map(&kmap);
            tma_prefetch_map(&vmap);
        }
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    // what follows reads memory that the kernel before this one may have written
    allow_dependent_launch();
    grid_dependency_wait();
    const int sel_tiles = SEL ? (a.sel_k + kAttnTileKeys - 1) / kAttnTileKeys : 0;
    Start start = {0, 0, 0, 0, 0};
    const bool loads = warp == kLoadWarp || (SEL && warp == kGatherWarp);
    const bool lead = warp == kLoadWarp;
    if (loads) {
        if constexpr (SEL) {
            const int per_item = sel_tiles + kItemUnits;
            const long long total = (long long)a.tokens * a.kv_heads * per_item;
            const long long s0 = range_start(total, gridDim.x, blockIdx.x);
            start.left = range_start(total, gridDim.x, blockIdx.x + 1) - s0;
            const long long item = s0 / per_item;
            start.at = (int)(s0 - item * per_item);
            start.b = (int)(item / a.kv_heads);
            start.head = (int)(item - (long long)start.b * a.kv_heads);
        } else {
            // units per request in the ring's memory, which nobody else
            // touches before the copies begin
            static_assert(kAttnMaxBatch * 8 <= C::kStages * C::kStageBytes, "a number per request fits the ring");
            start = find_start(a, reinterpret_cast<long long*>(smem + C::kRing), lane);
            __syncwarp();
            fence_proxy_async_smem();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= kSoftmaxWarps) {
        regs_dec<kLowRegs>();
    if (loads) {
        // ------------------------------------------------------------ producer
        int b = start.b, head = start.head, tile = start.tile, at = start.at;
        long long left = start.left;                 // units left in the range
        int* piece = a.pieces + (long long)blockIdx.x * 2 * kPieceInts;
        if (lead && lane < 2) piece[lane * kPieceInts + kPcUsed] = 0;
        __syncwarp();

        int pos = 0;                 // places of the ring taken so far
        int handed = 0;              // selected: those whose copies are complete
        int item = 0;
        uint32_t qcount = 0;         // Q halves filled so far
        bool ok = true;
        int tok0 = 0, nq = 0, kv = 0, tiles = 0, cur_b = -1;
        auto next_item = [&]() {
            at = 0;
            if constexpr (SEL) {
                if (++head == a.kv_heads) { head = 0; ++b; }
            } else {
                if (++tile == tiles) {
                    tile = 0;
                    if (++head == a.kv_heads) { head = 0; ++b; }
                }
            }
        };
        while (left > 0 && ok) {
            if (!SEL && b >= a.batch) break;     // lengths changed under the call
            Span sp;
            int req;
            if constexpr (SEL) {
                req = __ldg(a.requests + b);
                bool fine = req >= 0 && req < a.batch;
                if (!fine) {
                    if (req >= a.batch && lane == 0) atomicOr(a.status, kStatusBadRequest);
                    req = 0;
                }
                kv = fine ? max(__ldg(a.kv_lens + req), 0) : 0;
                kv = (int)min((long long)kv, (long long)a.bt_width * kBlockKeys);
                sp.t0 = 0;
                sp.ntok = 1;
                sp.lo = 0;
                sp.hi = kv;
                sp.j0 = 0;
                sp.n = sel_tiles;
                sp.cost = 1;
                tok0 = b;
            } else {
                if (b != cur_b) {
                    request_of(a, b, tok0, nq, kv);
                    tiles = tiles_of(a, nq);
                    cur_b = b;
                    if (tiles == 0) { ++b; head = 0; tile = 0; at = 0; continue; }
                }
                req = b;
                sp = tile_span(a, nq, kv, tile);
            }
            // the tiles of this range: j .. j + n - 1
            const int j = tiles_before(sp, at);
            const int used = (int)min(left, (long long)(units_of(sp) - at));
            const int n = tiles_before(sp, at + used) - j;
            left -= used;
            const bool first = j == 0, last = j + n == sp.n;
            if (n == 0) {
                if (!last) break;                // the range ends in the item's own units
                next_item();
                continue;
            }
            const bool alt = SEL || sp.ntok <= a.half_tokens;
            const int slot = first ? 1 : 0;          // workspace slot of a piece
            // ---- the item's descriptor and Q rows
            const int is = item % kItemSlots;
            if (lead) ok = warp_wait(itempty0 + 8u * is, ((item / kItemSlots) & 1) ^ 1, abort_flag, a.status);
            if (!ok) break;
            const int j0 = sp.j0 + j;
            if (lead && lane == 0) {
                int* it = items + is * kItemInts;
                it[kItN] = n;
                it[kItJ0] = j0;
                it[kItFlags] = (alt ? kAlt : 0) | (first && last ? kWhole : 0);
                it[kItTok0] = tok0 + sp.t0;
                it[kItNtok] = sp.ntok;
                it[kItHead] = head;
                it[kItPos0] = kv - nq + sp.t0;
                it[kItKvHi] = (int)min((long long)kv, (long long)a.bt_width * kBlockKeys);
                it[kItLo] = sp.lo;
                it[kItHi] = sp.hi;
                it[kItSlot] = slot;
                if (!(first && last)) {
                    int* p = piece + slot * kPieceInts;
                    p[kPcUsed] = 1;
                    p[kPcTok0] = tok0 + sp.t0;
                    p[kPcNtok] = sp.ntok;
                    p[kPcHead] = head;
                    p[kPcLast] = last ? 1 : 0;
                }
                mbar_arrive(itfull0 + 8u * is);
            }
            // an item of one half takes the Q halves in turn, so its rows come
            // while the item before it is still at work
            for (int h = 0; lead && h < (alt ? 1 : 2) && ok; ++h, ++qcount) {
                const uint32_t qs = qcount & 1u;
                ok = warp_wait(qempty0 + 8u * qs, ((qcount >> 1) & 1u) ^ 1u, abort_flag, a.status);
                if (ok && lane == 0) {
                    const uint32_t fb = qfull0 + 8u * qs;
                    mbar_arrive_expect_tx(fb, (uint32_t)(C::kBlocks * 128 * a.group * a.half_tokens));
                    for (int kb = 0; kb < C::kBlocks; ++kb)
                        tma_load_3d(base + C::kQ + qs * C::kHalfBytes + kb * C::kBlockBytes, &qmap, fb,
                                    kb * 64, head * a.group, tok0 + sp.t0 + h * a.half_tokens);
                }
            }
            if (!ok) break;
            __syncwarp();
            ++item;

            // ---- K and V tiles: K runs `ahead` tiles before V
            const int ahead = alt ? 2 : 1;
            if constexpr (SEL) {
                const int32_t* list = a.selected + (long long)b * a.sel_stride;
                const int32_t* table = a.block_table + (long long)req * a.bt_stride;
                const int row0 = lead ? 0 : 64;
                // This lane's two rows of a tile (row0 + lane and 32 on), in
                // three steps a tile apart, so that no step waits for a load
                // of its own: the positions (-1: not there), their pages, the
                // rows' offsets in the cache.
                auto positions = [&](int t) {
                    const int i = (j0 + t) * kAttnTileKeys + row0 + lane;
                    int x = t < n && i < a.sel_k ? __ldg(list + i) : -1;
                    int y = t < n && i + 32 < a.sel_k ? __ldg(list + i + 32) : -1;
                    return make_int2(x < kv ? x : -1, y < kv ? y : -1);
                };
                auto pages = [&](int2 p) {
                    return make_int2(p.x >= 0 ? __ldg(table + (p.x >> 6)) : 0,
                                     p.y >= 0 ? __ldg(table + (p.y >> 6)) : 0);
                };
                auto settle = [&](int2& g) {
                    const bool bx = g.x < 0 || g.x >= a.num_pages, by = g.y < 0 || g.y >= a.num_pages;
                    if (bx || by) atomicOr(a.status, kStatusBadBlock);
                    if (bx) g.x = 0;
                    if (by) g.y = 0;
                };
                // the oldest tile whose copies are under way is handed over
                auto hand_over = [&]() {
                    switch (pos - handed - 1) {
                    case 0: cp_async_wait<0>(); break;
                    case 1: cp_async_wait<1>(); break;
                    case 2: cp_async_wait<2>(); break;
                    default: cp_async_wait<3>(); break;
                    }
                    fence_proxy_async_smem();     // the tensor core reads what this lane has copied
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full_bar(handed % S));
                    ++handed;
                };
                auto gather = [&](const void* cache, long long page_stride, long long slot_stride,
                                  long long head_stride, int2 p, int2 g) {
                    const int st = pos % S;
                    const uint32_t parity = (uint32_t)((pos / S) & 1) ^ 1u;
                    while (!__all_sync(0xffffffffu, mbar_test(empty_bar(st), parity))) {
                        // (a stage may wait for one that is still under way here)
                        if (handed < pos) {
                            hand_over();
                        } else {
                            if (!warp_wait(empty_bar(st), parity, abort_flag, a.status)) return false;
                            break;
                        }
                    }
                    // Four lanes copy a row, 64 bytes of it at a time, eight rows
                    // to an instruction: a lane needs the offset of one row in
                    // eight (told by the lane that looked it up), and all its
                    // addresses are constants away from two.  (Consecutive
                    // lanes' rows are four apart, so that their 16-byte chunks
                    // fall into different banks.)
                    const int sub = ((lane >> 2) & 1) * 4 + (lane >> 3), chunk = lane & 3;
                    const uint32_t dst0 = base + C::kRing + st * C::kStageBytes + (row0 + sub) * 128;
                    const uint32_t to[2] = {dst0 + ((chunk ^ sub) << 4), dst0 + (((chunk + 4) ^ sub) << 4)};
                    const uint16_t* src0 = static_cast<const uint16_t*>(cache) + head * head_stride + chunk * 8;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int at = half ? p.y : p.x, page = half ? g.y : g.x;
                        const long long off = at < 0 ? -1 : page * page_stride + (at & 63) * slot_stride;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const long long o = __shfl_sync(0xffffffffu, off, 8 * i + sub);
                            const uint16_t* src = src0 + max(o, 0ll);
                            const uint32_t bytes = o < 0 ? 0u : 16u;
#pragma unroll
                            for (int c = 0; c < D / 32; ++c)
                                cp_async16(to[c & 1] + (c >> 1) * C::kBlockBytes + (32 * half + 8 * i) * 128,
                                           src + 32 * c, bytes);
                        }
                    }
                    cp_async_commit();
                    ++pos;
                    if (pos - handed > min(3, S - 2)) hand_over();
                    return true;
                };
                // tile nk's rows (settled), the two tiles' after it on their
                // way, and those of the one or two tiles whose K is in and V
                // is not
                int2 p0 = positions(0), p1 = positions(1), p2 = positions(2);
                int2 g0 = pages(p0), g1 = pages(p1);
                int2 vp0 = {}, vg0 = {}, vp1 = {}, vg1 = {};
                settle(g0);
#pragma unroll 1
                for (int nk = 0, nv = 0; nv < n && ok;) {
                    const bool is_k = nk < n && nk - nv < ahead;
                    ok = gather(is_k ? a.k_cache : a.v_cache, is_k ? a.k_page : a.v_page,
                                is_k ? a.k_slot : a.v_slot, is_k ? a.k_head : a.v_head, is_k ? p0 : vp0,
                                is_k ? g0 : vg0);
                    if (is_k) {
                        if (nk == nv) { vp0 = p0; vg0 = g0; }
                        else { vp1 = p0; vg1 = g0; }
                        ++nk;
                        p0 = p1; g0 = g1; settle(g0);
                        p1 = p2; g1 = pages(p1);
                        p2 = positions(nk + 2);
                    } else {
                        vp0 = vp1; vg0 = vg1;
                        ++nv;
                    }
                }
                // (what is under way is handed over with the next item's
                // first tiles, or at the end)
            } else {
                const int32_t* table = a.block_table + (long long)req * a.bt_stride;
                // pages with visible keys; others are neither looked up nor read
                const int page_begin = sp.lo / kBlockKeys;
                const int page_end = (sp.hi + kBlockKeys - 1) / kBlockKeys;
                int win = -1, entry = 0;       // 32 table entries from page `win` on, one a lane
                auto pages = [&](int t, int& g0, int& g1, int& want) {
                    const int p = 2 * (j0 + t);
                    if (win < 0 || p >= win + 32) {
                        win = p;
                        long long g = p + lane >= page_begin && p + lane < page_end ? __ldg(table + p + lane) : 0;
                        if (g < 0 || g >= a.num_pages) {
                            atomicOr(a.status, kStatusBadBlock);
                            g = 0;
                        }
                        entry = (int)g;
                    }
                    g0 = __shfl_sync(0xffffffffu, entry, p - win);
                    g1 = __shfl_sync(0xffffffffu, entry, p - win + 1);
                    want = (p >= page_begin && p < page_end ? 1 : 0) | (p + 1 < page_end ? 2 : 0);
                };
                // pages of tile nk's K, and of the one or two tiles whose K is
                // in and V is not
                int x = 0, y = 0, c = 0, x0 = 0, y0 = 0, c0 = 0, x1 = 0, y1 = 0, c1 = 0;
#pragma unroll 1
                for (int nk = 0, nv = 0; nv < n && ok;) {
                    const bool is_k = nk < n && nk - nv < ahead;
                    if (is_k) {
                        pages(nk, x, y, c);
                        if (nk == nv) { x0 = x; y0 = y; c0 = c; }
                        else { x1 = x; y1 = y; c1 = c; }
                        ++nk;
                    } else {
                        x = x0; y = y0; c = c0;
                        x0 = x1; y0 = y1; c0 = c1;
                        ++nv;
                    }
                    const int st = pos % S;
                    ok = warp_wait(empty_bar(st), (uint32_t)((pos / S) & 1) ^ 1u, abort_flag, a.status);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(full_bar(st), (uint32_t)(__popc(c) * C::kBlocks * 8192));
                    __syncwarp();
                    const int pg = lane / C::kBlocks, kb = lane - pg * C::kBlocks;
                    if (pg < 2 && ((c >> pg) & 1))
                        tma_load_4d(base + C::kRing + st * C::kStageBytes + kb * C::kBlockBytes + pg * 8192,
                                    is_k ? &kmap : &vmap, full_bar(st), kb * 64, 0, head, pg ? y : x);
                    ++pos;
                }
            }
            if (last) next_item();
        }
        if constexpr (SEL) {
            for (; handed < pos; ++handed) {
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full_bar(handed % S));
            }
        }
        if (lead) {
            if (ok) {
                const int is = item % kItemSlots;
                ok = warp_wait(itempty0 + 8u * is, ((item / kItemSlots) & 1) ^ 1, abort_flag, a.status);
                if (ok && lane == 0) {
                    items[is * kItemInts + kItFlags] = kEnd;
                    mbar_arrive(itfull0 + 8u * is);
                }
            }
            if (lane == 0) *total_places = pos;
            // copies in flight land before the CTA may leave
            for (int t = pos > S ? pos - S : 0; t < pos; ++t)
                mbar_wait_drain<false>(full_bar(t % S), (uint32_t)((t / S) & 1));
            for (uint32_t c = qcount > 2 ? qcount - 2 : 0; c < qcount; ++c)
                mbar_wait_drain<false>(qfull0 + 8u * (c & 1u), (c >> 1) & 1u);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        // One thread, which issues about as fast as the tensor core computes:
        // whatever else it does, the tensor core waits for.  An mbarrier wait
        // costs it some 230 cycles even when the phase is over and a commit
        // 130, so in the loop over tiles there is one commit per product
        // pair, "scores ready", which covers the products before it (stages
        // and O are released by the softmax groups when they see it), and
        // stages and P are announced by plain words in shared memory.
        if (lane == 0) {
            constexpr uint32_t kFmt = FP16 ? 0u : 1u;
            constexpr uint32_t idesc_s = make_idesc(kFmt, kFmt, 128, 128);
            constexpr uint32_t idesc_o = make_idesc(kFmt, kFmt, 128, D) | (1u << 16);   // B transposed
            const uint64_t q_desc = smem_desc_sw128(base + C::kQ);
            const uint64_t k_desc = smem_desc_sw128(base + C::kRing);
            const uint64_t v_desc = desc_mn_sw128(base + C::kRing, C::kBlockBytes);
            uint32_t stage = 0;                  // of the next place of the ring
            uint32_t place = 0;                  // places consumed
            uint32_t qcount = 0;                 // Q halves used
            uint32_t pcount0 = 0, pcount1 = 0;   // P tiles consumed of each half
            bool ok = true, skip = false;
            auto wait = [&](uint32_t b, uint32_t parity) {
                return mbar_wait<false>(b, parity, abort_flag, a.status);
            };
            auto take = [&]() {
                const uint32_t st = stage;
                if (++stage == S) stage = 0;
                ++place;
                return st;
            };
            auto issue_s = [&](int h, uint64_t ad, uint32_t st) {
                const uint64_t bd = k_desc + st * (uint32_t)(C::kStageBytes >> 4);
#pragma unroll
                for (int kb = 0; kb < C::kBlocks; ++kb)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(tmem + kColS + 128u * h, ad + (uint32_t)(kb * (C::kBlockBytes >> 4) + 2 * k),
                                bd + (uint32_t)(kb * (C::kBlockBytes >> 4) + 2 * k), idesc_s,
                                (kb | k) ? 1u : 0u);
                mma_commit(sfull0 + 8u * h);
            };
            auto issue_pv = [&](int h, uint32_t st, bool acc) {
                tc_fence_after();
                if (skip) return;                // the group has added this tile itself
                const uint64_t bd = v_desc + st * (uint32_t)(C::kStageBytes >> 4);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_tmem_a(tmem + kColO + 128u * h, tmem + kColS + 128u * h + 8u * k,
                                   bd + (uint32_t)(k * (2048 >> 4)), idesc_o, (acc || k) ? 1u : 0u);
            };
            // places below `place` have landed, and (words != 0) a half's P number `count`
            auto wait_words = [&](uint32_t words, uint32_t count) {
                return words_ready(landed_word, place, words, count, skip, abort_flag, a.status);
            };
            for (int item = 0; ok; ++item) {
                const int is = item % kItemSlots;
                ok = wait(itfull0 + 8u * is, (item / kItemSlots) & 1);
                if (!ok) break;
                const volatile int* it = items + is * kItemInts;
                const int flags = it[kItFlags], n = it[kItN];
                mbar_arrive(itempty0 + 8u * is);
                if (flags & kEnd) break;
                const bool alt = flags & kAlt;
                const uint32_t q0 = qcount & 1u;             // Q halves of this item
                for (int i = alt ? 1 : 0; i < 2 && ok; ++i, ++qcount)
                    ok = wait(qfull0 + 8u * (qcount & 1u), (qcount >> 1) & 1u);
                if (!alt) {
                    // both halves see every tile; written out, since with
                    // these items the tensor core's time is what counts
                    uint32_t ks = take(), vs = 0;
                    const uint64_t ad0 = q_desc + q0 * (uint32_t)(C::kHalfBytes >> 4);
                    const uint64_t ad1 = q_desc + (q0 ^ 1u) * (uint32_t)(C::kHalfBytes >> 4);
                    ok = ok && wait_words(0u, 0u);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(0, ad0, ks);
                    issue_s(1, ad1, ks);
                    ok = wait(oempty, (uint32_t)(item & 1) ^ 1u);
#pragma unroll 1
                    for (int t = 0; t < n && ok; ++t) {
                        const bool more = t + 1 < n;
                        vs = take();
                        if (more) ks = take();
                        ok = wait_words(ready0, ++pcount0);
                        if (!ok) break;
                        issue_pv(0, vs, t > 0);
                        if (more) issue_s(0, ad0, ks);
                        else mma_commit(pvdone0);
                        ok = wait_words(ready0 + 16u, ++pcount1);
                        if (!ok) break;
                        issue_pv(1, vs, t > 0);
                        if (more) issue_s(1, ad1, ks);
                        else mma_commit(pvdone0 + 8u);
                    }
                } else {
                    // the halves take the tiles in turn; two steps of scores
                    // alone, then each the product with V of a tile and the
                    // scores of the half's next (one copy of the code: these
                    // items are short or wait for memory)
                    const uint64_t ad = q_desc + q0 * (uint32_t)(C::kHalfBytes >> 4);
                    uint32_t ks = 0, vs = 0;
#pragma unroll 1
                    for (int t = -2; t < n && ok; ++t) {
                        const int h = t & 1;
                        const bool more = t + 2 < n;
                        if (t >= 0) vs = take();
                        if (more) ks = take();
                        if (t == 0) ok = wait(oempty, (uint32_t)(item & 1) ^ 1u);
                        if (t >= 0) {
                            if (h) ++pcount1;
                            else ++pcount0;
                        }
                        ok = ok && (t >= 0 ? wait_words(ready0 + 16u * h, h ? pcount1 : pcount0) : wait_words(0u, 0u));
                        if (!ok) break;
                        tc_fence_after();
                        if (t >= 0) issue_pv(h, vs, t > 1);
                        if (more) issue_s(h, ad, ks);
                        else if (t >= 0) mma_commit(pvdone0 + 8u * h);
                    }
                }
            }
            // every MMA and every arrival it owes is through before the CTA leaves
            mma_commit(drain);
            mbar_wait_drain<false>(drain, 0);
        }
        __syncwarp();
    } else if (warp == kLandWarp) {
        // ------------------------------------------------------------ landed stages
        // Counts, in order, the places of the ring whose copies have landed.
        // It ends with the producer's last place, or with an abort (every
        // other role's waits are bounded and raise it).
        if (lane == 0) {
            for (int pos = 0;; ) {
                if (mbar_try_wait_suspend(full_bar(pos % S), (uint32_t)((pos / S) & 1), kWaitSuspendNs)) {
                    ++pos;
                    st_release_shared(landed_word, (uint32_t)pos);
                } else if (*total_places == pos || *abort_flag) {
                    break;
                }
            }
        }
        __syncwarp();
    }
    } else {
        regs_inc<kHighRegs>();
        // ------------------------------------------------------------ softmax
        const int h = warp >> 2;                 // half
        const int quad = warp & 3;
        const int row = quad * 32 + lane;        // row of the half = TMEM lane
        const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = lane_addr + kColS + 128u * h;
        const uint32_t t_o = lane_addr + kColO + 128u * h;
        const float c = a.scale_log2;
        const int G = a.group;
        const int row_tok = row / G;
        const int row_head = row - row_tok * G;
        uint32_t qcount = 0, scount = 0, pvcount = 0, done_phase = 0, group_phase = 0, alt_phase = 0;
        int pos_base = 0;
        bool ok = true;
        for (int item = 0; ok; ++item) {
            const int is = item % kItemSlots;
            ok = warp_wait(itfull0 + 8u * is, (item / kItemSlots) & 1, abort_flag, a.status);
            if (!ok) break;
            // (read again where they are needed: the slot is released at the
            // item's end, and the registers are the row of S's)
            const volatile int* it = items + is * kItemInts;
            if (it[kItFlags] & kEnd) break;
            const bool alt = it[kItFlags] & kAlt;
            const int n = it[kItN], j0 = it[kItJ0];
            const int half_tok0 = alt ? 0 : h * a.half_tokens;
            const int half_ntok = min(a.half_tokens, it[kItNtok] - half_tok0);
            const bool valid = row_tok < half_ntok;
            // warps without a valid row have nothing to compute
            const bool active = quad * 32 < half_ntok * G;
            // keys that this row may see, and the range that all rows see
            int row_lo = it[kItLo], row_hi = it[kItHi], all_lo = row_lo, all_hi = row_hi;
            if constexpr (!SEL) {
                const int kv_hi = it[kItKvHi];
                const int p_first = it[kItPos0] + half_tok0, p_last = p_first + half_ntok - 1;
                const int p_row = p_first + row_tok;
                if (a.causal) {
                    row_hi = min(kv_hi, p_row + 1);
                    all_hi = min(kv_hi, p_first + 1);
                }
                if (a.window > 0) {
                    row_lo = p_row < a.window ? 0 : p_row - a.window + 1;
                    all_lo = p_last < a.window ? 0 : p_last - a.window + 1;
                }
            }
            const int tiles_here = alt ? (n + 1 - h) / 2 : n;
            float m = -INFINITY, l = 0.0f;
            int v_place = 0;                     // of the last tile's V
            for (int i = 0; i < tiles_here && ok; ++i) {
                const int t = alt ? 2 * i + h : i;
                const int key0 = (j0 + t) * kAttnTileKeys;
                // selected: which of the 128 entries are there (bit k / 4 of word k % 4)
                uint32_t there[4] = {0, 0, 0, 0};
                if constexpr (SEL) {
                    const int32_t* list = a.selected + (long long)it[kItTok0] * a.sel_stride;
                    const int item_hi = it[kItHi];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = key0 + 4 * lane + e;
                        const int p = at < a.sel_k ? __ldg(list + at) : -1;
                        there[e] = __ballot_sync(0xffffffffu, p >= 0 && p < item_hi);
                    }
                }
                ok = warp_wait(sfull0 + 8u * h, scount & 1, abort_flag, a.status);
                if (!ok) break;
                ++scount;
                tc_fence_after();
                // the scores' commit covers every product issued before it:
                // this tile's K has been read, and the V and P of this half's
                // last tile (of both halves' where they share it, since half 1
                // comes second)
                if ((alt || h == 1) && threadIdx.x % 128 == 96) {
                    const int kp = pos_base + (t < (alt ? 2 : 1) ? t : 2 * t - (alt ? 1 : 0));
                    mbar_arrive(empty_bar(kp % S));
                    if (i > 0) mbar_arrive(empty_bar(v_place % S));
                    if (t == n - 1) {
                        mbar_arrive(qempty0 + 8u * (qcount & 1u));
                        if (!alt) mbar_arrive(qempty0 + 8u * (~qcount & 1u));
                    }
                }
                v_place = pos_base + t + min(n, t + (alt ? 2 : 1));
                bool masked;
                if constexpr (SEL) masked = (there[0] & there[1] & there[2] & there[3]) != 0xffffffffu;
                else masked = key0 < all_lo || all_hi - key0 < kAttnTileKeys;

                if (active) {
                    // bit k % 32 of word k / 32 (selected: k / 4 of k % 4): key k is shown
                    uint32_t shown[4];
                    if constexpr (SEL) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) shown[e] = there[e];
                    } else if (masked) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int lo = min(max(row_lo - key0 - 32 * e, 0), 32);
                            const int hi = min(max(row_hi - key0 - 32 * e, 0), 32);
                            shown[e] = lo < hi ? (0xffffffffu >> (32 - hi + lo)) << lo : 0u;
                        }
                    }
                    uint32_t x[4][32];
                    auto load = [&]() {
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_ld32_async(t_s + 32 * q, x[q]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_wait_bind32(x[q]);
                        if (masked) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if (!SEL && __all_sync(0xffffffffu, shown[q] == 0xffffffffu)) continue;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const uint32_t w = SEL ? shown[k & 3] >> (8 * q + (k >> 2)) : shown[q] >> k;
                                    if (!(w & 1u)) x[q][k] = 0xff800000u;    // -inf
                                }
                            }
                        }
                    };
                    load();
                    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 128; k += 2)
                        t[(k >> 1) & 3] = fmaxf(t[(k >> 1) & 3], fmaxf(__uint_as_float(x[k >> 5][k & 31]),
                                                                       __uint_as_float(x[k >> 5][(k & 31) + 1])));
                    // a new reference when the old one is too low by 2^8
                    const float m_new = fmaxf(m, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])));
                    const bool grow = valid && (m_new - m) * c > 8.0f;   // m = -inf: yes unless m_new is
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? exp2_approx((m - m_new) * c) : 1.0f;
                        if (grow) m = m_new;
                        l *= f;
                        // eight columns at a time: the row of S stays in registers
#pragma unroll 1
                        for (int d = 0; i > 0 && d < D; d += 8) {
                            float o[8];
                            tmem_ld8(t_o + d, o);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] *= f;
                            tmem_st8(t_o + d, o);
                        }
                    }
                    // c x - c m in one fused product and sum: c m is rounded
                    // once, a factor that all of the row shares but the next
                    // reference and the other pieces do not, 2^-15 for |c m| up
                    // to 2^10.  Past that the difference is taken first, in
                    // tensor memory.
                    float mc = m == -INFINITY ? 0.0f : m * c;
                    if (__any_sync(0xffffffffu, fabsf(mc) > 1024.0f)) {
                        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
                        for (int k = 0; k < 128; ++k)
                            x[k >> 5][k & 31] = __float_as_uint(__uint_as_float(x[k >> 5][k & 31]) - ref);
                        mc = 0.0f;
                    }
                    const float shift = PScale<FP16>::kLog2 - mc;
                    const uint64_t cc = pack2(c, c), nm = pack2(shift, shift);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t(&y)[32] = x[q];
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint64_t v =
                                fma2(pack2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), cc, nm);
                            float lo, hi;
                            unpack2(v, lo, hi);
                            lo = exp2_approx(lo);
                            hi = exp2_approx(hi);
                            sum[e & 1] = add2(sum[e & 1], pack2(lo, hi));
                            p[e] = pack16<FP16>(lo, hi);
                        }
                        tmem_st16(t_s + 16 * q, p);
                    }
                    l += sum2(add2(sum[0], sum[1]));
                    tmem_wait_st();
                }
                // V rows that must not count (selected ones came as zeros)
                bool added = false;             // this tile's product is in O already
                if (!SEL && masked) {
                    const int vs = v_place % S;
                    // (the parity of v_place cannot be an older one's: these
                    // scores were issued after place v_place - S was consumed)
                    ok = warp_wait(full_bar(vs), (uint32_t)((v_place / S) & 1), abort_flag, a.status);
                    if (!ok) break;
                    uint8_t* vt = smem + C::kRing + vs * C::kStageBytes;
                    // thread = key of the tile
                    const int key = key0 + row;
                    const int item_lo = it[kItLo], item_hi = it[kItHi];
                    const bool none = key < item_lo || key >= item_hi;    // no row of the item sees it
                    const bool some = !none && (key < all_lo || key >= all_hi);    // some rows of this half do not
                    if (none) {
#pragma unroll
                        for (int e = 0; e < 8 * C::kBlocks; ++e)
                            *reinterpret_cast<uint4*>(vt + (e >> 3) * C::kBlockBytes + row * 128 +
                                                      (((e + row) & 7) << 4)) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();     // the tensor core reads it
                    }
                    // (a tile with such keys, the same for all of the half)
                    if (max(key0, item_lo) < all_lo || (item_hi > all_hi && all_hi - key0 < kAttnTileKeys)) {
                        bool bad = false;
                        if (some) {
#pragma unroll 2
                            for (int e = 0; e < 8 * C::kBlocks; ++e) {
                                const uint4 w = *reinterpret_cast<const uint4*>(
                                    vt + (e >> 3) * C::kBlockBytes + row * 128 + (((e + row) & 7) << 4));
                                bad |= not_finite<FP16>(w.x) || not_finite<FP16>(w.y) ||
                                       not_finite<FP16>(w.z) || not_finite<FP16>(w.w);
                            }
                        }
                        const bool any_bad = __any_sync(0xffffffffu, bad);
                        const int par = group_phase & 1;
                        if (lane == 0) {
                            votes[(h * 2 + par) * 4 + quad] = any_bad ? 1 : 0;
                            mbar_arrive(group0 + 8u * h);
                        }
                        ok = warp_wait(group0 + 8u * h, group_phase & 1, abort_flag, a.status);
                        if (!ok) break;
                        ++group_phase;
                        const volatile int* v4 = votes + (h * 2 + par) * 4;
                        if (v4[0] | v4[1] | v4[2] | v4[3]) {
                            // this tile's product, row by row over the keys it
                            // may see (P as the tensor core would read it).  O
                            // is this item's once both groups have read the
                            // last one's, which the issuer waits for before its
                            // own first product
                            if (i == 0) {
                                ok = warp_wait(oempty, (uint32_t)(item & 1) ^ 1u, abort_flag, a.status);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            if (active) {
                                const int lo = row_lo - key0, hi = row_hi - key0;
#pragma unroll 1
                                for (int d = 0; d < D; d += 8) {
                                    float acc[8];
                                    tmem_ld8(t_o + d, acc);
                                    if (i == 0)
#pragma unroll
                                        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
                                    const uint8_t* col = vt + (d >> 6) * C::kBlockBytes;
#pragma unroll 1
                                    for (int k = 0; k < 128; k += 2) {
                                        const float2 p = unpack16<FP16>(tmem_ld1(t_s + (k >> 1)));
#pragma unroll
                                        for (int b = 0; b < 2; ++b) {
                                            const int kk = k + b;
                                            if (kk < lo || kk >= hi) continue;
                                            const uint4 w = *reinterpret_cast<const uint4*>(
                                                col + kk * 128 + ((((d & 63) >> 3) ^ (kk & 7)) << 4));
                                            const float pk = b ? p.y : p.x;
                                            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                            for (int e = 0; e < 4; ++e) {
                                                const float2 vv = unpack16<FP16>(ww[e]);
                                                acc[2 * e] += pk * vv.x;
                                                acc[2 * e + 1] += pk * vv.y;
                                            }
                                        }
                                        __syncwarp();
                                    }
                                    tmem_st8(t_o + d, acc);
                                }
                                tmem_wait_st();
                            }
                            added = true;
                        }
                    }
                }
                // (P is in place: its stores were waited for)
                __syncwarp();
                ++pvcount;
                if (lane == 0) st_release_shared(ready0 + 16u * h + 4u * quad, 2u * pvcount + (added ? 1u : 0u));
            }
            if (!ok) break;
            pos_base += 2 * n;
            qcount += alt ? 1u : 2u;

            // ---------------------------------------------------- the item's end
            if (tiles_here > 0) {
                ok = warp_wait(pvdone0 + 8u * h, done_phase, abort_flag, a.status);
                if (!ok) break;
                done_phase ^= 1;
                if ((alt || h == 1) && threadIdx.x % 128 == 96) mbar_arrive(empty_bar(v_place % S));
            }
            tc_fence_after();
            const bool whole = it[kItFlags] & kWhole;
            float top = m, sum = l, g0 = 1.0f, g1 = 0.0f;
            if (alt) {
                // both halves hold these rows: they join, and group h writes
                // columns h D / 2 .. of the result
                // (A group without a tile, h = 1 where n = 1, leaves nothing: it may
                // be here while the other one still reads what it left for the item
                // before.  One that had a tile has seen its product end, which
                // began after both groups' ends of that item.)
                if (tiles_here > 0) stats[h * 128 + row] = make_float2(m, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(altbar);
                ok = warp_wait(altbar, alt_phase & 1, abort_flag, a.status);
                if (!ok) break;
                ++alt_phase;
                tc_fence_after();
                const float2 s0 = stats[row];
                const float2 s1 = n > 1 ? stats[128 + row] : make_float2(-INFINITY, 0.0f);
                top = fmaxf(s0.x, s1.x);
                g0 = s0.x == -INFINITY ? 0.0f : exp2_approx((s0.x - top) * c);
                g1 = s1.x == -INFINITY ? 0.0f : exp2_approx((s1.x - top) * c);
                sum = s0.y * g0 + s1.y * g1;
            }
            if (active) {
                if (whole) {
                    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
                    g0 *= inv;
                    g1 *= inv;
                }
                const int token = it[kItTok0] + half_tok0 + row_tok;
                const int qhead = it[kItHead] * G + row_head;
                const long long ws_row = ((long long)blockIdx.x * 2 + it[kItSlot]) * kAttnSlotRows +
                                         (alt ? 0 : h * kAttnHalfRows) + row;
                uint16_t* orow = static_cast<uint16_t*>(a.out) + (long long)token * a.out_token +
                                 (long long)qhead * a.out_head;
                // partial results lie column by column (four at a time): the
                // rows of a warp are neighbours
                float* prow = a.partial + partial_at<D>(blockIdx.x, it[kItSlot], 0, (alt ? 0 : h * kAttnHalfRows) + row);
                const bool both = alt && n > 1;          // half 1 saw a tile, too
                const uint32_t o0 = alt ? lane_addr + kColO : t_o;
                const int d_end = alt ? (h + 1) * (D / 2) : D;
#pragma unroll 1
                for (int d = alt ? h * (D / 2) : 0; d < d_end; d += 16) {
                    uint32_t o[16], u[16];
                    tmem_ld16_async(o0 + d, o);
                    if (both) tmem_ld16_async(lane_addr + kColO + 128u + d, u);
                    tmem_wait_bind16(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * g0);
                    if (both) {
                        tmem_wait_bind16(u);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(u[e]), g1, __uint_as_float(o[e])));
                    }
                    if (valid && whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack16<FP16>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                        uint4* dst = reinterpret_cast<uint4*>(orow + d);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else if (valid) {
                        uint4* dst = reinterpret_cast<uint4*>(prow) + (d >> 2) * kAttnSlotRows;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e * kAttnSlotRows] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
                if (valid && (h == 0 || !alt)) {
                    if (!whole) a.stats[ws_row] = make_float2(top, sum);
                    else if (a.lse != nullptr)
                        a.lse[(long long)token * a.kv_heads * G + qhead] =
                            sum == 0.0f ? -INFINITY : top * a.scale + logf(sum * PScale<FP16>::kInverse);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(oempty);
                mbar_arrive(itempty0 + 8u * is);
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool FP16, bool SEL>
cudaError_t launch_kernel(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    auto kernel = paged_attention_kernel<D, FP16, SEL>;
    static int configured_device = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_device != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kTotal);
        if (e != cudaSuccess) return e;
        // the warpgroups' shares must fit the block's allocation, else the
        // softmax groups' setmaxnreg.inc would wait forever
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs || 2 * kHighRegs + kLowRegs > 3 * kLaunchRegs)
            return cudaErrorInvalidConfiguration;
        configured_device = dev;
    }
    return launch_dependent(kernel, dim3((unsigned)num_ctas), kThreads, Cfg<D>::kTotal, stream, qmap, kmap,
                            vmap, a);
}

}  // namespace attn
}  // namespace pml
