// Attention of new tokens over K/V caches held in 4 bits, on sm_103a.
//
//   out[t, h] = sum_p softmax_p(scale * q[t, h] . k_p) v_p
//
// over values code * s * g (codes E2M1, s the E4M3 scale of sixteen values, g
// the cache's power of two) and the positions p that token t may see: those of
// its request up to its own (causal), past position - window (window > 0), or
// the ones a list names.  code * s has at most six significant bits and lies
// between 2^-10 and 2688: exact in fp16, the type of both products.  One pass
// with a running maximum m and sum l: P = 2^(c (S - m) + 7), O += P V, rescaled
// only when c m has grown by more than 8.
//
// What it is bound by.  A row of 128 values is 72 bytes, read once for 8 or 16
// query rows: at HBM's rate an SM gets a key and its value every 6.5 cycles.
// The tensor work is a fiftieth of what the tensor core could do in that time;
// turning codes into fp16 is what takes instructions, so the codes go straight
// from shared memory into the operand registers of the warp's own matrix
// instructions.  (Operands of the larger tensor-core instruction lie in shared
// memory: its tiles would have to be written there and read again, four times
// the bytes of the codes, with a hand-over for each tile.)
//
// Warps work alone.  An item is 8 or 16 rows ((token, head) pairs that share a
// kv head) and the keys they see, in steps of 32.  The steps of all items, in
// order, are cut into one contiguous range per warp.  A warp copies its keys'
// codes and scales into a ring of its own (cp.async, a few steps ahead) and
// waits for nobody.  Pieces of items that several warps of a CTA shared are
// joined at the CTA's end, those of several CTAs by a second kernel; all in a
// fixed order.  One request, or lists, which are equally long, may have a
// cluster of CTAs for each item instead, which joins its pieces itself.
//
// Operands (m16n8k16; g = lane / 4, t = lane % 4), eight rows of Q at a time:
//   S^T = K Q^T   K is A, 16 keys.  The order of the summed elements is free, so
//               lane t takes elements (D/4) t .. of every row: of a key 16 (8)
//               bytes in one load, two (one) scales
//   O^T = V^T P^T   V^T is A: its rows are elements, lane g takes (D/8) g .. of
//               a value, one scale; its columns are keys, two to a register:
//               the nibbles of two keys are interleaved into bytes before they
//               are converted.  P^T is B: S^T's fragments, transposed between
//               lanes (movmatrix)
// Key c of eight is row (c / 2) + 4 (c & 1): with K's rows stored in that order
// and V's 16-byte chunks swapped in every other pair of rows all loads are free
// of bank conflicts.  (Q as A, which leaves P as B without the transposition,
// takes twice the instructions for eight rows: 16 of Q's are not there.)
//
// Masked places never reach a result, whatever they hold: their scores are
// -inf; rows outside the item's keys are zeros in shared memory; and in a step
// that some rows see in part, values under a NaN scale are taken out of the
// product and put into the rows that see them.
//
// Measured (heads of 128, a copy reaches 6794 GB/s):
//   64 single tokens over U[1024, 32768] keys, 64 heads over 8, bf16
//       225 us, 1.33 GB: 87 % of the copy.  A third of it under the profiler:
//       instructions issued in 66 % of the cycles, the ALU busy in 54 %, HBM
//       5.2 TB/s.  (Q as A 370 us; with spilled registers 310)
//   16 requests x 8 kv heads over 8500 keys each, 8 rows of q to a head 44 us, 16
//       rows 54, 24 and 32 rows 90 (21 for the bytes alone).  With 16
//       rows a scheduler has three warps, issues in 46 % of the cycles, and its
//       matrix unit is as busy: latencies within a step, which more warps (of 128
//       registers: spills) or items of 32 rows (255 registers, two warps a
//       scheduler: 88 -> 91) do not shorten.  (168 registers are all in use then:
//       64 bytes of stack, 196 of spill stores; lists 56 and 68)
//   31 requests of 4 tokens over up to 16000 keys, 28 / 4 heads: 85 us, a floor of
//       21, two items of 14 rows to a key.  (Fourteen warps: 114)
//   64 tokens x 500 listed positions, 64 heads over 1: 17.7 us, a floor of 0.8; two
//       steps a warp after a fixed part of 10 us
//   one token, 4000 keys, 32 heads over 8
//       12.2 us, eight CTAs to a kv head (15.2 cut over all, with the second
//       kernel, as it also is under a table of more than about 110 pages): a
//       launch, first copies and Q 3, joined in the CTA 3-5
// Steps are of 32 keys, a whole number of times in a page: an item's end costs
// half of what steps of 64 would waste.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dependent.cuh"
#include "nvfp4_cache.h"
#include "ptx.cuh"

namespace pml {
namespace nvattn {

constexpr int kStepKeys = 32;
// Units of work: a step is one, beginning and ending an item three.
constexpr int kItemUnits = 3;
// P = 2^(c (S - m) + 7): 2^7 times the weights, so that fp16 keeps the small ones'
// bits, up to 2^15 before a larger maximum moves m.
constexpr float kPLog2 = 7.0f, kPMost = 15.0f;
// c S - c m is one fused product and sum while |c m| is below this (c m is
// rounded once, to 2^-14); past it the difference is taken first.
constexpr float kFar = 1024.0f;

// a piece's record
enum { kPcUsed, kPcTok0, kPcNtok, kPcHead, kPcHeads, kPcLast };
constexpr int kPcInts = 8;

// NT: groups of eight rows in an item, one or two.  With two, Q lies in shared
// memory.
template <int D, int NT>
struct Cfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kWarps = NT == 1 ? 16 : 12;       // 128 or 168 registers a thread
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCode = D / 2, kScale = D / 16;   // bytes of a row
    static constexpr int kStageBytes = 2 * kStepKeys * (kCode + kScale);
    static constexpr int kStages = D == 128 ? (NT == 1 ? 3 : 2) : 5;
    static constexpr int kRing = kStages * kStageBytes;    // of a warp
    static constexpr int kQ = kWarps * kRing;
    static constexpr int kQBytes = NT == 1 ? 0 : kRows * D * 2;    // of a warp
    static constexpr int kMasks = kQ + kWarps * kQBytes;   // uint32 [kWarps][8]
    static constexpr int kSums = kMasks + kWarps * 32;     // long long [kWarps]
    static constexpr int kRecs = kSums + kWarps * 8;       // pieces of the CTA
    static constexpr int kPieces = kRecs + kWarps * 8;     // int [kWarps][2][kPcInts]
    static constexpr int kTotal = kPieces + kWarps * 2 * kPcInts * 4;
    static_assert(kTotal <= 232448, "shared memory of a CTA");
    static_assert(kAttnMaxBatch * 8 <= kMasks, "a number per request fits the ring and Q");
    static_assert(kRows * (D * 4 + 8) <= kRing, "a piece fits the ring");
};

// Where pieces lie: those of warps (slot 0 alone has rows here: slot 1, and the
// last piece of a warp, stay in shared memory) and those of CTAs.
struct Pieces {
    int* rec;          // [n][2][kPcInts], of CTAs' pieces
    float2* stats;     // [n][slots][rows] (maximum, sum)
    float* part;       // [n][slots][rows][D]
};

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi)
{
    uint32_t r;
    if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// c += A B, A 16 x 16 and B 16 x 8 in fp16
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bytes, or zeros (bytes = 0: src is not read).
template <int N>
__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void* src, uint32_t bytes)
{
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "n"(N)
                     : "memory");
}

// The same with c = 0 before.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// An 8 x 8 matrix of 16-bit elements, lane (g, t) holding row g's elements 2 t
// and 2 t + 1, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Two E4M3 codes (low byte -> low half) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

// ------------------------------------------------------------------ items

__device__ __forceinline__ void request_of(const NvAttnArgs& a, int b, int& tok0, int& nq, int& kv)
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

// The tokens of tile `tile` of a request with nq new tokens of kv, and the keys
// that some of them may see.
struct Span {
    int t0, ntok;
    int lo, hi;
    int j0, n;       // steps
};

__device__ __forceinline__ Span span_of(const NvAttnArgs& a, int nq, int kv, int tile)
{
    Span s;
    s.t0 = tile * a.tile_tokens;
    s.ntok = min(a.tile_tokens, nq - s.t0);
    const long long there = min((long long)kv, (long long)a.bt_width * kBlockKeys);
    const long long pos0 = (long long)kv - nq + s.t0;      // position of the tile's first token
    long long hi = there, lo = 0;
    if (a.causal) hi = min(hi, pos0 + s.ntok);
    if (a.window > 0) lo = max(lo, pos0 - a.window + 1);
    if (hi <= lo) { hi = 0; lo = 0; }
    s.lo = (int)lo;
    s.hi = (int)hi;
    s.j0 = s.lo / kStepKeys;
    s.n = s.hi > 0 ? (s.hi - 1) / kStepKeys + 1 - s.j0 : 0;
    return s;
}

__device__ __forceinline__ int tiles_of(const NvAttnArgs& a, int nq)
{
    return (nq + a.tile_tokens - 1) / a.tile_tokens;
}

// Where a warp's range begins, and how many units it has.
struct Start {
    int b, tile, head;   // selected: b is the token; head: of kv_heads * head_blocks
    int at;              // unit of the item
    long long left;
};

template <int D, int NT>
__device__ __forceinline__ Start find_start(const NvAttnArgs& a, uint8_t* smem)
{
    using C = Cfg<D, NT>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = a.kv_heads * a.head_blocks;
    long long* units = reinterpret_cast<long long*>(smem);
    long long* sums = reinterpret_cast<long long*>(smem + C::kSums);
    long long total = 0;
    for (int b0 = warp * 32; b0 < a.batch; b0 += C::kThreads) {
        const int b = b0 + lane;
        int tok0 = 0, nq = 0, kv = 0;
        if (b < a.batch) request_of(a, b, tok0, nq, kv);
        const int tiles = tiles_of(a, nq);
        long long u = 0;
        if (tiles <= 4)
            for (int i = 0; i < tiles; ++i) u += kItemUnits + span_of(a, nq, kv, i).n;
        // long ones by the whole warp
        for (unsigned who = __ballot_sync(0xffffffffu, tiles > 4); who; who &= who - 1) {
            const int l = __ffs(who) - 1;
            const int n = __shfl_sync(0xffffffffu, nq, l), k = __shfl_sync(0xffffffffu, kv, l);
            long long v = 0;
            for (int i = lane; i < tiles_of(a, n); i += 32) v += kItemUnits + span_of(a, n, k, i).n;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == l) u = v;
        }
        if (b < a.batch) units[b] = u;
        total += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) sums[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < C::kWarps; ++w) total += sums[w];
    total *= heads;
    Start s = {0, 0, 0, 0, 0};
    const int workers = gridDim.x * C::kWarps, me = blockIdx.x * C::kWarps + warp;
    long long rem = range_start(total, workers, me);
    s.left = range_start(total, workers, me + 1) - rem;
    if (s.left == 0) return s;
    // the request that holds unit `rem`, 32 at a time
    bool found = false;
    for (int c = 0; c < a.batch; c += 32) {
        long long incl = c + lane < a.batch ? units[c + lane] * heads : 0;
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
            rem -= __shfl_sync(0xffffffffu, incl - mine, l);
            found = true;
            break;
        }
        rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    // its tile, 32 at a time
    int tok0, nq, kv;
    request_of(a, s.b, tok0, nq, kv);
    const int tiles = tiles_of(a, nq);
    for (int c = 0; found && c < tiles; c += 32) {
        const int per = c + lane < tiles ? kItemUnits + span_of(a, nq, kv, c + lane).n : 0;
        long long incl = (long long)per * heads;
        const long long mine = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned who = __ballot_sync(0xffffffffu, incl - mine <= rem && rem < incl);
        if (who) {
            const int l = __ffs(who) - 1;
            s.tile = c + l;
            const int n = __shfl_sync(0xffffffffu, per, l);
            rem -= __shfl_sync(0xffffffffu, incl - mine, l);
            s.head = (int)(rem / n);
            s.at = (int)(rem - (long long)s.head * n);
            return s;
        }
        rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    s.left = 0;            // never
    return s;
}

// ------------------------------------------------------------------ pieces joined

// Parts of a row joined in turn: N of its columns under a running maximum.
template <int N>
struct Joined {
    float top = -INFINITY, sum = 0.0f, acc[N] = {};

    // (maxima are scores; times scale_log2 they are exponents)
    __device__ void add(float m, float l, const float (&v)[N], float scale_log2)
    {
        const float next = fmaxf(top, m);
        const float f = top == -INFINITY ? 0.0f : exp2_approx((top - next) * scale_log2);
        const float g = m == -INFINITY ? 0.0f : exp2_approx((m - next) * scale_log2);
        top = next;
        sum = sum * f + l * g;
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = fmaf(v[k], g, acc[k] * f);
    }
};

template <int N>
__device__ __forceinline__ void load_cols(const float* p, float (&v)[N])
{
    static_assert(N == 2 || N == 4, "columns");
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x; v[1] = x.y;
    }
}

// A row's scaled output and log-sum from its sums, which are 2^7 2^-top times too
// large.
__device__ __forceinline__ float inverse_of(float sum, float v_scale)
{
    return sum > 0.0f || sum != sum ? v_scale / sum : 0.0f;
}

__device__ __forceinline__ float log_sum_of(float top, float sum)
{
    return sum == 0.0f ? -INFINITY : (top - kPLog2) * 0.6931471805599453f + logf(sum);
}

// N columns of row `row` of an item, joined.
template <bool FP16, int N>
__device__ __forceinline__ void write_joined(const NvAttnArgs& a, const Joined<N>& x, int tok0, int head0, int heads,
                                             int row, int col)
{
    const float inv = inverse_of(x.sum, a.vc.scale);
    const long long token = tok0 + row / heads;
    const int head = head0 + row % heads;
    uint16_t* out = static_cast<uint16_t*>(a.out) + token * a.out_token + head * a.out_head + col;
    if constexpr (N == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_out<FP16>(x.acc[0] * inv, x.acc[1] * inv),
                                                    pack_out<FP16>(x.acc[2] * inv, x.acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(out) = pack_out<FP16>(x.acc[0] * inv, x.acc[1] * inv);
    if (col == 0 && a.lse != nullptr)
        a.lse[token * a.kv_heads * a.group + head] = log_sum_of(x.top * a.scale_log2, x.sum);
}

// The pieces of a cluster's item, when all of its CTAs are through: a row to a warp.
template <int D, bool FP16, int NT>
__device__ __forceinline__ void join_cluster(const NvAttnArgs& a, const Pieces& cp)
{
    constexpr int N = D / 32, kRows = 8 * NT;
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % a.cluster, row = warp * a.cluster + rank, col = lane * N;
    const long long q0 = (blockIdx.x - rank) * 2LL;
    const int* r = cp.rec + (q0 + 1) * kPcInts;
    if (!r[kPcUsed] || row >= r[kPcNtok] * r[kPcHeads]) return;
    Joined<N> x;
#pragma unroll 4
    for (int p = 0; p < a.cluster; ++p) {
        const long long q = q0 + 2 * p + (p == 0 ? 1 : 0);
        const bool used = cp.rec[q * kPcInts + kPcUsed];       // (a range without a step left none)
        float2 st = cp.stats[q * kRows + row];
        float v[N];
        load_cols<N>(cp.part + (q * kRows + row) * D + col, v);
        if (!used) {
            st = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = 0.0f;
        }
        x.add(st.x, st.y, v, a.scale_log2);
    }
    write_joined<FP16, N>(a, x, r[kPcTok0], r[kPcHead], r[kPcHeads], row, col);
}

// ------------------------------------------------------------------ the kernel

template <int D, bool FP16, bool SEL, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    nvfp4_attention_kernel(const NvAttnArgs a, const Pieces wp, const Pieces cp)
{
    using C = Cfg<D, NT>;
    constexpr int S = C::kStages;
    constexpr int KS = D / 16;             // 16-element steps of a score, 16-element blocks of an output
    constexpr int CB = C::kCode, SB = C::kScale;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    allow_dependent_launch();
    grid_dependency_wait();

    Start start;
    const int sel_n = SEL ? (a.sel_k + kStepKeys - 1) / kStepKeys : 0;
    const int heads = a.kv_heads * a.head_blocks;
    if constexpr (SEL) {
        const int per = sel_n + kItemUnits;
        const long long items = (long long)a.tokens * heads;
        long long s0, s1;
        if (a.cluster > 1) {
            const long long i0 = blockIdx.x / a.cluster;
            const int workers = a.cluster * C::kWarps, me = blockIdx.x % a.cluster * C::kWarps + warp;
            s0 = i0 * per + range_start(per, workers, me);
            s1 = i0 * per + range_start(per, workers, me + 1);
        } else if (a.whole_items) {        // a CTA's items, shared out over its warps
            const long long i0 = range_start(items, gridDim.x, blockIdx.x);
            const long long units = (range_start(items, gridDim.x, blockIdx.x + 1) - i0) * per;
            s0 = i0 * per + range_start(units, C::kWarps, warp);
            s1 = i0 * per + range_start(units, C::kWarps, warp + 1);
        } else {
            const int workers = gridDim.x * C::kWarps, me = blockIdx.x * C::kWarps + warp;
            s0 = range_start(items * per, workers, me);
            s1 = range_start(items * per, workers, me + 1);
        }
        start.left = s1 - s0;
        const long long item = s0 / per;
        start.at = (int)(s0 - item * per);
        start.b = (int)(item / heads);
        start.head = (int)(item - (long long)start.b * heads);
        start.tile = 0;
    } else {
        if (a.cluster > 1) {               // one request
            const int item = blockIdx.x / a.cluster;
            start = {0, item / heads, item % heads, 0, 0};
            int tok0, nq, kv;
            request_of(a, 0, tok0, nq, kv);
            if (start.tile < tiles_of(a, nq)) {
                const int per = kItemUnits + span_of(a, nq, kv, start.tile).n;
                const int workers = a.cluster * C::kWarps, me = blockIdx.x % a.cluster * C::kWarps + warp;
                start.at = (int)range_start(per, workers, me);
                start.left = range_start(per, workers, me + 1) - start.at;
            }
        } else {
            start = find_start<D, NT>(a, smem);
            __syncthreads();               // (the numbers lie in the ring)
        }
    }

    const uint32_t ring = smem_addr(smem) + warp * C::kRing;
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::kMasks) + warp * 8;
    constexpr int kKC = 0, kVC = kStepKeys * CB, kKS = 2 * kStepKeys * CB, kVS = kKS + kStepKeys * SB;
    const long long worker = (long long)blockIdx.x * C::kWarps + warp;
    int* rec = reinterpret_cast<int*>(smem + C::kPieces) + warp * 2 * kPcInts;
    uint8_t* used = smem + C::kRecs + warp * 8;           // [2] used, [2] last
    if (lane < 8) used[lane] = 0;

    // copies: this lane's row and 16-byte chunk of 8 (16) rows of codes
    constexpr int kRowLanes = CB / 16, kInstRows = 32 / kRowLanes;
    const int sub = lane / kRowLanes, chunk = lane % kRowLanes;
    auto column = [](int r) { return (r & ~7) | ((r & 3) << 1) | ((r >> 2) & 1); };
    const uint32_t k_to = kKC + column(sub) * CB + chunk * 16;
    const uint32_t v_to = kVC + sub * CB + (D == 128 ? (chunk ^ (((sub >> 1) & 1) << 1)) : chunk) * 16;
    const uint32_t ks_to = kKS + column(lane) * SB, vs_to = kVS + lane * SB;

    const bool same = a.kc.page == a.vc.page && a.kc.slot == a.vc.slot;

    int b = start.b, tile = start.tile, head = start.head, at = start.at;
    long long left = start.left;
    int cur_b = -1, tok0 = 0, nq = 0, kv = 0, tiles = 0;
    while (left > 0) {
        Span sp;
        int req, token;
        if constexpr (SEL) {
            req = __ldg(a.requests + b);
            if (req >= a.batch && lane == 0) atomicOr(a.status, kStatusBadRequest);
            const bool fine = req >= 0 && req < a.batch;
            kv = fine ? max(__ldg(a.kv_lens + req), 0) : 0;
            kv = (int)min((long long)kv, (long long)a.bt_width * kBlockKeys);
            req = fine ? req : 0;
            sp = {0, 1, 0, kv, 0, sel_n};
            token = b;
        } else {
            if (b >= a.batch) break;       // lengths changed under the call
            if (b != cur_b) {
                request_of(a, b, tok0, nq, kv);
                tiles = tiles_of(a, nq);
                cur_b = b;
                if (tiles == 0) { ++b; tile = 0; head = 0; at = 0; continue; }
            }
            req = b;
            sp = span_of(a, nq, kv, tile);
            token = tok0 + sp.t0;
        }
        const int kvh = head / a.head_blocks, hb = head - kvh * a.head_blocks;
        const int head0 = kvh * a.group + hb * a.block_heads;
        const int nh = min(a.block_heads, a.group - hb * a.block_heads);
        // the steps of this range: j .. j + n - 1
        const int take = (int)min(left, (long long)(kItemUnits + sp.n - at));
        const int j = max(at - kItemUnits, 0), n = max(at + take - kItemUnits, 0) - j;
        const bool whole = n == sp.n;
        const bool nothing = at == 0 && sp.n == 0;        // rows that see no key
        left -= take;
        const bool done = at + take == kItemUnits + sp.n;
        const bool first = j == 0;
        at = 0;
        if (done) {
            if (++head == heads) {
                head = 0;
                if (SEL || ++tile == tiles) { tile = 0; ++b; }
            }
        }
        if (n == 0 && !nothing) continue;

        // ---- copies, a few steps ahead
        const int32_t* table = a.block_table + (long long)req * a.bt_stride;
        const int32_t* list = SEL ? a.selected + (long long)token * a.sel_stride : nullptr;
        const uint8_t* k_from = a.kc.codes + kvh * a.kc.head + chunk * 16;
        const uint8_t* v_from = a.vc.codes + kvh * a.vc.head + chunk * 16;
        const uint8_t* ks_from = a.kc.scales + kvh * a.kc.s_head;
        const uint8_t* vs_from = a.vc.scales + kvh * a.vc.s_head;
        if constexpr (!SEL) {              // this lane's rows of a page's first step
            k_from += sub * a.kc.slot;
            v_from += sub * a.vc.slot;
            ks_from += lane * a.kc.s_slot;
            vs_from += lane * a.vc.s_slot;
        }
        const int j0 = sp.j0 + j;
        // dense: 32 table entries from page `win` on, one a lane
        int win = -1, entry = 0;
        // selected: this lane's position and page of the next step to copy, the
        // page of the one after it on its way, the position of the third
        int p0 = -1, p1 = -1, p2 = -1, g0 = 0, g1 = 0;
        auto position = [&](int s) {
            const int i = (j0 + s) * kStepKeys + lane;
            const int p = s < n && i < a.sel_k ? __ldg(list + i) : -1;
            return p < kv ? p : -1;
        };
        auto page_at = [&](int p) { return p >= 0 ? __ldg(table + (p >> 6)) : 0; };
        if constexpr (SEL) {
            p0 = position(0);
            p1 = position(1);
            p2 = position(2);
        }
        // ---- Q's rows on their way: lane (g, t) takes part of row g of each eight
        const int rows = sp.ntok * nh;
        uint4 qw[NT][KS / 2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int c = 0; c < KS / 2; ++c) qw[x][c] = make_uint4(0u, 0u, 0u, 0u);
            if (const int r = g + 8 * x; r < rows) {
                const int i = r / nh;
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(a.q) + (long long)(token + i) * a.q_token +
                    (long long)(head0 + r - i * nh) * a.q_head + t * (D / 4));
#pragma unroll
                for (int c = 0; c < KS / 2; ++c) qw[x][c] = __ldg(src + c);
            }
        }

        if constexpr (SEL) {
            g0 = page_at(p0);
            g1 = page_at(p1);
        }
        auto copy = [&](int s, int st) {
            const uint32_t to = ring + st * C::kStageBytes;
            if constexpr (SEL) {
                if (g0 < 0 || g0 >= a.num_pages) {
                    atomicOr(a.status, kStatusBadBlock);
                    g0 = 0;
                }
                const unsigned valid = __ballot_sync(0xffffffffu, p0 >= 0);
                if (lane == 0) masks[st] = valid;
                const int slot = p0 & 63;
                const long long k_off = g0 * a.kc.page + slot * a.kc.slot, v_off = g0 * a.vc.page + slot * a.vc.slot;
#pragma unroll
                for (int i = 0; i < kStepKeys / kInstRows; ++i) {
                    const int r = i * kInstRows + sub;
                    const uint32_t bytes = (valid >> r) & 1 ? 16u : 0u;
                    const long long ko = __shfl_sync(0xffffffffu, k_off, r);
                    const long long vo = same ? ko : __shfl_sync(0xffffffffu, v_off, r);
                    cp_async_zfill<16>(to + k_to + i * kInstRows * CB, k_from + ko, bytes);
                    cp_async_zfill<16>(to + v_to + i * kInstRows * CB, v_from + vo, bytes);
                }
                const uint32_t bytes = p0 >= 0 ? SB : 0u;
                cp_async_zfill<SB>(to + ks_to, ks_from + g0 * a.kc.s_page + slot * a.kc.s_slot, bytes);
                cp_async_zfill<SB>(to + vs_to, vs_from + g0 * a.vc.s_page + slot * a.vc.s_slot, bytes);
                p0 = p1;
                g0 = g1;
                p1 = p2;
                g1 = page_at(p1);
                p2 = position(s + 3);
            } else {
                const int key0 = (j0 + s) * kStepKeys, pg = key0 >> 6;
                if (win < 0 || pg >= win + 32) {
                    win = pg;
                    entry = pg + lane <= (sp.hi - 1) >> 6 ? __ldg(table + pg + lane) : 0;
                    if (entry < 0 || entry >= a.num_pages) {
                        atomicOr(a.status, kStatusBadBlock);
                        entry = 0;
                    }
                }
                const int page = __shfl_sync(0xffffffffu, entry, pg - win);
                const uint8_t* kp = k_from + page * a.kc.page;
                const uint8_t* vp = v_from + page * a.vc.page;
                const uint8_t* ksp = ks_from + page * a.kc.s_page;
                const uint8_t* vsp = vs_from + page * a.vc.s_page;
                if (key0 & kStepKeys) {    // the page's second step
                    kp += kStepKeys * a.kc.slot;
                    vp += kStepKeys * a.vc.slot;
                    ksp += kStepKeys * a.kc.s_slot;
                    vsp += kStepKeys * a.vc.s_slot;
                }
                auto rows_in = [&](auto bytes_of) {
#pragma unroll
                    for (int i = 0; i < kStepKeys / kInstRows; ++i) {
                        const uint32_t bytes = bytes_of(i * kInstRows + sub, 16);
                        cp_async_zfill<16>(to + k_to + i * kInstRows * CB, kp, bytes);
                        cp_async_zfill<16>(to + v_to + i * kInstRows * CB, vp, bytes);
                        kp += kInstRows * a.kc.slot;
                        vp += kInstRows * a.vc.slot;
                    }
                    const uint32_t bytes = bytes_of(lane, SB);
                    cp_async_zfill<SB>(to + ks_to, ksp, bytes);
                    cp_async_zfill<SB>(to + vs_to, vsp, bytes);
                };
                if (key0 >= sp.lo && key0 + kStepKeys <= sp.hi)
                    rows_in([](int, int bytes) { return bytes; });
                else                       // (rows outside the item's keys become zeros)
                    rows_in([&](int r, int bytes) { return key0 + r >= sp.lo && key0 + r < sp.hi ? bytes : 0; });
            }
        };

        // the first copies, and what the steps work on while those are under way
#pragma unroll 1
        for (int s = 0; s < S - 1; ++s) {
            if (s < n) copy(s, s);
            cp_async_commit();
        }

        // ---- the rows scaled to fp16, and of rows 2 t and 2 t + 1 the factor, the reference and the sum
        uint32_t qb[KS][2];                    // (of eight rows)
        const uint32_t q_at = smem_addr(smem) + C::kQ + warp * C::kQBytes + lane * 16;
        float f[NT][2], ref[NT][2], l[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            uint4 (&w)[KS / 2] = qw[x];
            float scale = a.scale_log2;
            if constexpr (!FP16) {
                // the row's largest exponent, which becomes 0
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < KS / 2; ++c) {
                    const uint32_t m = 0x7fff7fffu;
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[c].x & m, w[c].y & m), __vmaxu2(w[c].z & m, w[c].w & m)));
                }
                top = max(top & 0xffffu, top >> 16) >> 7;
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = min(max(top, 1u), 253u);
                scale *= __uint_as_float(top << 23);
                const float inv = __uint_as_float((254u - top) << 23);
                auto half = [&](uint32_t v) {
                    return pack_f16(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv);
                };
#pragma unroll
                for (int c = 0; c < KS / 2; ++c)
                    w[c] = make_uint4(half(w[c].x), half(w[c].y), half(w[c].z), half(w[c].w));
            }
#pragma unroll
            for (int c = 0; c < KS / 2; ++c) {
                if constexpr (NT == 1) {
                    qb[2 * c][0] = w[c].x;
                    qb[2 * c][1] = w[c].y;
                    qb[2 * c + 1][0] = w[c].z;
                    qb[2 * c + 1][1] = w[c].w;
                } else {                           // (a lane reads what it has written)
                    st_shared_v4(q_at + (x * (KS / 2) + c) * 512, w[c].x, w[c].y, w[c].z, w[c].w);
                }
            }
            scale = fminf(fmaxf(scale, 1.2e-38f), 3.4e38f);    // (times -inf it stays -inf, times 0 it is 0)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f[x][c] = __shfl_sync(0xffffffffu, scale, 8 * t + 4 * c);
                ref[x][c] = -INFINITY;
                l[x][c] = 0.0f;
            }
        }
        // the keys that row 8 x + 2 t + c sees: [x, y)
        auto sees = [&](int x, int c) {
            const int pos = kv - nq + sp.t0 + min((8 * x + 2 * t + c) / nh, sp.ntok - 1);
            return make_int2(a.window > 0 ? (int)max((long long)pos - a.window + 1, 0ll) : 0,
                             a.causal ? min(max(pos + 1, 0), sp.hi) : sp.hi);
        };
        // steps that every row sees all of lie in [all_lo, all_hi)
        int all_lo = 0, all_hi = 0;
        if constexpr (!SEL) {
            const long long pos = (long long)kv - nq + sp.t0;
            all_lo = a.window > 0 ? (int)max(pos + sp.ntok - a.window, 0ll) : 0;
            all_hi = a.causal ? (int)min(max(pos + 1, 0ll), (long long)sp.hi) : sp.hi;
        }
        float o[NT][KS][4];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][i][e] = 0.0f;

        // whether a row of this lane's has seen no key yet, or its exponents are large
        bool far = true;
        // ---- one step's keys in stage `st`
        auto compute = [&](int s, int st) {
            const uint32_t from = ring + st * C::kStageBytes;
            // element 2 h + c of sc[x][y] is key 16 y + 8 h + (g / 2) + 4 (g & 1),
            // row 8 x + 2 t + c
            float sc[NT][2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t w[2][KS / 2], m[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 16 * y + 8 * h + g;
                    if constexpr (D == 128) {
                        const uint4 v = ld_shared_v4(from + kKC + row * CB + t * (CB / 4));
                        w[h][0] = v.x; w[h][1] = v.y; w[h][2] = v.z; w[h][3] = v.w;
                        const uint32_t s2 = e4m3x2_to_f16x2(ld_shared_u16(from + kKS + row * SB + 2 * t));
                        m[h][0] = __byte_perm(s2, s2, 0x1010);
                        m[h][1] = __byte_perm(s2, s2, 0x3232);
                    } else {
                        const uint2 v = ld_shared_v2_u32(from + kKC + row * CB + t * (CB / 4));
                        w[h][0] = v.x; w[h][1] = v.y;
                        m[h][0] = m[h][1] = e4m3_to_f16x2_dup(ld_shared_u8(from + kKS + row * SB + t));
                    }
                }
#pragma unroll
                for (int c = 0; c < KS / 2; ++c) {
                    uint4 q[NT];
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        if constexpr (NT == 1) q[x] = make_uint4(qb[2 * c][0], qb[2 * c][1], qb[2 * c + 1][0], qb[2 * c + 1][1]);
                        else q[x] = ld_shared_v4(q_at + (x * (KS / 2) + c) * 512);
                    }
                    uint32_t u[4], v[4];
                    e2m1x8_to_f16x2x4(w[0][c], u);
                    e2m1x8_to_f16x2x4(w[1][c], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        u[e] = mul_f16x2(u[e], m[0][2 * c < KS / 2 ? 0 : 1]);
                        v[e] = mul_f16x2(v[e], m[1][2 * c < KS / 2 ? 0 : 1]);
                    }
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        if (c == 0) mma_first(sc[x][y], u[0], v[0], u[1], v[1], q[x].x, q[x].y);
                        else mma(sc[x][y], u[0], v[0], u[1], v[1], q[x].x, q[x].y);
                    }
#pragma unroll
                    for (int x = 0; x < NT; ++x) mma(sc[x][y], u[2], v[2], u[3], v[3], q[x].z, q[x].w);
                }
            }
            const int key0 = (j0 + s) * kStepKeys;
            bool parted = false;
            if constexpr (SEL) {
                const uint32_t valid = masks[st] >> ((g >> 1) + 4 * (g & 1));
                if (valid != 0xffffffffu >> ((g >> 1) + 4 * (g & 1))) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (!((valid >> (16 * y + 8 * h)) & 1))
#pragma unroll
                                for (int x = 0; x < NT; ++x) sc[x][y][2 * h] = sc[x][y][2 * h + 1] = -INFINITY;
                }
            } else {
                parted = key0 < all_lo || key0 + kStepKeys > all_hi;
                if (parted) {
#pragma unroll
                    for (int x = 0; x < NT; ++x)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int2 see = sees(x, c);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int key = key0 + 8 * i + (g >> 1) + 4 * (g & 1);
                                if (key < see.x || key >= see.y) sc[x][i >> 1][2 * (i & 1) + c] = -INFINITY;
                            }
                        }
                }
            }
            // exponents of P, unless one is too large
            float most = -INFINITY;
            float z[NT][2][4];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                float off[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) off[c] = fmaf(-ref[x][c], f[x][c], kPLog2);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[x][y][e] = fmaf(sc[x][y][e], f[x][e & 1], off[e & 1]);
                    most = max3(most, z[x][y][0], z[x][y][1]);
                    most = max3(most, z[x][y][2], z[x][y][3]);
                }
            }
            if (__any_sync(0xffffffffu, far || most > kPMost)) {
                far = false;
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    float down[2], from_ref[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float m = fmaxf(fmaxf(sc[x][0][c], sc[x][0][2 + c]), fmaxf(sc[x][1][c], sc[x][1][2 + c]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        // (from -inf on: yes unless m is)
                        const float next = (m - ref[x][c]) * f[x][c] > kPMost - kPLog2 ? m : ref[x][c];
                        down[c] = ref[x][c] == -INFINITY ? 0.0f : exp2_approx((ref[x][c] - next) * f[x][c]);
                        ref[x][c] = next;
                        from_ref[c] = next == -INFINITY ? 0.0f : next;
                        far = far || fabsf(next) * f[x][c] > kFar;      // (-inf too)
                        l[x][c] *= down[c];
                    }
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[x][i][0] *= down[0];
                        o[x][i][1] *= down[1];
                        o[x][i][2] *= down[0];
                        o[x][i][3] *= down[1];
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            z[x][y][e] = fmaf(sc[x][y][e] - from_ref[e & 1], f[x][e & 1], kPLog2);
                }
            }
            uint32_t pb[NT][2][2];
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float u = exp2_approx(z[x][y][2 * h]), v = exp2_approx(z[x][y][2 * h + 1]);
                        l[x][0] += u;
                        l[x][1] += v;
                        pb[x][y][h] = transpose8(pack_f16(u, v));
                    }
            // values: keys k + {0, 4, 8, 12}, k = 16 y + t, elements (D / 8) g ..
            auto scales_at = [&](int y, uint32_t& sa, uint32_t& sb) {
                const uint32_t vs = from + kVS + (16 * y + t) * SB + (D == 128 ? g : g >> 1);
                sa = e4m3x2_to_f16x2(ld_shared_u8(vs) | (ld_shared_u8(vs + 4 * SB) << 8));
                sb = e4m3x2_to_f16x2(ld_shared_u8(vs + 8 * SB) | (ld_shared_u8(vs + 12 * SB) << 8));
            };
            auto words_at = [&](int y, int e, uint32_t (&w)[KS / 4]) {
                if constexpr (D == 128) {
                    const uint2 v = ld_shared_v2_u32(from + kVC + (16 * y + t + 4 * e) * CB +
                                                     (((g >> 1) ^ (((t >> 1) & 1) << 1)) << 4) + (g & 1) * 8);
                    w[0] = v.x; w[1] = v.y;
                } else {
                    w[0] = ld_shared_u32(from + kVC + (16 * y + t + 4 * e) * CB + g * 4);
                }
            };
            // two keys' words: bytes of (first, second) codes of even and of odd elements
            auto pairs_of = [](uint32_t u, uint32_t v, uint32_t m, uint32_t (&even)[4], uint32_t (&odd)[4]) {
                e2m1x8_to_f16x2x4((u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u), even);
                e2m1x8_to_f16x2x4(((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u), odd);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    even[e] = mul_f16x2(even[e], m);
                    odd[e] = mul_f16x2(odd[e], m);
                }
            };
            if (parted) {
                // NaN scales: the rows that see their keys become NaN where they
                // stand, and the scales 0 for the product
                const uint32_t mine = from + kVS + lane * SB;
                uint32_t s0 = ld_shared_u32(mine), s1 = SB == 8 ? ld_shared_u32(mine + SB - 4) : 0u;
                auto clean = [](uint32_t v) { return v & ~__vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu); };
                if (__any_sync(0xffffffffu, clean(s0) != s0 || clean(s1) != s1)) {
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        const int2 see0 = sees(x, 0), see1 = sees(x, 1);
                        float n0 = 0.0f, n1 = 0.0f;
#pragma unroll 1
                        for (int k = 0; k < kStepKeys; ++k) {
                            if ((ld_shared_u8(from + kVS + k * SB + (D == 128 ? g : g >> 1)) & 0x7fu) != 0x7fu) continue;
                            if (key0 + k >= see0.x && key0 + k < see0.y) n0 = NAN;
                            if (key0 + k >= see1.x && key0 + k < see1.y) n1 = NAN;
                        }
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[x][i][0] += n0;
                            o[x][i][1] += n1;
                            o[x][i][2] += n0;
                            o[x][i][3] += n1;
                        }
                    }
                    __syncwarp();
                    st_shared_u32(mine, clean(s0));
                    if (SB == 8) st_shared_u32(mine + SB - 4, clean(s1));
                    __syncwarp();
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t w[4][KS / 4], sa, sb;
#pragma unroll
                for (int e = 0; e < 4; ++e) words_at(y, e, w[e]);
                scales_at(y, sa, sb);
#pragma unroll
                for (int c = 0; c < KS / 4; ++c) {
                    uint32_t ea[4], oa[4], eb[4], ob[4];
                    pairs_of(w[0][c], w[1][c], sa, ea, oa);
                    pairs_of(w[2][c], w[3][c], sb, eb, ob);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            mma(o[x][4 * c + e], ea[e], oa[e], eb[e], ob[e], pb[x][y][0], pb[x][y][1]);
                }
            }
        };

        // ---- the steps
        {
            int put = S - 1, got = 0;      // stages
#pragma unroll 1
            for (int s = 0; s < n; ++s) {
                cp_async_wait<S - 2>();
                __syncwarp();              // step s is there, and step s - 1's stage is free
                if (s + S - 1 < n) copy(s + S - 1, put);
                cp_async_commit();
                if (++put == S) put = 0;
                compute(s, got);
                if (++got == S) got = 0;
            }
            __syncwarp();
        }

        // ---- the rows' results, or a piece of them.  Lane (g, t) has elements
        // (D / 8) g .. of rows 2 t and 2 t + 1
        constexpr int E = D / 8;
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[x][c] += __shfl_xor_sync(0xffffffffu, l[x][c], d);
        if (whole) {
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = 8 * x + 2 * t + c;
                    if (r >= rows) continue;
                    const float m = inverse_of(l[x][c], a.vc.scale);
                    const int i = r / nh;
                    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                                          (long long)(token + i) * a.out_token +
                                                          (long long)(head0 + r - i * nh) * a.out_head + g * E);
#pragma unroll
                    for (int v = 0; v < E / 8; ++v) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_out<FP16>(o[x][4 * v + e][c] * m, o[x][4 * v + e][2 + c] * m);
                        out[v] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (g == 0 && a.lse != nullptr)
                        a.lse[(long long)(token + i) * a.kv_heads * a.group + head0 + r - i * nh] =
                            log_sum_of(ref[x][c] * f[x][c], l[x][c]);
                }
        } else {
            // The last piece stays in the ring, which nothing else needs any more.
            const int slot = first ? 1 : 0;
            const long long at_piece = worker * C::kRows;
            const bool here = left == 0;
            float* part = here ? reinterpret_cast<float*>(smem + warp * C::kRing) : wp.part + at_piece * D;
            float2* stats = here ? reinterpret_cast<float2*>(smem + warp * C::kRing + C::kRows * D * 4)
                                 : wp.stats + at_piece;
            if (lane == 0) {
                int* p = rec + slot * kPcInts;
                p[kPcTok0] = token;
                p[kPcNtok] = sp.ntok;
                p[kPcHead] = head0;
                p[kPcHeads] = nh;
                used[slot] = here ? 2 : 1;
                used[2 + slot] = j + n == sp.n;
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = 8 * x + 2 * t + c;
                    // (the reference as a score of q itself: its own power of two undone)
                    if (g == 0) stats[r] = make_float2(ref[x][c] * (f[x][c] / a.scale_log2), l[x][c]);
                    float4* out = reinterpret_cast<float4*>(part + r * D + g * E);
#pragma unroll
                    for (int v = 0; v < E / 4; ++v)
                        out[v] = make_float4(o[x][2 * v][c], o[x][2 * v][2 + c], o[x][2 * v + 1][c], o[x][2 * v + 1][2 + c]);
                }
            }
        }
    }

    // ---- the CTA's pieces, in order: an item's begin with slot 1 of a warp and
    // go on with slot 0 of the warps after it
    __syncthreads();
    constexpr int N = D / 32;
    const uint32_t flags = lane < C::kWarps ? *reinterpret_cast<const uint32_t*>(smem + C::kRecs + lane * 8) : 0u;
    const unsigned begin = __ballot_sync(0xffffffffu, flags & 0xff00u), go = __ballot_sync(0xffffffffu, flags & 0xffu),
                   end = __ballot_sync(0xffffffffu, flags & 0xff0000u),
                   kept = __ballot_sync(0xffffffffu, (flags & 0xffu) == 2u);
    // pieces that go on an item begun before this CTA: from the first warp on
    const bool lead = go != 0 && (begin == 0 || __ffs(go) <= __ffs(begin));
    const int chains = __popc(begin) + (lead ? 1 : 0);
    int* crec = cp.rec + blockIdx.x * 2LL * kPcInts;
    if (threadIdx.x < 2) {
        // slot 0: the item from before; slot 1: the last one, if it does not end here
        const bool mine = threadIdx.x == 0 ? lead
                                           : begin != 0 && !(go & end & ~((2u << (31 - __clz(begin))) - 1u));
        const int w = threadIdx.x == 0 ? __ffs(go) - 1 : 31 - __clz(begin);
        int* r = crec + threadIdx.x * kPcInts;
        r[kPcUsed] = mine;
        if (mine) {
            const int* p = reinterpret_cast<const int*>(smem + C::kPieces) + (w * 2 + threadIdx.x) * kPcInts;
            r[kPcTok0] = p[kPcTok0];
            r[kPcNtok] = p[kPcNtok];
            r[kPcHead] = p[kPcHead];
            r[kPcHeads] = p[kPcHeads];
            r[kPcLast] = threadIdx.x == 0 && (go & end) != 0;
        }
    }
    for (int i = threadIdx.x; i < chains * C::kRows * 32; i += C::kThreads) {
        const int chain = i / (C::kRows * 32), row = (i >> 5) % C::kRows, col = (i & 31) * N;
        const bool led = lead && chain == 0;
        unsigned b0 = begin;                   // its first warp is the lowest bit left
        for (int k = lead ? 1 : 0; k < chain; ++k) b0 &= b0 - 1;
        const int w0 = __ffs(led ? go : b0) - 1;
        unsigned members = led ? go : go & ~((2u << w0) - 1u);
        const unsigned ends = members & end;
        if (ends) members &= ((ends & (0u - ends)) << 1) - 1u;
        const int* p = reinterpret_cast<const int*>(smem + C::kPieces) + (w0 * 2 + (led ? 0 : 1)) * kPcInts;
        const int c_heads = p[kPcHeads];
        if (row >= p[kPcNtok] * c_heads) continue;
        Joined<N> x;
        // (what an item begins with is its warp's last piece)
        const unsigned own = led ? 0u : 1u << w0;
        members |= own;
#pragma unroll 1
        for (; members; members &= members - 1) {
            const int w = __ffs(members) - 1;
            const bool here = ((kept | own) >> w) & 1;
            const long long q = (blockIdx.x * (long long)C::kWarps + w) * C::kRows;
            const float* part = here ? reinterpret_cast<const float*>(smem + w * C::kRing) : wp.part + q * D;
            const float2* stats = here ? reinterpret_cast<const float2*>(smem + w * C::kRing + C::kRows * D * 4)
                                       : wp.stats + q;
            const float2 st = stats[row];
            float y[N];
            load_cols<N>(part + row * D + col, y);
            x.add(st.x, st.y, y, a.scale_log2);
        }
        if (!led && ends) {
            write_joined<FP16, N>(a, x, p[kPcTok0], p[kPcHead], c_heads, row, col);
        } else {
            const long long q = (blockIdx.x * 2LL + (led ? 0 : 1)) * C::kRows + row;
            if (col == 0) cp.stats[q] = make_float2(x.top, x.sum);
#pragma unroll
            for (int e = 0; e < N; ++e) cp.part[q * D + col + e] = x.acc[e];
        }
    }
    if (a.cluster > 1) join_cluster<D, FP16, NT>(a, cp);
}

}  // namespace nvattn
}  // namespace pml
