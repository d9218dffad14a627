// Bookkeeping of a pool of cache pages on sm_103a: extending, forking and
// freeing requests, compacting the pool, and the page copies these ask for.
//
// The pool's state is one count per page (how many requests hold it; 0: free)
// and the requests' block tables and lengths.  There is no free list: the
// r-th page that a call takes is the r-th lowest free one, found by a scan of
// the counts, so a call's result depends on the state alone and not on the
// order in which threads get there.
//
// The planning kernels are bound by latency: a few passes over num_pages
// counts and the touched table rows.  They run as ONE cluster of eight CTAs
// (8192 threads), which splits the counts into eight slices, exchanges the
// slices' totals through distributed shared memory and meets at hardware
// barriers, where several launches or a single CTA would pay a launch or a
// longer scan per pass.  The page copies are bound by memory and run on the
// whole GPU.
//
// Measured: forking 160 requests of up to 8192 tokens 10.5 us, freeing them 4.3
// (a warp per request: 9); extending 64 requests by a token 8.0 over 8192 pages
// and 9.3 over 65536; the compaction plan of 64 requests' pages 14 us (its
// tables a warp per row: 19); copying 544 MB of pages 166 us, 6.55 TB/s of read
// and write, 97 % of a plain copy's 6776 GB/s.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dependent.cuh"
#include "serving.h"

namespace pml {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;
constexpr int kAhead = 4;     // table entries that a lane loads at once
constexpr unsigned int kStatusNoPages = 16u;     // PML_STATUS_NO_PAGES

// Exclusive prefix of v over the CTA, and the total; two barriers.
__device__ __forceinline__ int block_scan(int v, int* buf, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    int w = lane < kWarps ? buf[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
    __syncthreads();
    return before + incl - v;
}

// Counts of the pages for which keep(page, count) holds: this CTA's slice
// total goes to `mine`, and after the cluster barrier every CTA knows the
// total over the lower slices and over all.
struct Slice {
    int begin, end;
};

__device__ __forceinline__ Slice slice_of(int n, int rank)
{
    const int per = (n + kCtas - 1) / kCtas;
    Slice s;
    s.begin = min(n, rank * per);
    s.end = min(n, s.begin + per);
    return s;
}

template <class F>
__device__ __forceinline__ int count_slice(Slice s, const int32_t* refs, int* buf, F keep)
{
    int n = 0;
    for (int p = s.begin + threadIdx.x; p < s.end; p += kThreads) n += keep(p, refs[p]) ? 1 : 0;
    int total;
    block_scan(n, buf, total);
    return total;
}

// Calls emit(rank, page) for the slice's kept pages in ascending order, ranks
// from `first` on, until `limit` ranks are given out.
template <class F, class E>
__device__ __forceinline__ void emit_slice(Slice s, const int32_t* refs, int* buf, int first,
                                           int limit, F keep, E emit)
{
    int at = first;
    for (int base = s.begin; base < s.end && at < limit; base += kThreads) {
        const int p = base + threadIdx.x;
        const bool k = p < s.end && keep(p, refs[p]);
        int total;
        const int r = at + block_scan(k ? 1 : 0, buf, total);
        if (k && r < limit) emit(r, p);
        at += total;
    }
}

// The CTAs' values of shared[], summed below this rank and over all.
__device__ __forceinline__ void exchange(cg::cluster_group& cl, int* shared, int value, int& below,
                                         int& all)
{
    if (threadIdx.x == 0) *shared = value;
    cl.sync();
    below = 0;
    all = 0;
#pragma unroll
    for (int r = 0; r < kCtas; ++r) {
        const int v = *cl.map_shared_rank(shared, r);
        all += v;
        if (r < (int)cl.block_rank()) below += v;
    }
}

__device__ __forceinline__ int pages_of(int len) { return len > 0 ? (int)(((long long)len + 63) >> 6) : 0; }

// ------------------------------------------------------------------ fork

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    pages_fork_kernel(const ForkArgs a)
{
    __shared__ int buf[kWarps];
    __shared__ int ranks[kThreads];
    __shared__ int xfree;
    allow_dependent_launch();
    grid_dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    const PoolArgs& P = a.pool;

    auto valid = [&](int i, int& parent, int& child, int& len) {
        parent = __ldg(a.parents + i);
        child = __ldg(a.children + i);
        len = 0;
        if (parent < 0 || parent >= P.rows || child < 0 || child >= P.rows) return false;
        len = P.seq_lens[parent];
        return pages_of(len) <= P.bt_width;
    };

    // how many forks end in a part page: each needs a page of its own.  Every
    // CTA counts them all (a few reads per thread).
    int need = 0;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
        int parent, child, len;
        if (valid(i, parent, child, len) && len > 0 && (len & 63)) ++need;
    }
    int needed;
    block_scan(need, buf, needed);

    const Slice s = slice_of(P.num_pages, rank);
    auto is_free = [](int, int c) { return c == 0; };
    const int here = count_slice(s, P.ref_counts, buf, is_free);
    int below, all;
    exchange(cl, &xfree, here, below, all);
    const int taken = min(needed, all);
    emit_slice(s, P.ref_counts, buf, below, taken, is_free, [&](int r, int p) { a.dst[r] = p; });
    if (rank == 0) {
        for (int i = taken + threadIdx.x; i < a.n; i += kThreads) {
            a.src[i] = -1;
            a.dst[i] = -1;
        }
        if (threadIdx.x == 0) {
            *a.count = taken;
            if (needed > all) atomicOr(P.status, kStatusNoPages);
        }
    }
    __threadfence();
    cl.sync();

    // the forks, a warp each; the ranks of a step of 1024 come from a scan
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int at = 0;
    for (int base = 0; base < a.n; base += kThreads) {
        const int i0 = base + threadIdx.x;
        int parent, child, len;
        const bool part = i0 < a.n && valid(i0, parent, child, len) && len > 0 && (len & 63);
        int total;
        ranks[threadIdx.x] = at + block_scan(part ? 1 : 0, buf, total);
        at += total;
        __syncthreads();
        const int end = min(a.n, base + kThreads);
        for (int i = base + warp * kCtas + rank; i < end; i += kWarps * kCtas) {
            if (!valid(i, parent, child, len)) {
                if (lane == 0) atomicOr(P.status, kStatusBadRequest);
                continue;
            }
            const int full = len > 0 ? len >> 6 : 0;
            const bool own_page = len > 0 && (len & 63);
            const int r = ranks[i - base];
            const int32_t* from = P.block_table + (long long)parent * P.bt_stride;
            int32_t* to = P.block_table + (long long)child * P.bt_stride;
            if (own_page && r >= taken) {
                if (lane == 0) P.seq_lens[child] = 0;
                continue;
            }
            if (lane == 0) {
                if (own_page) {
                    const int p = a.dst[r];
                    a.src[r] = from[full];
                    to[full] = p;
                    P.ref_counts[p] = 1;
                }
                P.seq_lens[child] = max(len, 0);
            }
            // (several loads on their way at once: each takes longer than the rest)
            for (int c0 = lane; c0 < full; c0 += 32 * kAhead) {
                int p[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) p[k] = c0 + 32 * k < full ? from[c0 + 32 * k] : -1;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    if (c0 + 32 * k >= full) break;
                    to[c0 + 32 * k] = p[k];
                    if (p[k] >= 0 && p[k] < P.num_pages) atomicAdd(P.ref_counts + p[k], 1);
                    else atomicOr(P.status, kStatusBadBlock);
                }
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ extend

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    pages_extend_kernel(const ExtendArgs a)
{
    __shared__ int buf[kWarps];
    __shared__ int ranks[kThreads];
    __shared__ int xfree;
    allow_dependent_launch();
    grid_dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    const PoolArgs& P = a.pool;

    // pages that row i needs; a length past the table's width asks for none
    // (and is refused below)
    auto need_of = [&](int i, int& have) {
        const int want = pages_of(__ldg(a.new_lens + i));
        have = pages_of(P.seq_lens[i]);
        return want > P.bt_width ? 0 : max(0, want - have);
    };
    int sum = 0, have;
    for (int i = threadIdx.x; i < P.rows; i += kThreads) sum += need_of(i, have);
    int needed;
    block_scan(sum, buf, needed);

    const Slice s = slice_of(P.num_pages, rank);
    auto is_free = [](int, int c) { return c == 0; };
    const int here = count_slice(s, P.ref_counts, buf, is_free);
    int below, all;
    exchange(cl, &xfree, here, below, all);
    const int room = min(all, a.capacity);
    const int listed = min(needed, room);
    emit_slice(s, P.ref_counts, buf, below, listed, is_free,
               [&](int r, int p) { a.new_pages[r] = p; });
    __threadfence();
    cl.sync();

    // a row whose last page lies past the free ones keeps its length, and so
    // does every later row that needs one
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int at = 0, used = 0;
    for (int base = 0; base < P.rows; base += kThreads) {
        const int i0 = base + threadIdx.x;
        const int n0 = i0 < P.rows ? need_of(i0, have) : 0;
        int total;
        const int r0 = at + block_scan(n0, buf, total);
        ranks[threadIdx.x] = r0;
        // pages given out so far: the end of the last row that fits
        int fit = n0 > 0 && r0 + n0 <= room ? r0 + n0 : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) fit = max(fit, __shfl_xor_sync(0xffffffffu, fit, o));
        if (lane == 0) buf[warp] = fit;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) used = max(used, buf[w]);
        // every CTA has read the lengths of this step before any row changes
        cl.sync();
        const int end = min(P.rows, base + kThreads);
        for (int i = base + warp * kCtas + rank; i < end; i += kWarps * kCtas) {
            const int need = need_of(i, have);
            const int want = __ldg(a.new_lens + i);
            const int r = ranks[i - base];
            if (pages_of(want) > P.bt_width || (need > 0 && r + need > room)) {
                if (lane == 0)
                    atomicOr(P.status, pages_of(want) > P.bt_width ? kStatusBadBlock : kStatusNoPages);
                continue;
            }
            int32_t* row = P.block_table + (long long)i * P.bt_stride + have;
            for (int c = lane; c < need; c += 32) {
                const int p = a.new_pages[r + c];
                row[c] = p;
                P.ref_counts[p] = 1;
            }
            __syncwarp();
            if (lane == 0) P.seq_lens[i] = max(want, P.seq_lens[i]);
        }
        at += total;
        __syncthreads();
    }
    if (rank == 0) {
        if (threadIdx.x == 0) *a.count = used;
    }
    cl.sync();
    if (rank == 0)
        for (int i = used + threadIdx.x; i < a.capacity; i += kThreads) a.new_pages[i] = -1;
}

// ------------------------------------------------------------------ free

constexpr int kFreeThreads = 128;

// A CTA per request, a thread per page: one load and one atomic deep up to
// 128 pages.
__global__ void __launch_bounds__(kFreeThreads) pages_free_kernel(const FreeArgs a)
{
    allow_dependent_launch();
    grid_dependency_wait();
    const PoolArgs& P = a.pool;
    const int row = __ldg(a.list + blockIdx.x);
    if (row < 0 || row >= P.rows) {
        if (threadIdx.x == 0) atomicOr(P.status, kStatusBadRequest);
        return;
    }
    int n = pages_of(P.seq_lens[row]);
    if (n > P.bt_width) {
        if (threadIdx.x == 0) atomicOr(P.status, kStatusBadBlock);
        n = P.bt_width;
    }
    for (int c = threadIdx.x; c < n; c += kFreeThreads) {
        const int p = P.block_table[(long long)row * P.bt_stride + c];
        bool bad = p < 0 || p >= P.num_pages;
        if (!bad && atomicSub(P.ref_counts + p, 1) <= 0) {   // nobody held it: put it back
            atomicAdd(P.ref_counts + p, 1);
            bad = true;
        }
        if (bad) atomicOr(P.status, kStatusBadBlock);
    }
    __syncthreads();
    if (threadIdx.x == 0) P.seq_lens[row] = 0;
}

// ------------------------------------------------------------------ compact

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    pages_compact_kernel(const CompactArgs a)
{
    __shared__ int buf[kWarps];
    __shared__ int xlive, xmove, xhole;
    allow_dependent_launch();
    grid_dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    const PoolArgs& P = a.pool;
    const Slice s = slice_of(P.num_pages, rank);
    const int cluster_thread = rank * kThreads + threadIdx.x;
    constexpr int kStride = kCtas * kThreads;

    const int live_here = count_slice(s, P.ref_counts, buf, [](int, int c) { return c > 0; });
    int below, live;
    exchange(cl, &xlive, live_here, below, live);

    // pages to move: live ones at or past `live`; where to: free ones below it
    auto moves = [&](int p, int c) { return c > 0 && p >= live; };
    auto hole = [&](int p, int c) { return c <= 0 && p < live; };
    const int moves_here = count_slice(s, P.ref_counts, buf, moves);
    const int holes_here = count_slice(s, P.ref_counts, buf, hole);
    if (threadIdx.x == 0) xhole = holes_here;
    int mbelow, moved, hbelow = 0;
    exchange(cl, &xmove, moves_here, mbelow, moved);
    for (int r = 0; r < rank; ++r) hbelow += *cl.map_shared_rank(&xhole, r);
    emit_slice(s, P.ref_counts, buf, mbelow, a.capacity, moves, [&](int r, int p) { a.src[r] = p; });
    emit_slice(s, P.ref_counts, buf, hbelow, a.capacity, hole, [&](int r, int p) { a.dst[r] = p; });

    // pages that stay, and free ones
    for (int p = s.begin + threadIdx.x; p < s.end; p += kThreads) {
        const int c = P.ref_counts[p];
        if (c > 0 && p >= live) continue;
        a.remap[p] = c > 0 ? p : -1;
        if (c > 0 || p >= live) a.ref_counts_out[p] = c > 0 ? c : 0;
    }
    for (int i = moved + cluster_thread; i < a.capacity; i += kStride) {
        a.src[i] = -1;
        a.dst[i] = -1;
    }
    if (cluster_thread == 0) *a.count = moved;
    __threadfence();
    cl.sync();
    // pages that move (in place, too: no page is both a source and a target)
    for (int i = cluster_thread; i < moved; i += kStride) {
        const int from = a.src[i], to = a.dst[i];
        const int c = P.ref_counts[from];
        a.remap[from] = to;
        a.ref_counts_out[to] = c;
        a.ref_counts_out[from] = 0;
    }
    __threadfence();
    cl.sync();
    // the tables, an entry per thread, a few on their way at once
    const long long entries = (long long)P.rows * P.bt_width;
    for (long long e0 = cluster_thread; e0 < entries; e0 += (long long)kStride * kAhead) {
        int p[kAhead], at[kAhead], row[kAhead];
        bool used[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            used[k] = false;
            if (e0 + (long long)k * kStride >= entries) continue;
            const int e = (int)(e0 + (long long)k * kStride);
            row[k] = e / P.bt_width;
            at[k] = e - row[k] * P.bt_width;
            p[k] = P.block_table[row[k] * P.bt_stride + at[k]];
            used[k] = at[k] < pages_of(P.seq_lens[row[k]]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool there = p[k] >= 0 && p[k] < P.num_pages;
            if (used[k] && there) p[k] = a.remap[p[k]];
            else if (used[k]) atomicOr(P.status, kStatusBadBlock);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (e0 + (long long)k * kStride < entries)
                a.block_table_out[row[k] * a.bt_out_stride + at[k]] = p[k];
    }
}

// ------------------------------------------------------------------ copy

template <int VEC>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<1> { using type = uint8_t; };

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// Items of (pair, layer, piece of a page), dealt to the CTAs in turn.
template <int VEC>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyPagesArgs a,
                                                                  long long words, int pieces)
{
    using W = typename Word<VEC>::type;
    constexpr int kPiece = kCopyThreads * kCopyUnroll;
    allow_dependent_launch();
    grid_dependency_wait();
    const long long n = min(max(*a.count, 0), a.capacity);
    const long long items = n * a.layers * pieces;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int piece = (int)(it % pieces);
        const long long pl = it / pieces;
        const int layer = (int)(pl % a.layers);
        const int i = (int)(pl / a.layers);
        const int from = __ldg(a.src + i), to = __ldg(a.dst + i);
        if (from < 0 || to < 0 || from >= a.num_pages || to >= a.num_pages) {
            if (threadIdx.x == 0) atomicOr(a.status, kStatusBadBlock);
            continue;
        }
        const W* src = reinterpret_cast<const W*>(a.cache + layer * a.layer_stride + from * a.page_stride);
        W* dst = reinterpret_cast<W*>(a.cache + layer * a.layer_stride + to * a.page_stride);
        const long long w0 = (long long)piece * kPiece + threadIdx.x;
        W v[kCopyUnroll];
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k)
            if (w0 + k * kCopyThreads < words) v[k] = src[w0 + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k)
            if (w0 + k * kCopyThreads < words) dst[w0 + k * kCopyThreads] = v[k];
    }
}

template <int VEC>
cudaError_t launch_copy(const CopyPagesArgs& a, int sm_count, cudaStream_t stream)
{
    const long long words = a.page_bytes / VEC;
    const long long pieces = (words + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll);
    if (pieces > 0x7fffffffLL) return cudaErrorInvalidValue;
    long long grid = (long long)a.capacity * a.layers * pieces;
    if (grid > (long long)sm_count * 8) grid = (long long)sm_count * 8;
    return launch_dependent(pages_copy_kernel<VEC>, dim3((unsigned)grid), kCopyThreads, 0, stream, a, words,
                            (int)pieces);
}

}  // namespace

cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t stream)
{
    return launch_dependent(pages_fork_kernel, dim3(kCtas), kThreads, 0, stream, a);
}

cudaError_t launch_pages_extend(const ExtendArgs& a, cudaStream_t stream)
{
    return launch_dependent(pages_extend_kernel, dim3(kCtas), kThreads, 0, stream, a);
}

cudaError_t launch_pages_free(const FreeArgs& a, cudaStream_t stream)
{
    return launch_dependent(pages_free_kernel, dim3((unsigned)a.n), kFreeThreads, 0, stream, a);
}

cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream)
{
    return launch_dependent(pages_compact_kernel, dim3(kCtas), kThreads, 0, stream, a);
}

cudaError_t launch_pages_copy(const CopyPagesArgs& a, int sm_count, cudaStream_t stream)
{
    switch (a.vec) {
    case 16: return launch_copy<16>(a, sm_count, stream);
    case 4: return launch_copy<4>(a, sm_count, stream);
    default: return launch_copy<1>(a, sm_count, stream);
    }
}

}  // namespace pml
