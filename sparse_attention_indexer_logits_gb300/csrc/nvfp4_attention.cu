// Dispatch of the attention over caches held in 4 bits, and the kernel that
// joins the pieces of items that several CTAs shared.
#include "nvfp4_attention.cuh"

namespace pml {

template <int D>
cudaError_t launch_nvfp4_attention_dim(bool fp16, int tiles, const NvAttnArgs& a, const nvattn::Pieces& wp,
                                       const nvattn::Pieces& cp, int num_ctas, cudaStream_t stream);
extern template cudaError_t launch_nvfp4_attention_dim<64>(bool, int, const NvAttnArgs&, const nvattn::Pieces&,
                                                           const nvattn::Pieces&, int, cudaStream_t);
extern template cudaError_t launch_nvfp4_attention_dim<128>(bool, int, const NvAttnArgs&, const nvattn::Pieces&,
                                                            const nvattn::Pieces&, int, cudaStream_t);
template <int D>
int nvfp4_clusters_dim(bool select, int tiles, int size);
extern template int nvfp4_clusters_dim<64>(bool, int, int);
extern template int nvfp4_clusters_dim<128>(bool, int, int);

namespace {

using namespace nvattn;

constexpr int kJoinWarps = 8, kJoinRows = 4;
constexpr int kMaxCluster = 8;    // portable (of 16 the device runs 7 at a time)
// The joins' times in steps of a warp: by the second kernel, within a cluster.  One
// token over 4000 keys, 32 / 8 heads of 128, takes 15.2 us cut over all CTAs and
// 12.2 by clusters of eight; over 500 keys 13.5 and 11.4; 16 lists of 2048 for 64
// heads 22.6 whole and 18.1 by clusters of two; 7 lists of 500 for 16 / 2 heads of
// 64 8.3 whole and 9.6 by clusters; one token over 32768 keys 23.6 cut: clusters
// of eight would be of 64 CTAs alone.
constexpr int kJoinSteps = 3, kClusterSteps = 2;

// A CTA whose pieces ended with an item that it had begun (slot 1) owns the
// join: the item's other pieces are slot 0 of the following CTAs, up to the one
// that holds its end.  A CTA here takes four rows, two warps each, which take
// half of the pieces each in the order of their numbers, a lane two or four
// columns.  Bound by the latency of three dependent loads and its launch: about
// 4 us of a call's time, whatever the lengths.
template <int D, bool FP16, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) nvfp4_join_kernel(const NvAttnArgs a, const Pieces cp, int num_ctas)
{
    constexpr int N = D / 32, kRows = 8 * NT;
    __shared__ float part[kJoinRows][N + 2][32];
    allow_dependent_launch();
    grid_dependency_wait();
    const int owner = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.y * kJoinRows + (warp >> 1), half = warp & 1;
    const int* rec = cp.rec + (owner * 2LL + 1) * kPcInts;
    // the first CTA after the owner that holds the item's end
    auto ends = [&](int cta) {
        if (cta >= num_ctas) return false;
        const int* p = cp.rec + cta * 2LL * kPcInts;
        return p[kPcUsed] && p[kPcLast];
    };
    unsigned who = __ballot_sync(0xffffffffu, ends(owner + 1 + lane));
    const int rows = rec[kPcNtok] * rec[kPcHeads];
    if (!rec[kPcUsed] || (int)blockIdx.y * kJoinRows >= rows) return;
    int end = owner + 1;
    while (!who && end + 32 < num_ctas) {
        end += 32;
        who = __ballot_sync(0xffffffffu, ends(end + lane));
    }
    if (!who) return;                             // never: an item's end is in some range
    end += __ffs(who) - 1;
    const int pieces = end - owner + 1;
    Joined<N> x;
    if (row < rows) {
        const int last = half ? pieces : pieces / 2;
#pragma unroll 4
        for (int p = half ? pieces / 2 : 0; p < last; ++p) {
            const int slot = p == 0 ? 1 : 0;
            const long long at = (owner + p) * 2LL + slot;
            const bool used = cp.rec[at * kPcInts + kPcUsed];      // (a range without a step left none)
            float2 st = cp.stats[at * kRows + row];
            float v[N];
            load_cols<N>(cp.part + (at * kRows + row) * D + lane * N, v);
            if (!used) {
                st = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = 0.0f;
            }
            x.add(st.x, st.y, v, a.scale_log2);
        }
    }
    if (half) {
        part[warp >> 1][0][lane] = x.top;
        part[warp >> 1][1][lane] = x.sum;
#pragma unroll
        for (int k = 0; k < N; ++k) part[warp >> 1][2 + k][lane] = x.acc[k];
    }
    __syncthreads();
    if (half || row >= rows) return;
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = part[warp >> 1][2 + k][lane];
    x.add(part[warp >> 1][0][lane], part[warp >> 1][1][lane], v, a.scale_log2);
    write_joined<FP16, N>(a, x, rec[kPcTok0], rec[kPcHead], rec[kPcHeads], row, lane * N);
}

template <int D, bool FP16, int NT>
cudaError_t launch_join(const NvAttnArgs& a, const Pieces& cp, int num_ctas, cudaStream_t stream)
{
    return launch_dependent(nvfp4_join_kernel<D, FP16, NT>, dim3((unsigned)num_ctas, 8 * NT / kJoinRows), kJoinWarps * 32, 0,
                            stream, a, cp, num_ctas);
}

template <int D>
cudaError_t launch_join_dim(bool fp16, int tiles, const NvAttnArgs& a, const Pieces& cp, int num_ctas,
                            cudaStream_t stream)
{
    if (tiles == 1)
        return fp16 ? launch_join<D, true, 1>(a, cp, num_ctas, stream) : launch_join<D, false, 1>(a, cp, num_ctas, stream);
    return fp16 ? launch_join<D, true, 2>(a, cp, num_ctas, stream) : launch_join<D, false, 2>(a, cp, num_ctas, stream);
}

// `n` pieces from `at` on, the rows of `slots` of their two slots.
Pieces take(uint8_t*& at, int64_t n, int slots, int rows, int dim)
{
    Pieces p;
    p.part = reinterpret_cast<float*>(at);
    at += n * slots * rows * dim * 4;
    p.stats = reinterpret_cast<float2*>(at);
    at += n * slots * rows * 8;
    p.rec = nullptr;
    if (slots == 2) {                // (those of one are the CTA's own matter)
        p.rec = reinterpret_cast<int*>(at);
        at += n * 2 * kPcInts * 4;
    }
    return p;
}

}  // namespace

// (what the choice of the way counts with)
static_assert(Cfg<128, 2>::kWarps == 12 && Cfg<128, 2>::kRows == 16 && kStepKeys == 32, "steps of a warp");

cudaError_t launch_nvfp4_attention(int head_dim, bool fp16, NvAttnArgs& a, int num_ctas, void* workspace,
                                   int64_t workspace_bytes, cudaStream_t stream)
{
    const bool large = a.selected ? a.group > 8 : nvfp4_large_items(a.tokens, a.batch, a.group);
    const int tiles = large ? 2 : 1, rows = 8 * tiles;
    a.head_blocks = (a.group + rows - 1) / rows;
    a.block_heads = (a.group + a.head_blocks - 1) / a.head_blocks;
    a.tile_tokens = a.selected || a.group > rows ? 1 : rows / a.group;
    const int warps = tiles == 1 ? Cfg<128, 1>::kWarps : Cfg<128, 2>::kWarps;
    // Whether the steps are cut without regard to items, which a second kernel joins,
    // or an item is one CTA's or one cluster's, by a warp's most steps and the join.
    // Lists have equally many each; of one request the longest its table allows
    // counts; several requests may differ by any factor and are cut.
    const long long items = a.selected ? (long long)a.tokens * a.kv_heads * a.head_blocks
                                       : (long long)((a.tokens + a.tile_tokens - 1) / a.tile_tokens) * a.kv_heads * a.head_blocks;
    const long long steps = (a.selected ? (a.sel_k + kStepKeys - 1) / kStepKeys : 2LL * a.bt_width) + kItemUnits;
    int grid = num_ctas;
    if (a.selected || a.batch == 1) {
        double best = (double)items * steps / ((double)num_ctas * warps) + kJoinSteps;
        if (a.selected) {
            const double whole = (double)((items + num_ctas - 1) / num_ctas * steps) / warps;
            a.whole_items = whole <= best;
            if (a.whole_items) best = whole;
        }
        for (int size = 2; size <= kMaxCluster && items * size <= num_ctas; size *= 2) {
            const double mine = (double)steps / (size * warps) + kClusterSteps;
            if (mine >= best) continue;
            if ((head_dim == 128 ? nvfp4_clusters_dim<128>(a.selected, tiles, size)
                                 : nvfp4_clusters_dim<64>(a.selected, tiles, size)) < items)
                continue;
            best = mine;
            a.cluster = size;
            a.whole_items = 0;
            grid = (int)items * size;
        }
    }
    uint8_t* at = static_cast<uint8_t*>(workspace);
    const Pieces wp = take(at, (int64_t)num_ctas * warps, 1, rows, head_dim);
    const Pieces cp = take(at, num_ctas, 2, rows, head_dim);
    if (at - static_cast<uint8_t*>(workspace) > workspace_bytes) return cudaErrorInvalidValue;    // never
    cudaError_t e = head_dim == 128 ? launch_nvfp4_attention_dim<128>(fp16, tiles, a, wp, cp, grid, stream)
                                    : launch_nvfp4_attention_dim<64>(fp16, tiles, a, wp, cp, grid, stream);
    if (e != cudaSuccess || a.whole_items || a.cluster > 1) return e;
    return head_dim == 128 ? launch_join_dim<128>(fp16, tiles, a, cp, num_ctas, stream)
                           : launch_join_dim<64>(fp16, tiles, a, cp, num_ctas, stream);
}

}  // namespace pml
