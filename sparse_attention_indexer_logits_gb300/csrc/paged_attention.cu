// Dispatch of the attention over pages, and the kernel that joins the pieces
// of items that several CTAs shared.
#include "paged_attention.cuh"

namespace pml {

cudaError_t launch_attention_d64(bool, bool, const CUtensorMap&, const CUtensorMap&,
                                 const CUtensorMap&, const AttnArgs&, int, cudaStream_t);
cudaError_t launch_attention_d128(bool, bool, const CUtensorMap&, const CUtensorMap&,
                                  const CUtensorMap&, const AttnArgs&, int, cudaStream_t);

namespace {

using namespace attn;

constexpr int kJoinWarps = 8;

// A CTA whose range ended inside an item it had begun (slot 1) owns the join:
// the item's other pieces are slot 0 of the following CTAs, up to the one
// that holds its end.  A warp takes 32 rows (neighbours in the workspace) and
// 16 columns; a lane goes over its row's pieces twice, for the maximum and
// for the weighted sum.
template <int D, bool FP16>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const AttnArgs a, int num_ctas)
{
    allow_dependent_launch();
    grid_dependency_wait();
    const int owner = blockIdx.x;
    const int* rec = a.pieces + (owner * 2LL + 1) * kPieceInts;
    if (!rec[kPcUsed]) return;
    const int tok0 = rec[kPcTok0], ntok = rec[kPcNtok], head = rec[kPcHead];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group;
    const int half_rows = a.half_tokens * G;      // rows in use of a half
    constexpr int kColGroups = D / 16;
    // groups of 32 rows, four to a half
    const int unit = blockIdx.y * kJoinWarps + warp;
    const int cols = unit % kColGroups * 16, row = unit / kColGroups * 32 + lane;
    const int in_half = row % kAttnHalfRows;
    const int i = row / kAttnHalfRows * a.half_tokens + in_half / G, g = in_half % G;
    const bool valid = in_half < half_rows && i < ntok;
    if (!__any_sync(0xffffffffu, valid)) return;
    int end = owner + 1;              // the CTA that holds the item's end
    for (; end < num_ctas; end += 32) {
        const int cta = end + lane;
        const bool here = cta < num_ctas && a.pieces[cta * 2LL * kPieceInts + kPcLast] &&
                          a.pieces[cta * 2LL * kPieceInts + kPcUsed];
        const unsigned who = __ballot_sync(0xffffffffu, here);
        if (who) {
            end += __ffs(who) - 1;
            break;
        }
    }
    if (end >= num_ctas || !valid) return;      // (an item's end is in some range)
    const int pieces = end - owner + 1;
    // piece p: slot 1 of the owner, then slot 0 of its followers
    auto stat = [&](int p) {
        return a.stats[((owner + p) * 2LL + (p == 0 ? 1 : 0)) * kAttnSlotRows + row];
    };
    float top = -INFINITY;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) top = fmaxf(top, stat(p).x);
    float sum = 0.0f, acc[16] = {};
#pragma unroll 2
    for (int p = 0; p < pieces; ++p) {
        const float2 s = stat(p);
        const float f = s.x == -INFINITY ? 0.0f : exp2_approx((s.x - top) * a.scale_log2);
        sum += s.y * f;
        const float* o = a.partial + partial_at<D>(owner + p, p == 0 ? 1 : 0, cols / 4, row);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(o + k * 4 * kAttnSlotRows);
            acc[4 * k] = fmaf(v.x, f, acc[4 * k]);
            acc[4 * k + 1] = fmaf(v.y, f, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(v.z, f, acc[4 * k + 2]);
            acc[4 * k + 3] = fmaf(v.w, f, acc[4 * k + 3]);
        }
    }
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const long long token = tok0 + i;
    const int qhead = head * G + g;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack16<FP16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + token * a.out_token +
                                          qhead * a.out_head + cols);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (cols == 0 && a.lse != nullptr)
        a.lse[token * a.kv_heads * G + qhead] = sum == 0.0f ? -INFINITY : top * a.scale + logf(sum);
}

template <int D, bool FP16>
cudaError_t launch_join(const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    return launch_dependent(attention_join_kernel<D, FP16>, dim3((unsigned)num_ctas, kAttnSlotRows / 32 * (D / 16) / kJoinWarps),
                            kJoinWarps * 32, 0, stream, a, num_ctas);
}

}  // namespace

cudaError_t launch_paged_attention(int head_dim, bool fp16, bool select, const CUtensorMap& qmap,
                                   const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    cudaError_t e = head_dim == 128
                        ? launch_attention_d128(fp16, select, qmap, kmap, vmap, a, num_ctas, stream)
                        : launch_attention_d64(fp16, select, qmap, kmap, vmap, a, num_ctas, stream);
    if (e != cudaSuccess) return e;
    if (head_dim == 128)
        return fp16 ? launch_join<128, true>(a, num_ctas, stream) : launch_join<128, false>(a, num_ctas, stream);
    return fp16 ? launch_join<64, true>(a, num_ctas, stream) : launch_join<64, false>(a, num_ctas, stream);
}

}  // namespace pml
