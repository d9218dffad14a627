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
constexpr int kJoinSplit = 8;     // CTAs that share one item's rows

// A CTA whose range ended inside an item it had begun (slot 1) owns the join:
// the item's other pieces are slot 0 of the following CTAs, up to the one
// that holds its end.  A warp takes a row: lanes hold the pieces' maxima and
// sums, then D / 32 columns each.
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
    if (end >= num_ctas) return;      // never: an item's end is in some range
    const int pieces = end - owner + 1;
    const int G = a.group;
    constexpr int V = D / 32;
    for (int r = blockIdx.y * kJoinWarps + warp; r < ntok * G; r += gridDim.y * kJoinWarps) {
        const int i = r / G, g = r - i * G;
        const int half = i / a.half_tokens;
        const int row = half * kAttnHalfRows + (i - half * a.half_tokens) * G + g;
        // piece p: slot 1 of the owner, then slot 0 of its followers
        auto ws = [&](int p) {
            return ((owner + p) * 2LL + (p == 0 ? 1 : 0)) * kAttnSlotRows + row;
        };
        float top = -INFINITY;
        for (int p = lane; p < pieces; p += 32) top = fmaxf(top, a.stats[ws(p)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.0f, acc[V] = {};
        for (int p0 = 0; p0 < pieces; p0 += 32) {
            float f = 0.0f;
            if (p0 + lane < pieces) {
                const float2 s = a.stats[ws(p0 + lane)];
                if (s.x != -INFINITY) f = exp2_approx((s.x - top) * a.scale_log2);
                sum += s.y * f;
            }
            const int here = min(32, pieces - p0);
            for (int p = 0; p < here; ++p) {
                const float fp = __shfl_sync(0xffffffffu, f, p);
                const float* o = a.partial + ws(p0 + p) * D + lane * V;
                if constexpr (V == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(o);
                    acc[0] = fmaf(v.x, fp, acc[0]);
                    acc[1] = fmaf(v.y, fp, acc[1]);
                    acc[2] = fmaf(v.z, fp, acc[2]);
                    acc[3] = fmaf(v.w, fp, acc[3]);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(o);
                    acc[0] = fmaf(v.x, fp, acc[0]);
                    acc[1] = fmaf(v.y, fp, acc[1]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        const long long token = tok0 + i;
        const int qhead = head * G + g;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + token * a.out_token +
                                                    qhead * a.out_head + lane * V);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) out[e] = pack16<FP16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        if (lane == 0 && a.lse != nullptr)
            a.lse[token * a.kv_heads * G + qhead] =
                sum == 0.0f ? -INFINITY : top * a.scale + logf(sum);
    }
}

template <int D, bool FP16>
cudaError_t launch_join(const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    return launch_dependent(attention_join_kernel<D, FP16>, dim3((unsigned)num_ctas, kJoinSplit),
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
