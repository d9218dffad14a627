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
// that holds its end.  A CTA here takes 16 columns of an item's rows; a warp
// 32 rows (neighbours in the workspace), and where the rows leave warps over
// (a single token's few rows in many pieces) each a part of the pieces, in
// the order of their numbers, joined through shared memory.  Bound by the
// latency of dependent loads: the records of the owner and of the CTAs after
// it, then maxima, sums and values at once (one pass with a running maximum).
template <int D, bool FP16>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const AttnArgs a, int num_ctas)
{
    __shared__ float part[kJoinWarps][18][32];
    allow_dependent_launch();
    grid_dependency_wait();
    const int owner = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4* rec = reinterpret_cast<const int4*>(a.pieces + (owner * 2LL + 1) * kPieceInts);
    const int4 r0 = rec[0];                       // used, first token, tokens, kv head
    // the first CTA after the owner that holds the item's end
    auto ends = [&](int cta) {
        if (cta >= num_ctas) return false;
        const int* p = a.pieces + cta * 2LL * kPieceInts;
        return p[kPcUsed] && p[kPcLast];
    };
    unsigned who = __ballot_sync(0xffffffffu, ends(owner + 1 + lane));
    if (!r0.x) return;
    int end = owner + 1;
    while (!who && end + 32 < num_ctas) {
        end += 32;
        who = __ballot_sync(0xffffffffu, ends(end + lane));
    }
    if (!who) return;                             // never: an item's end is in some range
    end += __ffs(who) - 1;
    const int pieces = end - owner + 1;
    const int tok0 = r0.y, ntok = r0.z, head = r0.w;
    const int G = a.group;
    // groups of 32 rows, first half 0's, then half 1's; the pieces' parts
    const int rows0 = min(ntok, a.half_tokens) * G, rows1 = max(ntok - a.half_tokens, 0) * G;
    const int groups0 = (rows0 + 31) >> 5, groups = groups0 + ((rows1 + 31) >> 5);
    const int groups_log2 = groups <= 1 ? 0 : 32 - __clz(groups - 1);
    const int grp = warp & ((1 << groups_log2) - 1), split = warp >> groups_log2;
    const int splits = kJoinWarps >> groups_log2;
    const int half = grp >= groups0 ? 1 : 0;
    const int in_half = (grp - half * groups0) * 32 + lane;
    const bool valid = grp < groups && in_half < (half ? rows1 : rows0);
    const int row = half * kAttnHalfRows + in_half;
    const int cols = blockIdx.y * 16;
    const int p0 = pieces * split / splits, p1 = pieces * (split + 1) / splits;
    float top = -INFINITY, sum = 0.0f, acc[16] = {};
    auto add = [&](float m, float l, const float (&v)[16]) {
        const float next = fmaxf(top, m);
        const float f = top == -INFINITY ? 0.0f : exp2_approx((top - next) * a.scale_log2);
        const float g = m == -INFINITY ? 0.0f : exp2_approx((m - next) * a.scale_log2);
        top = next;
        sum = sum * f + l * g;
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = fmaf(v[k], g, acc[k] * f);
    };
    if (valid) {
#pragma unroll 2
        for (int p = p0; p < p1; ++p) {
            // piece p: slot 1 of the owner, then slot 0 of its followers
            const int slot = p == 0 ? 1 : 0;
            // (a range without a tile's first unit left none)
            const bool used = a.pieces[((owner + p) * 2LL + slot) * kPieceInts + kPcUsed];
            float2 st = a.stats[((owner + p) * 2LL + slot) * kAttnSlotRows + row];
            const float* o = a.partial + partial_at<D>(owner + p, slot, cols / 4, row);
            float v[16];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(v + 4 * k) = *reinterpret_cast<const float4*>(o + k * 4 * kAttnSlotRows);
            if (!used) {
                st = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = 0.0f;
            }
            add(st.x, st.y, v);
        }
    }
    if (splits > 1) {
        if (split > 0) {
            part[warp][16][lane] = top;
            part[warp][17][lane] = sum;
#pragma unroll
            for (int k = 0; k < 16; ++k) part[warp][k][lane] = acc[k];
        }
        __syncthreads();
        if (split > 0) return;
        for (int q = 1; q < splits; ++q) {
            const int w = (q << groups_log2) + grp;
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = part[w][k][lane];
            add(part[w][16][lane], part[w][17][lane], v);
        }
    }
    if (!valid) return;
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int i = half * a.half_tokens + in_half / G, g = in_half % G;
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
    return launch_dependent(attention_join_kernel<D, FP16>, dim3((unsigned)num_ctas, D / 16),
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
