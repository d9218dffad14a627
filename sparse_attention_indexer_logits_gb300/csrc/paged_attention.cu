// Dispatch of the attention over pages, and the kernel that joins the pieces
// of items that several CTAs shared.
#include "paged_attention.cuh"

namespace pml {

cudaError_t launch_attention_d64(bool, bool, const CUtensorMap&, const CUtensorMap&,
                                 const CUtensorMap&, const AttnArgs&, int, cudaStream_t);
cudaError_t launch_attention_d128(bool, bool, const CUtensorMap&, const CUtensorMap&,
                                  const CUtensorMap&, const AttnArgs&, int, cudaStream_t);

cudaError_t launch_attention_nvfp4_d64(bool, bool, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const AttnArgs&, int, cudaStream_t);
cudaError_t launch_attention_nvfp4_d128(bool, bool, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const AttnArgs&, int, cudaStream_t);

namespace {

using namespace attn;

constexpr int kJoinWarps = 8;

// Parts of a row joined in turn: N of its columns under a running maximum.
template <int N>
struct Joined {
    float top = -INFINITY, sum = 0.0f, acc[N] = {};

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
    // through shared memory, a warp's lanes side by side
    __device__ void put(float (*part)[32], int lane) const
    {
        part[0][lane] = top;
        part[1][lane] = sum;
#pragma unroll
        for (int k = 0; k < N; ++k) part[2 + k][lane] = acc[k];
    }
    __device__ void take(const float (*part)[32], int lane, float scale_log2)
    {
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = part[2 + k][lane];
        add(part[0][lane], part[1][lane], v, scale_log2);
    }
    __device__ float inverse(float scale) const { return sum > 0.0f || sum != sum ? scale / sum : 0.0f; }
    __device__ float log_sum(float scale, float sum_scale) const
    {
        return sum == 0.0f ? -INFINITY : top * scale + logf(sum * sum_scale);
    }

    // Pieces p0 .. p1 - 1 of an item: slot 1 of its owner, then slot 0 of the
    // following CTAs (a range without a tile's first unit left none), from
    // column `col` of row `row` on.
    template <int D>
    __device__ void add_pieces(const AttnArgs& a, int owner, int p0, int p1, int row, int col)
    {
#pragma unroll 2
        for (int p = p0; p < p1; ++p) {
            const int slot = p == 0 ? 1 : 0;
            const bool used = a.pieces[((owner + p) * 2LL + slot) * kPieceInts + kPcUsed];
            float2 st = a.stats[((owner + p) * 2LL + slot) * kAttnSlotRows + row];
            const float* o = a.partial + partial_at<D>(owner + p, slot, col / 4, row);
            float v[N];
#pragma unroll
            for (int k = 0; k < N / 4; ++k)
                *reinterpret_cast<float4*>(v + 4 * k) = *reinterpret_cast<const float4*>(o + k * 4 * kAttnSlotRows);
            if (!used) {
                st = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = 0.0f;
            }
            add(st.x, st.y, v, a.scale_log2);
        }
    }
};

// A CTA whose range ended inside an item it had begun (slot 1) owns the join:
// the item's other pieces are slot 0 of the following CTAs, up to the one
// that holds its end.  A CTA here takes 16 columns of an item's rows; a warp
// 32 rows (neighbours in the workspace), and where the rows leave warps over
// (a single token's few rows in many pieces) each a part of the pieces, in
// the order of their numbers, joined through shared memory.  Bound by the
// latency of dependent loads: the records of the owner and of the CTAs after
// it, then maxima, sums and values at once (one pass with a running maximum).
// (P16: P was fp16, whatever the output's type.)
template <int D, bool FP16, bool P16>
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
    const int cols = blockIdx.y * 16;
    uint16_t* out = static_cast<uint16_t*>(a.out) + cols;
    if (ntok * G <= 8) {
        // A single token's few rows, often in many pieces: a lane has a row
        // and four columns, a warp an eighth of the pieces.  One request of
        // 32000 keys, five heads to a kv head, takes 19.2 us this way and 21.4
        // with a row's sixteen columns to a lane (most of which have no row);
        // 64 requests of 100 to 800 keys 26.1 and 27.0.
        const int row = lane & 7, at = lane >> 3;
        const bool valid = row < ntok * G;
        Joined<4> x;
        if (valid)
            x.template add_pieces<D>(a, owner, pieces * warp / kJoinWarps, pieces * (warp + 1) / kJoinWarps, row,
                                     cols + 4 * at);
        if (warp > 0) x.put(part[warp], lane);
        __syncthreads();
        if (warp > 0) return;
        for (int q = 1; q < kJoinWarps; ++q) x.take(part[q], lane, a.scale_log2);
        if (!valid) return;
        const float inv = x.inverse(a.out_scale);
        const int i = row / G, g = row % G;
        const long long token = tok0 + i;
        const int qhead = head * G + g;
        *reinterpret_cast<uint2*>(out + token * a.out_token + qhead * a.out_head + 4 * at) =
            make_uint2(pack16<FP16>(x.acc[0] * inv, x.acc[1] * inv), pack16<FP16>(x.acc[2] * inv, x.acc[3] * inv));
        if (cols + at == 0 && a.lse != nullptr) a.lse[token * a.kv_heads * G + qhead] = x.log_sum(a.scale, PScale<P16>::kInverse);
        return;
    }
    // groups of 32 rows, first half 0's, then half 1's; the pieces' parts
    const int rows0 = min(ntok, a.half_tokens) * G, rows1 = max(ntok - a.half_tokens, 0) * G;
    const int groups0 = (rows0 + 31) >> 5, groups = groups0 + ((rows1 + 31) >> 5);
    const int groups_log2 = groups <= 1 ? 0 : 32 - __clz(groups - 1);
    const int grp = warp & ((1 << groups_log2) - 1), split = warp >> groups_log2;
    const int splits = kJoinWarps >> groups_log2;
    const int half = grp >= groups0 ? 1 : 0;
    const int in_half = (grp - half * groups0) * 32 + lane;
    const bool valid = grp < groups && in_half < (half ? rows1 : rows0);
    Joined<16> x;
    if (valid)
        x.template add_pieces<D>(a, owner, pieces * split / splits, pieces * (split + 1) / splits,
                                 half * kAttnHalfRows + in_half, cols);
    if (splits > 1) {
        if (split > 0) x.put(part[warp], lane);
        __syncthreads();
        if (split > 0) return;
        for (int q = 1; q < splits; ++q) x.take(part[(q << groups_log2) + grp], lane, a.scale_log2);
    }
    if (!valid) return;
    const float inv = x.inverse(a.out_scale);
    const int i = half * a.half_tokens + in_half / G, g = in_half % G;
    const long long token = tok0 + i;
    const int qhead = head * G + g;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack16<FP16>(x.acc[2 * e] * inv, x.acc[2 * e + 1] * inv);
    uint4* dst = reinterpret_cast<uint4*>(out + token * a.out_token + qhead * a.out_head);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (cols == 0 && a.lse != nullptr) a.lse[token * a.kv_heads * G + qhead] = x.log_sum(a.scale, PScale<P16>::kInverse);
}

template <int D, bool FP16, bool P16>
cudaError_t launch_join(const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    return launch_dependent(attention_join_kernel<D, FP16, P16>, dim3((unsigned)num_ctas, D / 16),
                            kJoinWarps * 32, 0, stream, a, num_ctas);
}

template <int D>
cudaError_t join(bool fp16, bool p16, const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    return fp16 ? launch_join<D, true, true>(a, num_ctas, stream)
           : p16 ? launch_join<D, false, true>(a, num_ctas, stream)
                 : launch_join<D, false, false>(a, num_ctas, stream);
}

}  // namespace

cudaError_t launch_paged_attention(int head_dim, bool fp16, bool select, const CUtensorMap& qmap,
                                   const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   const AttnArgs& a, int num_ctas, cudaStream_t stream)
{
    const cudaError_t e = head_dim == 128
                              ? launch_attention_d128(fp16, select, qmap, kmap, vmap, a, num_ctas, stream)
                              : launch_attention_d64(fp16, select, qmap, kmap, vmap, a, num_ctas, stream);
    if (e != cudaSuccess) return e;
    return head_dim == 128 ? join<128>(fp16, fp16, a, num_ctas, stream) : join<64>(fp16, fp16, a, num_ctas, stream);
}

cudaError_t launch_paged_attention_nvfp4(int head_dim, bool fp16, bool select, const CUtensorMap& qmap,
                                         const CUtensorMap& kmap, const CUtensorMap& vmap, const AttnArgs& a,
                                         int num_ctas, cudaStream_t stream)
{
    const cudaError_t e = head_dim == 128
                              ? launch_attention_nvfp4_d128(fp16, select, qmap, kmap, vmap, a, num_ctas, stream)
                              : launch_attention_nvfp4_d64(fp16, select, qmap, kmap, vmap, a, num_ctas, stream);
    if (e != cudaSuccess) return e;
    return head_dim == 128 ? join<128>(fp16, true, a, num_ctas, stream) : join<64>(fp16, true, a, num_ctas, stream);
}

}  // namespace pml
