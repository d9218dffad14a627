// C ABI of the serving operators (declared in include/pml.h): argument
// checks, choice of access width and launches.  No allocation, no
// synchronisation.
#include <cuda_runtime.h>

#include "common.cuh"
#include "host.h"
#include "pml.h"
#include "serving.h"

namespace {

using namespace pml;

constexpr int kMaxRopeDim = 512;
constexpr int kMaxListed = 0x7fffff00; // entries of a list, so that their tiles' ends fit an int
constexpr int kRopeMaxRows = 32768;    // of a token: the kernels divide by it in fp32

int check_rotary(const void* positions, const void* inv_freq, int positions_64, int freq_64,
                 int rot_dim, int rot_offset, int head_dim)
{
    if (rot_dim < 0 || (rot_dim & 1) || rot_offset < 0 || rot_dim + rot_offset > head_dim)
        return PML_ERR_INVALID_ARG;
    if (!positions || (rot_dim > 0 && !inv_freq)) return PML_ERR_INVALID_ARG;
    if (!aligned(positions, positions_64 ? 8 : 4) || !aligned(inv_freq, freq_64 ? 8 : 4))
        return PML_ERR_ALIGNMENT;
    return PML_OK;
}

RotaryArgs rotary(const void* positions, int positions_64, const void* inv_freq, int freq_64,
                  int rot_dim, int rot_offset, int interleaved, float mscale, int gradient)
{
    RotaryArgs r;
    r.positions = positions;
    r.inv_freq = inv_freq;
    r.pos64 = positions_64 ? 1 : 0;
    r.freq64 = freq_64 ? 1 : 0;
    r.half = rot_dim / 2;
    r.offset = rot_offset;
    r.interleaved = interleaved ? 1 : 0;
    r.mscale = mscale;
    r.sign = gradient ? -1.0f : 1.0f;
    return r;
}

// Whether `vec`-element accesses fit a row set: its pointers and strides.
bool rows_fit(const RopeRows& r, int elem, int vec)
{
    const uintptr_t bytes = (uintptr_t)elem * vec;
    return r.heads == 0 || (aligned(r.src, bytes) && aligned(r.dst, bytes) &&
                            r.src_token % vec == 0 && r.src_head % vec == 0 &&
                            r.dst_token % vec == 0 && r.dst_head % vec == 0 && r.dst_page % vec == 0);
}

// The widest access that divides the heads' parts and every address: 16
// bytes, two elements or one.
int rope_vec(const RopeArgs& a)
{
    const int wide = 16 / a.elem;
    const int pairs = a.rot.interleaved ? 2 * a.rot.half : a.rot.half;
    for (int v : {wide, 2}) {
        if (pairs % v || a.rot.offset % v || a.dim % v || (a.dim - 2 * a.rot.half) % v) continue;
        if (rows_fit(a.q, a.elem, v) && rows_fit(a.k, a.elem, v) && rows_fit(a.v, a.elem, v)) return v;
    }
    return 1;
}

// Rows of a CTA that takes `side` at once: `units` times that, fewer if that
// would leave SMs without work, and no more than lie in max_tokens tokens
// wherever the first one begins.
int cta_rows(int units, int side, long long rows_per_token, int max_tokens, long long tokens, int sm_count)
{
    while (units > 1 && tokens * rows_per_token < (long long)units * side * 2 * sm_count) --units;
    const long long most = (max_tokens - 1) * rows_per_token + 1;
    const long long rows = (long long)units * side;
    return (int)(rows < most ? rows : most);
}

int dtype_bytes(int dtype)
{
    return dtype == PML_DTYPE_FLOAT32 ? 4
           : dtype == PML_DTYPE_BFLOAT16 || dtype == PML_DTYPE_FLOAT16 ? 2 : 0;
}

int rope_launch(RopeArgs& a, void* stream)
{
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    a.slot.status = dev.status;
    a.vec = rope_vec(a);
    // a row's units of two accesses: those that turn, then the rest
    const int rot = 2 * a.rot.half;
    const int turn = a.rot.interleaved && a.vec > 1 ? 0 : a.rot.half / a.vec;
    const int rest = (turn ? a.dim - rot : a.dim) / a.vec;
    int units = turn + (rest + 1) / 2;
    if (a.paged && units < (a.dim / a.vec + 1) / 2) units = (a.dim / a.vec + 1) / 2;    // v's rows
    while ((1 << a.row_lanes_log2) < units && a.row_lanes_log2 < 8) ++a.row_lanes_log2;
    if ((1 << a.row_lanes_log2) < units) return PML_ERR_UNSUPPORTED;    // never: head_dim <= 512
    const long long rows = a.q.heads + a.k.heads + a.v.heads;
    a.rows_per_cta = cta_rows(kRopeUnits, kRopeThreads >> a.row_lanes_log2, rows, kRopeMaxTokens, a.tokens,
                              dev.sm_count);
    if (a.tokens * rows / a.rows_per_cta >= 0x7fffffffLL) return PML_ERR_UNSUPPORTED;    // CTAs
    e = launch_rope(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int check_pool(const int32_t* ref_counts, int num_pages, const int32_t* block_table,
               int64_t bt_stride, int bt_width, const int32_t* seq_lens, int rows)
{
    if (num_pages < 0 || rows < 0 || bt_width < 0 || bt_stride < bt_width) return PML_ERR_INVALID_ARG;
    if ((num_pages > 0 && !ref_counts) || (rows > 0 && (!block_table || !seq_lens)))
        return PML_ERR_INVALID_ARG;
    if ((long long)rows * (bt_width + 1LL) > 0x7fffffffLL) return PML_ERR_UNSUPPORTED;
    if (!aligned(ref_counts, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return PML_ERR_ALIGNMENT;
    return PML_OK;
}

PoolArgs pool(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
              int bt_width, int32_t* seq_lens, int rows, unsigned int* status)
{
    PoolArgs p;
    p.ref_counts = ref_counts;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.status = status;
    p.bt_stride = bt_stride;
    p.bt_width = bt_width;
    p.num_pages = num_pages;
    p.rows = rows;
    return p;
}

// Strides of a dimension of one element are never used: any valid one will do.
int64_t used(int64_t stride, int64_t size, int64_t other) { return size > 1 ? stride : other; }

// The checks, tensor maps and launches that both attention calls share; `a`
// comes with what is theirs.
int attention_call(AttnArgs& a, const void* q, int64_t q_token, int64_t q_head, const void* k_cache,
                   int64_t k_page, int64_t k_slot, int64_t k_head, const void* v_cache,
                   int64_t v_page, int64_t v_slot, int64_t v_head, int dtype, int64_t num_pages,
                   const int32_t* block_table, int64_t bt_stride, int bt_width,
                   const int32_t* kv_lens, int tokens, int num_heads, int kv_heads, int head_dim,
                   float softmax_scale, void* out, int64_t out_token, int64_t out_head, float* lse,
                   void* workspace, int64_t workspace_bytes, void* stream)
{
    if (tokens < 0 || num_heads < 1 || kv_heads < 1 || num_heads % kv_heads) return PML_ERR_INVALID_ARG;
    if (dtype != PML_DTYPE_BFLOAT16 && dtype != PML_DTYPE_FLOAT16) return PML_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PML_ERR_UNSUPPORTED;
    const int group = num_heads / kv_heads;
    if (group > kAttnHalfRows) return PML_ERR_UNSUPPORTED;
    if (!(softmax_scale > 0.0f) || softmax_scale > 1e30f) return PML_ERR_INVALID_ARG;
    if (tokens == 0) return PML_OK;
    if (!q || !k_cache || !v_cache || !block_table || !kv_lens || !out || !workspace)
        return PML_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > 0x7fffffffLL || bt_width < 1 || bt_stride < bt_width)
        return PML_ERR_INVALID_ARG;
    if (bt_width > 0x7fffffff / kBlockKeys) return PML_ERR_UNSUPPORTED;
    const bool select = a.selected != nullptr;
    // strides in elements, multiples of 16 bytes
    int64_t qs[2] = {used(q_head, num_heads, head_dim), used(q_token, tokens, head_dim)};
    int64_t ks[3] = {k_slot, used(k_head, kv_heads, head_dim), used(k_page, num_pages, head_dim)};
    int64_t vs[3] = {v_slot, used(v_head, kv_heads, head_dim), used(v_page, num_pages, head_dim)};
    for (int64_t s : {qs[0], qs[1], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2]})
        if (s <= 0 || s % 8) return PML_ERR_ALIGNMENT;
    if ((tokens > 1 && out_token % 8) || (num_heads > 1 && out_head % 8)) return PML_ERR_ALIGNMENT;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
        !aligned(kv_lens, 4) || !aligned(a.cu_q, 4))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int num_ctas = dev.sm_count;
    if (workspace_bytes < pml_attention_workspace_bytes(num_ctas, head_dim)) return PML_ERR_INVALID_ARG;

    const int64_t slots = 2LL * num_ctas;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.partial = reinterpret_cast<float*>(ws);
    ws += slots * kAttnSlotRows * head_dim * 4LL;
    a.stats = reinterpret_cast<float2*>(ws);
    ws += slots * kAttnSlotRows * 8;
    a.pieces = reinterpret_cast<int*>(ws);
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_slot = ks[0];
    a.k_head = ks[1];
    a.k_page = ks[2];
    a.v_slot = vs[0];
    a.v_head = vs[1];
    a.v_page = vs[2];
    a.block_table = block_table;
    a.kv_lens = kv_lens;
    a.out = out;
    a.lse = lse;
    a.status = dev.status;
    a.bt_stride = bt_stride;
    a.bt_width = bt_width;
    a.out_token = out_token;
    a.out_head = out_head;
    a.num_pages = num_pages;
    a.tokens = tokens;
    a.kv_heads = kv_heads;
    a.group = group;
    a.half_tokens = kAttnHalfRows / group;
    a.scale = softmax_scale;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;

    const bool fp16 = dtype == PML_DTYPE_FLOAT16;
    const CUtensorMapDataType type = fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap qmap, kmap, vmap;
    {
        const uint64_t dims[3] = {(uint64_t)head_dim, (uint64_t)num_heads, (uint64_t)tokens};
        const uint64_t strides[2] = {(uint64_t)qs[0] * 2, (uint64_t)qs[1] * 2};
        const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)a.half_tokens};
        e = encode_tiled(qmap, type, 3, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    kmap = vmap = qmap;
    for (int i = 0; i < 2 && !select; ++i) {
        const int64_t* s = i ? vs : ks;
        const uint64_t dims[4] = {(uint64_t)head_dim, (uint64_t)kBlockKeys, (uint64_t)kv_heads,
                                  (uint64_t)num_pages};
        const uint64_t strides[3] = {(uint64_t)s[0] * 2, (uint64_t)s[1] * 2, (uint64_t)s[2] * 2};
        const uint32_t box[4] = {64, (uint32_t)kBlockKeys, 1, 1};
        e = encode_tiled(i ? vmap : kmap, type, 4, i ? v_cache : k_cache, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    e = launch_paged_attention(head_dim, fp16, select, qmap, kmap, vmap, a, num_ctas,
                               static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

int pml_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
             int64_t out_token_stride, int64_t out_head_stride, int dtype, const void* positions,
             int positions_64, const void* inv_freq, int freq_64, int rot_dim, int rot_offset,
             int interleaved, float mscale, int gradient, int tokens, int heads, int head_dim,
             void* stream)
{
    if (tokens < 0 || heads < 0 || head_dim < 1) return PML_ERR_INVALID_ARG;
    const int elem = dtype_bytes(dtype);
    if (elem == 0 || head_dim > kMaxRopeDim) return PML_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return PML_OK;
    if (heads > kRopeMaxRows) return PML_ERR_UNSUPPORTED;
    if (!x || !out) return PML_ERR_INVALID_ARG;
    const int rc = check_rotary(positions, inv_freq, positions_64, freq_64, rot_dim, rot_offset, head_dim);
    if (rc != PML_OK) return rc;
    if (!aligned(x, elem) || !aligned(out, elem)) return PML_ERR_ALIGNMENT;
    RopeArgs a = {};
    a.rot = rotary(positions, positions_64, inv_freq, freq_64, rot_dim, rot_offset, interleaved,
                   mscale, gradient);
    a.q = {x, out, x_token_stride, x_head_stride, out_token_stride, out_head_stride, 0, heads};
    a.tokens = tokens;
    a.dim = head_dim;
    a.skip_rest = x == out && x_token_stride == out_token_stride && x_head_stride == out_head_stride;
    a.elem = elem;
    a.fp16 = dtype == PML_DTYPE_FLOAT16;
    return rope_launch(a, stream);
}

int pml_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                    int64_t q_out_token_stride, int64_t q_out_head_stride, const void* k,
                    int64_t k_token_stride, int64_t k_head_stride, const void* v,
                    int64_t v_token_stride, int64_t v_head_stride, int dtype, const void* positions,
                    int positions_64, const int32_t* requests, int num_requests,
                    const void* inv_freq, int freq_64, int rot_dim, int rot_offset, int interleaved,
                    float mscale, void* k_cache, int64_t k_page_stride, int64_t k_slot_stride,
                    int64_t k_cache_head_stride, void* v_cache, int64_t v_page_stride,
                    int64_t v_slot_stride, int64_t v_cache_head_stride, int64_t num_pages,
                    const int32_t* block_table, int64_t bt_stride, int bt_width, int tokens,
                    int num_heads, int kv_heads, int head_dim, void* stream)
{
    if (tokens < 0 || num_heads < 0 || kv_heads < 1 || head_dim < 1) return PML_ERR_INVALID_ARG;
    const int elem = dtype_bytes(dtype);
    if (elem != 2 || head_dim > kMaxRopeDim) return PML_ERR_UNSUPPORTED;
    if (tokens == 0) return PML_OK;
    if (num_heads + 2LL * kv_heads > kRopeMaxRows) return PML_ERR_UNSUPPORTED;
    if (!k || !v || !k_cache || !v_cache || !requests || !block_table) return PML_ERR_INVALID_ARG;
    if (num_heads > 0 && (!q || !q_out)) return PML_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > 0x7fffffffLL || num_requests < 1) return PML_ERR_INVALID_ARG;
    if (bt_width < 1 || bt_stride < bt_width) return PML_ERR_INVALID_ARG;
    const int rc = check_rotary(positions, inv_freq, positions_64, freq_64, rot_dim, rot_offset, head_dim);
    if (rc != PML_OK) return rc;
    if (!aligned(q, elem) || !aligned(q_out, elem) || !aligned(k, elem) || !aligned(v, elem) ||
        !aligned(k_cache, elem) || !aligned(v_cache, elem) || !aligned(requests, 4) ||
        !aligned(block_table, 4))
        return PML_ERR_ALIGNMENT;
    RopeArgs a = {};
    a.rot = rotary(positions, positions_64, inv_freq, freq_64, rot_dim, rot_offset, interleaved,
                   mscale, 0);
    a.slot.requests = requests;
    a.slot.block_table = block_table;
    a.slot.bt_stride = bt_stride;
    a.slot.bt_width = bt_width;
    a.slot.num_pages = num_pages;
    a.slot.num_requests = num_requests;
    a.q = {q, q_out, q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride, 0, num_heads};
    a.k = {k, k_cache, k_token_stride, k_head_stride, k_slot_stride, k_cache_head_stride,
           k_page_stride, kv_heads};
    a.v = {v, v_cache, v_token_stride, v_head_stride, v_slot_stride, v_cache_head_stride,
           v_page_stride, kv_heads};
    a.tokens = tokens;
    a.dim = head_dim;
    a.paged = 1;
    a.skip_rest = num_heads > 0 && q == q_out && q_token_stride == q_out_token_stride &&
                  q_head_stride == q_out_head_stride;
    a.elem = elem;
    a.fp16 = dtype == PML_DTYPE_FLOAT16;
    return rope_launch(a, stream);
}

int pml_index_quant_append(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                           const void* k, int64_t k_token_stride, const float* weights,
                           float weight_scale, const void* positions, int positions_64,
                           const int32_t* requests, int num_requests, const void* inv_freq,
                           int freq_64, int rot_dim, int rot_offset, int interleaved, float mscale,
                           uint8_t* q_out, float* w_out, uint8_t* kv_fused, int64_t num_blocks,
                           const int32_t* block_table, int64_t bt_stride, int bt_width, int tokens,
                           int num_heads, void* stream)
{
    if (tokens < 0 || num_heads < 1) return PML_ERR_INVALID_ARG;
    if (num_heads > 1024) return PML_ERR_UNSUPPORTED;
    if (rot_dim % 16 || rot_offset % 8) return PML_ERR_UNSUPPORTED;
    if (tokens == 0) return PML_OK;
    if (!q || !weights || !q_out || !w_out) return PML_ERR_INVALID_ARG;
    if (k) {
        if (!kv_fused || !requests || !block_table) return PML_ERR_INVALID_ARG;
        if (num_blocks < 1 || num_blocks > 0x7fffffffLL || num_requests < 1) return PML_ERR_INVALID_ARG;
        if (bt_width < 1 || bt_stride < bt_width) return PML_ERR_INVALID_ARG;
    }
    const int rc = check_rotary(positions, inv_freq, positions_64, freq_64, rot_dim, rot_offset, kHeadDim);
    if (rc != PML_OK) return rc;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(weights, 4) || !aligned(q_out, 16) ||
        !aligned(w_out, 4) || !aligned(kv_fused, 16) || !aligned(requests, 4) ||
        !aligned(block_table, 4) || q_token_stride % 8 || q_head_stride % 8 || k_token_stride % 8)
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    IndexQuantArgs a = {};
    a.rot = rotary(positions, positions_64, inv_freq, freq_64, rot_dim, rot_offset, interleaved,
                   mscale, 0);
    a.slot.requests = requests;
    a.slot.block_table = block_table;
    a.slot.bt_stride = bt_stride;
    a.slot.bt_width = bt_width;
    a.slot.num_pages = num_blocks;
    a.slot.num_requests = num_requests;
    a.slot.status = dev.status;
    a.q = q;
    a.k = k;
    a.weights = weights;
    a.q_out = q_out;
    a.w_out = w_out;
    a.kv_fused = kv_fused;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.k_token = k_token_stride;
    a.weight_scale = weight_scale;
    a.tokens = tokens;
    a.heads = num_heads;
    const long long rows = num_heads + (k != nullptr ? 1 : 0);
    a.rows_per_cta = cta_rows(kQuantRows, kQuantThreads / kQuantLanes, rows, kQuantMaxTokens, tokens, dev.sm_count);
    if (tokens * rows / a.rows_per_cta >= 0x7fffffffLL) return PML_ERR_UNSUPPORTED;    // CTAs
    e = launch_index_quant(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_pages_fork(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                   int bt_width, int32_t* seq_lens, int rows, const int32_t* parents,
                   const int32_t* children, int n, int32_t* copy_src, int32_t* copy_dst,
                   int32_t* copy_count, void* stream)
{
    const int rc = check_pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows);
    if (rc != PML_OK) return rc;
    if (n < 0 || !copy_count || (n > 0 && (!parents || !children || !copy_src || !copy_dst)))
        return PML_ERR_INVALID_ARG;
    if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(copy_src, 4) ||
        !aligned(copy_dst, 4) || !aligned(copy_count, 4))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    ForkArgs a = {pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows, dev.status),
                  parents, children, copy_src, copy_dst, copy_count, n};
    e = launch_pages_fork(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_pages_extend(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                     int bt_width, int32_t* seq_lens, int rows, const int32_t* new_lens,
                     int32_t* new_pages, int capacity, int32_t* new_count, void* stream)
{
    const int rc = check_pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows);
    if (rc != PML_OK) return rc;
    if (capacity < 0 || !new_count || (rows > 0 && !new_lens) || (capacity > 0 && !new_pages))
        return PML_ERR_INVALID_ARG;
    if (!aligned(new_lens, 4) || !aligned(new_pages, 4) || !aligned(new_count, 4)) return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    ExtendArgs a = {pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows, dev.status),
                    new_lens, new_pages, new_count, capacity};
    e = launch_pages_extend(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_pages_free(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                   int bt_width, int32_t* seq_lens, int rows, const int32_t* list, int n, void* stream)
{
    const int rc = check_pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows);
    if (rc != PML_OK) return rc;
    if (n < 0 || (n > 0 && !list)) return PML_ERR_INVALID_ARG;
    if (!aligned(list, 4)) return PML_ERR_ALIGNMENT;
    if (n == 0) return PML_OK;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    FreeArgs a = {pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows, dev.status),
                  list, n};
    e = launch_pages_free(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_pages_compact(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                      int bt_width, const int32_t* seq_lens, int rows, int32_t* ref_counts_out,
                      int32_t* block_table_out, int64_t bt_out_stride, int32_t* remap,
                      int32_t* copy_src, int32_t* copy_dst, int capacity, int32_t* copy_count,
                      void* stream)
{
    const int rc = check_pool(ref_counts, num_pages, block_table, bt_stride, bt_width, seq_lens, rows);
    if (rc != PML_OK) return rc;
    if (!copy_count || capacity < num_pages / 2 || (capacity > 0 && (!copy_src || !copy_dst)))
        return PML_ERR_INVALID_ARG;
    if ((num_pages > 0 && (!ref_counts_out || !remap)) || (rows > 0 && !block_table_out))
        return PML_ERR_INVALID_ARG;
    if (bt_out_stride < bt_width || (block_table_out == block_table && bt_out_stride != bt_stride))
        return PML_ERR_INVALID_ARG;
    if (!aligned(ref_counts_out, 4) || !aligned(block_table_out, 4) || !aligned(remap, 4) ||
        !aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(copy_count, 4))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    CompactArgs a = {pool(ref_counts, num_pages, block_table, bt_stride, bt_width,
                          const_cast<int32_t*>(seq_lens), rows, dev.status),
                     ref_counts_out, block_table_out, bt_out_stride, remap, copy_src, copy_dst,
                     copy_count, capacity};
    e = launch_pages_compact(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_pages_copy(void* cache, int layers, int64_t layer_stride_bytes, int num_pages,
                   int64_t page_stride_bytes, int64_t page_bytes, const int32_t* copy_src,
                   const int32_t* copy_dst, const int32_t* copy_count, int capacity, void* stream)
{
    if (layers < 0 || num_pages < 0 || capacity < 0 || page_bytes < 0) return PML_ERR_INVALID_ARG;
    if (num_pages > 1 && page_stride_bytes < page_bytes) return PML_ERR_INVALID_ARG;
    if (layers == 0 || capacity == 0 || page_bytes == 0 || num_pages == 0) return PML_OK;
    if (!cache || !copy_src || !copy_dst || !copy_count) return PML_ERR_INVALID_ARG;
    if (!aligned(copy_src, 4) || !aligned(copy_dst, 4) || !aligned(copy_count, 4))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    CopyPagesArgs a = {static_cast<uint8_t*>(cache), copy_src, copy_dst, copy_count, dev.status,
                       layer_stride_bytes, page_stride_bytes, page_bytes, layers, capacity, num_pages, 1};
    for (int v : {16, 4}) {
        if (aligned(cache, v) && layer_stride_bytes % v == 0 && page_stride_bytes % v == 0 &&
            page_bytes % v == 0) {
            a.vec = v;
            break;
        }
    }
    e = launch_pages_copy(a, dev.sm_count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int64_t pml_attention_workspace_bytes(int num_ctas, int head_dim)
{
    if (num_ctas < 1 || (head_dim != 64 && head_dim != 128)) return 0;
    const int64_t slots = 2LL * num_ctas;
    return slots * kPieceInts * 4 + slots * kAttnSlotRows * 8 + slots * kAttnSlotRows * head_dim * 4LL;
}

int pml_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                        const void* k_cache, int64_t k_page_stride, int64_t k_slot_stride,
                        int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                        int64_t v_slot_stride, int64_t v_head_stride, int dtype, int64_t num_pages,
                        const int32_t* block_table, int64_t bt_stride, int bt_width,
                        const int32_t* kv_lens, const int32_t* cu_q, int batch, int tokens,
                        int num_heads, int kv_heads, int head_dim, float softmax_scale, int causal,
                        int window, void* out, int64_t out_token_stride, int64_t out_head_stride,
                        float* lse, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (batch < 0) return PML_ERR_INVALID_ARG;
    if (batch > kAttnMaxBatch) return PML_ERR_UNSUPPORTED;
    if (tokens > 0 && batch == 0) return PML_ERR_INVALID_ARG;
    if (cu_q == nullptr && batch > 0 && tokens % batch != 0) return PML_ERR_INVALID_ARG;
    if (window < 0) return PML_ERR_INVALID_ARG;
    AttnArgs a = {};
    a.cu_q = cu_q;
    a.q_per_request = batch > 0 ? tokens / batch : 0;
    a.batch = batch;
    a.causal = causal ? 1 : 0;
    a.window = window;
    return attention_call(a, q, q_token_stride, q_head_stride, k_cache, k_page_stride, k_slot_stride,
                          k_head_stride, v_cache, v_page_stride, v_slot_stride, v_head_stride, dtype,
                          num_pages, block_table, bt_stride, bt_width, kv_lens, tokens, num_heads,
                          kv_heads, head_dim, softmax_scale, out, out_token_stride, out_head_stride,
                          lse, workspace, workspace_bytes, stream);
}

int pml_sparse_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                         const void* k_cache, int64_t k_page_stride, int64_t k_slot_stride,
                         int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                         int64_t v_slot_stride, int64_t v_head_stride, int dtype, int64_t num_pages,
                         const int32_t* block_table, int64_t bt_stride, int bt_width,
                         const int32_t* kv_lens, const int32_t* requests, int num_requests,
                         const int32_t* selected, int64_t selected_stride, int k, int tokens,
                         int num_heads, int kv_heads, int head_dim, float softmax_scale, void* out,
                         int64_t out_token_stride, int64_t out_head_stride, float* lse,
                         void* workspace, int64_t workspace_bytes, void* stream)
{
    if (k < 1 || selected_stride < k || num_requests < (tokens > 0 ? 1 : 0)) return PML_ERR_INVALID_ARG;
    if (k > kMaxListed) return PML_ERR_UNSUPPORTED;
    if (tokens > 0 && (!requests || !selected)) return PML_ERR_INVALID_ARG;
    if (!aligned(requests, 4) || !aligned(selected, 4)) return PML_ERR_ALIGNMENT;
    AttnArgs a = {};
    a.batch = num_requests;
    a.requests = requests;
    a.selected = selected;
    a.sel_stride = selected_stride;
    a.sel_k = k;
    return attention_call(a, q, q_token_stride, q_head_stride, k_cache, k_page_stride, k_slot_stride,
                          k_head_stride, v_cache, v_page_stride, v_slot_stride, v_head_stride, dtype,
                          num_pages, block_table, bt_stride, bt_width, kv_lens, tokens, num_heads,
                          kv_heads, head_dim, softmax_scale, out, out_token_stride, out_head_stride,
                          lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
