// C ABI of the operators over K/V caches held in 4 bits (declared in
// include/pml.h): argument checks and launches.  No allocation, no
// synchronisation.
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "host.h"
#include "nvfp4_cache.h"
#include "pml.h"

namespace {

using namespace pml;

constexpr int kMaxListed = 0x7fffff00; // entries of a list, so that their tiles' ends fit an int
constexpr int kMaxHeads = 8192;
constexpr int kMaxScaleExponent = 32;

// Strides of a dimension of one element are never used: any valid one will do.
int64_t used(int64_t stride, int64_t size, int64_t other) { return size > 1 ? stride : other; }

bool half_type(int dtype) { return dtype == PML_DTYPE_BFLOAT16 || dtype == PML_DTYPE_FLOAT16; }

// 2^e, |e| at most kMaxScaleExponent
bool scale_fits(float s)
{
    int e;
    return s > 0.0f && isfinite(s) && frexpf(s, &e) == 0.5f && e - 1 >= -kMaxScaleExponent && e - 1 <= kMaxScaleExponent;
}

int take_cache(const pml_nvfp4_cache* c, int64_t num_pages, int heads, int dim, NvCache& out)
{
    if (!c || !c->codes || !c->scales || !scale_fits(c->scale)) return PML_ERR_INVALID_ARG;
    const int64_t codes = dim / 2, scales = dim / kNvGroup;
    out.codes = c->codes;
    out.scales = c->scales;
    out.scale = c->scale;
    out.page = used(c->page_stride, num_pages, codes);
    out.slot = c->slot_stride;
    out.head = used(c->head_stride, heads, codes);
    out.s_page = used(c->scale_page_stride, num_pages, scales);
    out.s_slot = c->scale_slot_stride;
    out.s_head = used(c->scale_head_stride, heads, scales);
    if (!aligned(c->codes, 16) || !aligned(c->scales, scales)) return PML_ERR_ALIGNMENT;
    for (int64_t s : {out.page, out.slot, out.head})
        if (s <= 0 || s % 16) return PML_ERR_ALIGNMENT;
    for (int64_t s : {out.s_page, out.s_slot, out.s_head})
        if (s <= 0 || s % scales) return PML_ERR_ALIGNMENT;
    return PML_OK;
}

// The checks that both attention calls share; `a` comes with what is theirs.
int attention_call(NvAttnArgs& a, const void* q, int64_t q_token, int64_t q_head, int dtype,
                   const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache, int64_t num_pages,
                   const int32_t* block_table, int64_t bt_stride, int bt_width,
                   const int32_t* kv_lens, int tokens, int num_heads, int kv_heads, int head_dim,
                   float softmax_scale, void* out, int64_t out_token, int64_t out_head, float* lse,
                   void* workspace, int64_t workspace_bytes, void* stream)
{
    if (tokens < 0 || num_heads < 1 || kv_heads < 1 || num_heads % kv_heads) return PML_ERR_INVALID_ARG;
    if (!half_type(dtype)) return PML_ERR_UNSUPPORTED;
    if ((head_dim != 64 && head_dim != 128) || num_heads > kMaxHeads) return PML_ERR_UNSUPPORTED;
    if (!(softmax_scale > 0.0f) || softmax_scale > 1e30f) return PML_ERR_INVALID_ARG;
    if (tokens == 0) return PML_OK;
    if (!q || !block_table || !kv_lens || !out || !workspace) return PML_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > 0x7fffffffLL || bt_width < 1 || bt_stride < bt_width)
        return PML_ERR_INVALID_ARG;
    if (bt_width > 0x7fffffff / kBlockKeys) return PML_ERR_UNSUPPORTED;
    int rc = take_cache(k_cache, num_pages, kv_heads, head_dim, a.kc);
    if (rc == PML_OK) rc = take_cache(v_cache, num_pages, kv_heads, head_dim, a.vc);
    if (rc != PML_OK) return rc;
    // (c as a normal number, and its quotients too)
    const float scale = softmax_scale * a.kc.scale;
    if (!(scale >= 1e-30f && scale <= 1e30f)) return PML_ERR_INVALID_ARG;
    const int64_t qs[2] = {used(q_head, num_heads, head_dim), used(q_token, tokens, head_dim)};
    if (qs[0] <= 0 || qs[0] % 8 || qs[1] <= 0 || qs[1] % 8) return PML_ERR_ALIGNMENT;
    if ((tokens > 1 && out_token % 8) || (num_heads > 1 && out_head % 8)) return PML_ERR_ALIGNMENT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) ||
        !aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(a.cu_q, 4))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (workspace_bytes < pml_attention_workspace_bytes(dev.sm_count, head_dim)) return PML_ERR_INVALID_ARG;
    const int group = num_heads / kv_heads;
    const bool fp16 = dtype == PML_DTYPE_FLOAT16;
    const bool by_tiles = a.selected ? nvfp4_lists_by_tiles(tokens, num_heads, group, a.sel_k, dev.sm_count)
                                     : nvfp4_by_tiles(tokens, a.batch, num_heads, group);
    if (by_tiles) {
        AttnArgs w = {};
        attention_workspace(w, workspace, dev.sm_count, head_dim);
        w.kc4 = a.kc;
        w.vc4 = a.vc;
        w.out_scale = a.vc.scale;
        w.block_table = block_table;
        w.bt_stride = bt_stride;
        w.bt_width = bt_width;
        w.kv_lens = kv_lens;
        w.cu_q = a.cu_q;
        w.requests = a.requests;
        w.selected = a.selected;
        w.sel_stride = a.sel_stride;
        w.sel_k = a.sel_k;
        w.out = out;
        w.out_token = out_token;
        w.out_head = out_head;
        w.lse = lse;
        w.status = dev.status;
        w.num_pages = num_pages;
        w.batch = a.batch;
        w.tokens = tokens;
        w.q_per_request = a.q_per_request;
        w.kv_heads = kv_heads;
        w.group = group;
        w.half_tokens = kAttnHalfRows / group;
        w.causal = a.causal;
        w.window = a.window;
        w.scale = scale;
        w.scale_log2 = scale * 1.4426950408889634f;
        CUtensorMap qmap, kmap, vmap;
        const uint64_t dims[3] = {(uint64_t)head_dim, (uint64_t)num_heads, (uint64_t)tokens};
        const uint64_t strides[2] = {(uint64_t)qs[0] * 2, (uint64_t)qs[1] * 2};
        const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)w.half_tokens};
        e = encode_tiled(qmap, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims,
                         strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return cuda_fail(e);
        kmap = vmap = qmap;
        for (int i = 0; i < 2 && !a.selected; ++i) {      // the codes of a page's head
            const NvCache& c = i ? a.vc : a.kc;
            const uint64_t bytes = head_dim / 2;
            const uint64_t cdims[4] = {bytes, (uint64_t)kBlockKeys, (uint64_t)kv_heads, (uint64_t)num_pages};
            const uint64_t cstrides[3] = {(uint64_t)c.slot, (uint64_t)c.head, (uint64_t)c.page};
            const uint32_t cbox[4] = {(uint32_t)bytes, (uint32_t)kBlockKeys, 1, 1};
            e = encode_tiled(i ? vmap : kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.codes, cdims, cstrides, cbox,
                             head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
            if (e != cudaSuccess) return cuda_fail(e);
        }
        e = launch_paged_attention_nvfp4(head_dim, fp16, a.selected != nullptr, qmap, kmap, vmap, w, dev.sm_count,
                                         static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PML_OK : cuda_fail(e);
    }
    a.q = q;
    a.q_token = q_token;
    a.q_head = q_head;
    a.out = out;
    a.out_token = out_token;
    a.out_head = out_head;
    a.lse = lse;
    a.block_table = block_table;
    a.bt_stride = bt_stride;
    a.bt_width = bt_width;
    a.kv_lens = kv_lens;
    a.status = dev.status;
    a.num_pages = num_pages;
    a.tokens = tokens;
    a.kv_heads = kv_heads;
    a.group = group;
    a.scale_log2 = scale * 1.4426950408889634f;
    e = launch_nvfp4_attention(head_dim, fp16, a, dev.sm_count, workspace, workspace_bytes,
                               static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

int pml_append_nvfp4(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                     int64_t v_token_stride, int64_t v_head_stride, int dtype, const void* positions,
                     int positions_64, const int32_t* requests, int num_requests,
                     const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache, int64_t num_pages,
                     const int32_t* block_table, int64_t bt_stride, int bt_width, int tokens,
                     int kv_heads, int head_dim, void* stream)
{
    if (tokens < 0 || kv_heads < 1) return PML_ERR_INVALID_ARG;
    if (!half_type(dtype) || (head_dim != 64 && head_dim != 128) || kv_heads > kMaxHeads) return PML_ERR_UNSUPPORTED;
    if (tokens == 0) return PML_OK;
    if (!k || !v || !positions || !requests || !block_table) return PML_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > 0x7fffffffLL || num_requests < 1 || bt_width < 1 || bt_stride < bt_width)
        return PML_ERR_INVALID_ARG;
    NvAppendArgs a = {};
    int rc = take_cache(k_cache, num_pages, kv_heads, head_dim, a.kc);
    if (rc == PML_OK) rc = take_cache(v_cache, num_pages, kv_heads, head_dim, a.vc);
    if (rc != PML_OK) return rc;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(positions, positions_64 ? 8 : 4) ||
        !aligned(requests, 4) || !aligned(block_table, 4) ||
        (tokens > 1 && (k_token_stride % 8 || v_token_stride % 8)) ||
        (kv_heads > 1 && (k_head_stride % 8 || v_head_stride % 8)))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    a.slot.requests = requests;
    a.slot.block_table = block_table;
    a.slot.bt_stride = bt_stride;
    a.slot.bt_width = bt_width;
    a.slot.num_pages = num_pages;
    a.slot.num_requests = num_requests;
    a.slot.status = dev.status;
    a.positions = positions;
    a.pos64 = positions_64 ? 1 : 0;
    a.k = k;
    a.v = v;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.fp16 = dtype == PML_DTYPE_FLOAT16;
    a.tokens = tokens;
    a.heads = kv_heads;
    a.dim = head_dim;
    e = launch_nvfp4_append(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_read_nvfp4(const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache, int64_t num_pages,
                   const int32_t* block_table, int64_t bt_stride, const int32_t* kv_lens, int batch,
                   int width, void* k_out, int64_t k_page_stride, int64_t k_slot_stride,
                   int64_t k_head_stride, void* v_out, int64_t v_page_stride, int64_t v_slot_stride,
                   int64_t v_head_stride, int dtype, int64_t out_pages, const int32_t* out_table,
                   int64_t ot_stride, int kv_heads, int head_dim, void* stream)
{
    if (batch < 0 || width < 0 || kv_heads < 1) return PML_ERR_INVALID_ARG;
    if (!half_type(dtype) || (head_dim != 64 && head_dim != 128) || kv_heads > kMaxHeads) return PML_ERR_UNSUPPORTED;
    if (batch == 0 || width == 0) return PML_OK;
    if (!block_table || !kv_lens || !out_table || !k_out || !v_out) return PML_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > 0x7fffffffLL || out_pages < 1 || out_pages > 0x7fffffffLL ||
        bt_stride < width || ot_stride < width)
        return PML_ERR_INVALID_ARG;
    NvReadArgs a = {};
    int rc = take_cache(k_cache, num_pages, kv_heads, head_dim, a.kc);
    if (rc == PML_OK) rc = take_cache(v_cache, num_pages, kv_heads, head_dim, a.vc);
    if (rc != PML_OK) return rc;
    a.k_page = used(k_page_stride, out_pages, head_dim);
    a.k_slot = k_slot_stride;
    a.k_head = used(k_head_stride, kv_heads, head_dim);
    a.v_page = used(v_page_stride, out_pages, head_dim);
    a.v_slot = v_slot_stride;
    a.v_head = used(v_head_stride, kv_heads, head_dim);
    for (int64_t s : {a.k_page, a.k_slot, a.k_head, a.v_page, a.v_slot, a.v_head})
        if (s <= 0 || s % 8) return PML_ERR_ALIGNMENT;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(block_table, 4) || !aligned(out_table, 4) ||
        !aligned(kv_lens, 4))
        return PML_ERR_ALIGNMENT;
    DeviceInfo dev;
    cudaError_t e = device_info(dev);
    if (e != cudaSuccess) return cuda_fail(e);
    a.block_table = block_table;
    a.out_table = out_table;
    a.kv_lens = kv_lens;
    a.status = dev.status;
    a.k_out = k_out;
    a.v_out = v_out;
    a.bt_stride = bt_stride;
    a.ot_stride = ot_stride;
    a.num_pages = num_pages;
    a.out_pages = out_pages;
    a.width = width;
    a.batch = batch;
    a.heads = kv_heads;
    a.dim = head_dim;
    a.fp16 = dtype == PML_DTYPE_FLOAT16;
    e = launch_nvfp4_read(a, dev.sm_count, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PML_OK : cuda_fail(e);
}

int pml_paged_attention_nvfp4(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
                              const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache,
                              int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                              int bt_width, const int32_t* kv_lens, const int32_t* cu_q, int batch,
                              int tokens, int num_heads, int kv_heads, int head_dim,
                              float softmax_scale, int causal, int window, void* out,
                              int64_t out_token_stride, int64_t out_head_stride, float* lse,
                              void* workspace, int64_t workspace_bytes, void* stream)
{
    if (batch < 0) return PML_ERR_INVALID_ARG;
    if (batch > kAttnMaxBatch) return PML_ERR_UNSUPPORTED;
    if (tokens > 0 && batch == 0) return PML_ERR_INVALID_ARG;
    if (cu_q == nullptr && batch > 0 && tokens % batch != 0) return PML_ERR_INVALID_ARG;
    if (window < 0) return PML_ERR_INVALID_ARG;
    NvAttnArgs a = {};
    a.cu_q = cu_q;
    a.q_per_request = batch > 0 ? tokens / batch : 0;
    a.batch = batch;
    a.causal = causal ? 1 : 0;
    a.window = window;
    return attention_call(a, q, q_token_stride, q_head_stride, dtype, k_cache, v_cache, num_pages, block_table,
                          bt_stride, bt_width, kv_lens, tokens, num_heads, kv_heads, head_dim, softmax_scale, out,
                          out_token_stride, out_head_stride, lse, workspace, workspace_bytes, stream);
}

int pml_sparse_attention_nvfp4(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
                               const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache,
                               int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                               int bt_width, const int32_t* kv_lens, const int32_t* requests,
                               int num_requests, const int32_t* selected, int64_t selected_stride,
                               int k, int tokens, int num_heads, int kv_heads, int head_dim,
                               float softmax_scale, void* out, int64_t out_token_stride,
                               int64_t out_head_stride, float* lse, void* workspace,
                               int64_t workspace_bytes, void* stream)
{
    if (k < 1 || selected_stride < k || num_requests < (tokens > 0 ? 1 : 0)) return PML_ERR_INVALID_ARG;
    if (k > kMaxListed) return PML_ERR_UNSUPPORTED;
    if (tokens > 0 && (!requests || !selected)) return PML_ERR_INVALID_ARG;
    if (!aligned(requests, 4) || !aligned(selected, 4)) return PML_ERR_ALIGNMENT;
    NvAttnArgs a = {};
    a.batch = num_requests;
    a.requests = requests;
    a.selected = selected;
    a.sel_stride = selected_stride;
    a.sel_k = k;
    return attention_call(a, q, q_token_stride, q_head_stride, dtype, k_cache, v_cache, num_pages, block_table,
                          bt_stride, bt_width, kv_lens, tokens, num_heads, kv_heads, head_dim, softmax_scale, out,
                          out_token_stride, out_head_stride, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
