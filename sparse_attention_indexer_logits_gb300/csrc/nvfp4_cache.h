// Host-side launch records of the operators over K/V caches held in 4 bits.
// Internal to the library: the public C ABI is include/pml.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "serving.h"

namespace pml {

struct NvAppendArgs {
    SlotArgs slot;
    const void* positions;         // int32 or int64, one per token
    const void* k;
    const void* v;
    long long k_token, k_head;     // elements
    long long v_token, v_head;
    NvCache kc, vc;
    int pos64;
    int fp16;                      // 1 fp16, 0 bf16
    int tokens;
    int heads;
    int dim;
};

constexpr int kNvAppendThreads = 256;
constexpr int kNvAppendTokens = 16;    // of a CTA

struct NvReadArgs {
    NvCache kc, vc;
    const int32_t* block_table;
    const int32_t* out_table;
    const int32_t* kv_lens;
    unsigned int* status;
    void* k_out;
    void* v_out;
    long long k_page, k_slot, k_head;   // elements, of the outputs
    long long v_page, v_slot, v_head;
    long long bt_stride, ot_stride;
    long long num_pages, out_pages;
    int width;                     // columns that both tables have
    int batch;
    int heads;
    int dim;
    int fp16;
};

struct NvAttnArgs {
    NvCache kc, vc;
    const void* q;
    void* out;
    float* lse;                    // [tokens][heads], may be null
    const int32_t* block_table;
    const int32_t* kv_lens;        // per request
    const int32_t* cu_q;           // batch + 1 token offsets; null: q_per_request each
    const int32_t* requests;       // selected: one per token
    const int32_t* selected;       // selected: [tokens][sel_stride] positions
    unsigned int* status;
    long long q_token, q_head;     // elements
    long long out_token, out_head;
    long long bt_stride;
    long long sel_stride;
    long long num_pages;
    int bt_width;
    int batch;                     // requests (rows of the block table)
    int tokens;
    int q_per_request;
    int kv_heads;
    int group;                     // query heads per kv head
    int tile_tokens;               // tokens of an item
    int head_blocks;               // items that share a kv head's query heads
    int block_heads;               // query heads of one
    int sel_k;                     // selected: entries per token
    int whole_items;               // selected: no item is split between CTAs
    int cluster;                   // > 1: each item is one cluster's of so many CTAs
    int causal;
    int window;                    // > 0: only keys past position - window
    float scale;                   // softmax scale times the keys' scale
    float scale_log2;              // the same times log2(e)
};

cudaError_t launch_nvfp4_append(const NvAppendArgs& a, cudaStream_t stream);
cudaError_t launch_nvfp4_read(const NvReadArgs& a, int sm_count, cudaStream_t stream);
// Lists of k positions for groups of more than eight heads: steps of all warps,
// and the warps.
long long nvfp4_list_steps(int k, int group, long long lists);
int nvfp4_list_warps(int num_ctas);

// Fills in the items' shape.  `workspace` holds pml_attention_workspace_bytes.
cudaError_t launch_nvfp4_attention(int head_dim, bool fp16, NvAttnArgs& a, int num_ctas, void* workspace,
                                   int64_t workspace_bytes, cudaStream_t stream);

}  // namespace pml
