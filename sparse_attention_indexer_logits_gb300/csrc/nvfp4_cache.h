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
    float scale_log2;              // softmax scale times the keys' scale, times log2(e)
};

cudaError_t launch_nvfp4_append(const NvAppendArgs& a, cudaStream_t stream);
cudaError_t launch_nvfp4_read(const NvReadArgs& a, int sm_count, cudaStream_t stream);
// Items of `rows` rows ((token, head) pairs of a kv head: whole tokens, or some of
// one's heads) for each kv head, the tokens shared out evenly over the requests.
inline long long nvfp4_items(long long tokens, long long batch, int group, int rows)
{
    const long long per = group > rows ? 1 : rows / group, blocks = (group + rows - 1) / rows;
    const long long full = tokens / batch, more = tokens % batch;      // (`more` requests have one more)
    return blocks * ((batch - more) * ((full + per - 1) / per) + more * ((full + per) / per));
}

// Whether warps alone take items of 16 rows, else of 8.  One of 16 takes 1.2 to 1.4
// times as long: 128 request-heads of 8500 keys, heads of 128, 54 and 44 us; 512 of
// them, 8 heads to each, 166-172 us for 65 to 128 tokens in items of 16, 121 for 64
// in items of 8.
inline bool nvfp4_large_items(long long tokens, long long batch, int group)
{
    return 4 * nvfp4_items(tokens, batch, group, 16) < 3 * nvfp4_items(tokens, batch, group, 8);
}

// Whether a call goes by tiles: where some request, the tokens shared out evenly,
// has more than 32 rows, and all of them together more than 19/8 items each.  By
// warps a call's time is that of its items of 16 rows, by tiles that of a tile for
// every 128 rows: the same 64 requests with 12 heads, one item a token, 169 us for
// 64 tokens, 230 for 90, 281 for 110, 317 for 128; by tiles 378-386 for any of them,
// which is 19/8 items a request.  (Up to 32 rows may be three items too, 5 tokens of
// 6 heads: 64 requests 485 us and 386, but one over 500 keys 11.5 and 15.2, over
// 2000 14.0 and 18.1.)  A call of fewer than 128 rows in all, of which a warp has no
// more than a step or two, is left to warps: one request-head of 40 or 64 rows 21 us
// that way and 31 by tiles, 4 of them 23 and 26, 16 of 40 rows 32 and 28.
inline bool nvfp4_by_tiles(long long tokens, long long batch, int num_heads, int group)
{
    return group <= kAttnHalfRows && tokens * num_heads >= 128 && (tokens + batch - 1) / batch * group > 32 &&
           8 * nvfp4_items(tokens, batch, group, 16) > 19 * batch;
}

// Lists for groups of more than eight heads, of which 12 warps a CTA take 32
// positions for 16 heads a step.  Up to 32 heads go that way, and others while a
// warp has no more than eight steps: 64 heads over 1, 64 tokens of 64 positions 9.2
// us by warps and 13.9 by tiles, of 500 17.7 and 20.3, of 1500 28.8 and 30.1, of
// 2048 37.3 and 34.6; 200 tokens of 2048 132 and 83.
inline bool nvfp4_lists_by_tiles(long long tokens, int num_heads, int group, int k, int num_ctas)
{
    const long long steps = tokens * (num_heads / group) * nvfp4_items(1, 1, group, 16) * ((k + 31LL) / 32);
    return group > 32 && group <= kAttnHalfRows && steps > 8LL * 12 * num_ctas;
}

// Fills in the items' shape.  `workspace` holds pml_attention_workspace_bytes.
cudaError_t launch_nvfp4_attention(int head_dim, bool fp16, NvAttnArgs& a, int num_ctas, void* workspace,
                                   int64_t workspace_bytes, cudaStream_t stream);

}  // namespace pml
