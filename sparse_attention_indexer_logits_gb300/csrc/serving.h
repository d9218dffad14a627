// Host-side launch records of the serving operators: rotary positions, the
// cache writers, page bookkeeping and attention over pages.  Internal to the
// library: the public C ABI is include/pml.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pml {

// Where a token's cache slot is: page table[request][position / 64], slot
// position % 64.
struct SlotArgs {
    const int32_t* requests;       // one per token; < 0: the token is padding
    const int32_t* block_table;
    long long bt_stride;
    long long bt_width;            // columns that may be read
    long long num_pages;
    int num_requests;
    unsigned int* status;
};

// The frequencies and positions of a rotation.
struct RotaryArgs {
    const void* positions;         // int32 or int64, one per token
    const void* inv_freq;          // fp32 or fp64, `half` values, radians per position
    int pos64;
    int freq64;
    int half;                      // rotated pairs per head
    int offset;                    // first rotated element of a head
    int interleaved;               // pairs (2i, 2i+1), else (i, half + i)
    float mscale;                  // multiplies cosine and sine
    float sign;                    // -1: the transposed rotation (the gradient)
};

// One of up to three row sets of a rope launch: `heads` rows per token.
struct RopeRows {
    const void* src;
    void* dst;
    long long src_token, src_head; // elements
    long long dst_token, dst_head; // elements; paged: slot and head strides
    long long dst_page;            // elements between pages (paged sets)
    int heads;
};

struct RopeArgs {
    RotaryArgs rot;
    SlotArgs slot;                 // used when paged
    RopeRows q, k, v;              // k and v only when paged
    int tokens;
    int dim;
    int paged;
    int skip_rest;                 // q is rotated in place: unrotated elements stay
    int elem;                      // bytes of an element: 2 or 4
    int fp16;                      // 2-byte elements: 1 fp16, 0 bf16
    int vec;                       // elements per access: a power of two up to 16 bytes
    int rows_per_cta;
    int row_lanes_log2;            // threads of a row: a power of two, at most 256
};

constexpr int kRopeThreads = 256;
constexpr int kRopeUnits = 4;      // rows of a thread
constexpr int kRopeMaxTokens = 8;  // of a CTA, in part

// The indexer's inputs: q rows [tokens][heads][128] and key rows [tokens][128].
struct IndexQuantArgs {
    RotaryArgs rot;
    SlotArgs slot;
    const void* q;                 // bf16
    const void* k;                 // bf16, may be null (no keys written)
    const float* weights;
    uint8_t* q_out;
    float* w_out;
    uint8_t* kv_fused;
    long long q_token, q_head;     // elements
    long long k_token;
    float weight_scale;
    int tokens;
    int heads;
    int rows_per_cta;              // of the tokens' heads + 1 rows each (no keys: heads)
};

constexpr int kQuantThreads = 256;
constexpr int kQuantLanes = 4;     // of a row
constexpr int kQuantRows = 2;      // rows of a lane
constexpr int kQuantMaxTokens = 8; // of a CTA, in part

// A pool of pages: ref_counts[page] requests hold the page (0: free), and the
// first ceil(seq_lens[row] / 64) entries of a row's block table are its pages.
struct PoolArgs {
    int32_t* ref_counts;
    int32_t* block_table;
    int32_t* seq_lens;
    unsigned int* status;
    long long bt_stride;
    int bt_width;
    int num_pages;
    int rows;
};

struct ForkArgs {
    PoolArgs pool;
    const int32_t* parents;
    const int32_t* children;
    int32_t* src;          // pages to copy, n entries each, -1 past the count
    int32_t* dst;
    int32_t* count;
    int n;
};

struct ExtendArgs {
    PoolArgs pool;
    const int32_t* new_lens;   // one per row
    int32_t* new_pages;        // the pages taken, in (row, page) order; -1 past the count
    int32_t* count;
    int capacity;
};

struct FreeArgs {
    PoolArgs pool;
    const int32_t* list;
    int n;
};

struct CompactArgs {
    PoolArgs pool;
    int32_t* ref_counts_out;   // may be pool.ref_counts
    int32_t* block_table_out;  // may be pool.block_table (then the same stride)
    long long bt_out_stride;
    int32_t* remap;            // num_pages: where each page went, -1 for a free one
    int32_t* src;              // `capacity` entries each, -1 past the count
    int32_t* dst;
    int32_t* count;
    int capacity;
};

struct CopyPagesArgs {
    uint8_t* cache;            // layer l, page p at l * layer_stride + p * page_stride
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;      // device; at most `capacity` pairs are copied
    unsigned int* status;
    long long layer_stride;    // bytes
    long long page_stride;
    long long page_bytes;
    int layers;
    int capacity;
    int num_pages;
    int vec;                   // bytes per access: 16, 4 or 1
};

// Attention of new tokens over pages.  Rows of a tile are (token, head of the
// kv head's group): row = token * group + head.
constexpr int kAttnTileKeys = 128;     // keys of a tile: two pages, or 128 list entries
constexpr int kAttnHalfRows = 128;     // rows of one MMA accumulator
constexpr int kAttnSlotRows = 2 * kAttnHalfRows;
constexpr int kAttnMaxBatch = 16384;

struct AttnArgs {
    const int32_t* block_table;
    const int32_t* kv_lens;        // per request
    const int32_t* cu_q;           // batch + 1 token offsets; null: q_per_request each
    const int32_t* requests;       // selected: one per token
    const int32_t* selected;       // selected: [tokens][sel_stride] positions
    void* out;
    float* lse;                    // [tokens][heads], may be null
    unsigned int* status;
    int* pieces;                   // workspace: [num_ctas][2][kPieceInts]
    float2* stats;                 // workspace: [num_ctas][2][kAttnSlotRows] (maximum, sum)
    float* partial;                // workspace: [num_ctas][2][head_dim / 4][kAttnSlotRows][4]
    const void* k_cache;           // selected: read row by row
    const void* v_cache;
    long long k_page, k_slot, k_head;   // elements
    long long v_page, v_slot, v_head;
    long long bt_stride;
    long long sel_stride;
    long long out_token, out_head; // elements
    long long num_pages;
    int bt_width;
    int batch;                     // requests (rows of the block table when selected)
    int tokens;
    int q_per_request;
    int kv_heads;
    int group;                     // query heads per kv head
    int half_tokens;               // tokens of a 128-row half: 128 / group
    int sel_k;                     // selected: entries per token
    int causal;
    int window;                    // > 0: only keys past position - window
    float scale_log2;              // softmax scale * log2(e)
    float scale;
};

constexpr int kPieceInts = 8;

cudaError_t launch_paged_attention(int head_dim, bool fp16, bool select, const CUtensorMap& qmap,
                                   const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   const AttnArgs& a, int num_ctas, cudaStream_t stream);

cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t stream);
cudaError_t launch_pages_extend(const ExtendArgs& a, cudaStream_t stream);
cudaError_t launch_pages_free(const FreeArgs& a, cudaStream_t stream);
cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream);
cudaError_t launch_pages_copy(const CopyPagesArgs& a, int sm_count, cudaStream_t stream);

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_index_quant(const IndexQuantArgs& a, cudaStream_t stream);

}  // namespace pml
