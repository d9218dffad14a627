/*
 * pml -- paged MQA logits for the sparse-attention indexer, on GB300 (sm_103a).
 *
 * C ABI of libpml.so.  All tensor arguments are DEVICE pointers owned by the
 * caller; the library never allocates, frees or synchronises, and enqueues all
 * work on `stream` (a cudaStream_t passed as void*; NULL is the legacy default
 * stream).  Every entry point is one or two kernel launches with no host
 * round-trip, so it can be captured in a CUDA graph.
 *
 * Return value: PML_OK (0) or one of the PML_ERR_* codes.  Only conditions the
 * host can see are reported synchronously (null or misaligned pointers, shapes
 * outside the supported set, a CUDA launch error); nothing is launched when a
 * check fails.  Problems only the device can see -- a block-table entry outside
 * the cache, a bounded wait that ran out -- set bits of a sticky per-device
 * status word (pml_device_status) and the offending access is skipped.
 *
 * Sources: FlashInfer documentation pages "flashinfer.attn_scores" (the
 * definition, the output contract, "Scheduling and Setup") and
 * "flashinfer.sdsa.indexer_scores" (the single-head case and its arguments).
 */
#ifndef PML_H
#define PML_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    PML_OK = 0,
    PML_ERR_INVALID_ARG = 1,  /* null pointer, negative size, inconsistent sizes */
    PML_ERR_UNSUPPORTED = 2,  /* next_n, num_heads or group size outside the supported set */
    PML_ERR_ALIGNMENT = 3,    /* a pointer or stride not aligned as stated below */
    PML_ERR_CUDA = 4          /* a CUDA call failed; see pml_last_cuda_error() */
};

/* Device status bits (see pml_device_status). */
#define PML_STATUS_WAIT_TIMEOUT 1u  /* an in-kernel wait exceeded its limit; that CTA stopped early */
#define PML_STATUS_BAD_BLOCK 2u     /* a block_table entry was outside [0, num_blocks) */
#define PML_STATUS_BAD_REQUEST 4u   /* a group's request was outside [0, num_requests) */
#define PML_STATUS_FP4_INEXACT 8u   /* MXFP4 scales so far apart that tiny products may have been dropped (see pml_fp4_paged_mqa_logits) */

/* Version of this ABI (major*100 + minor). */
int pml_version(void);

/* Static description of an error code. */
const char* pml_error_string(int code);

/* The cudaError_t of the last PML_ERR_CUDA returned on this host thread. */
int pml_last_cuda_error(void);

/* Default persistent grid size for `device`: its SM count (0 on error). */
int pml_default_num_ctas(int device);

/* Number of int32 elements of a schedule for `num_ctas` CTAs: (num_ctas+1)*2. */
int pml_schedule_meta_elems(int num_ctas);

/* Block-table width that covers `max_seq_len` keys: ceil(max_seq_len / 64).
 * ("flashinfer.attn_scores", "Scheduling and Setup": min_block_table_width.) */
int pml_min_block_table_width(int max_seq_len);

/* `max_seq_len` rounded up to whole 64-key blocks.  (Same section:
 * padded_seq_len.) */
int pml_padded_seq_len(int max_seq_len);

/*
 * pml_schedule -- the persistent CTA work assignment
 * ("flashinfer.attn_scores", "Scheduling and Setup").
 *
 * Request b owns ceil(seq_lens[b]/64) blocks of 64 keys (none if
 * seq_lens[b] <= 0).  All blocks, in request order, are cut into num_ctas
 * contiguous ranges whose sizes differ by at most one, the first
 * (total mod num_ctas) one block longer.  schedule_meta (device, int32
 * [num_ctas+1][2], written) receives for each range the (request,
 * block-within-request) where it starts; a start at the end and the closing
 * entry are (batch, 0).
 *
 * The schedule depends on seq_lens and num_ctas only (next_n is accepted for
 * the pages' signature and must be 1..4).  A schedule is valid only while the
 * contents of seq_lens are unchanged: recompute it whenever they change,
 * including on every graph replay in which they change.
 */
int pml_schedule(const int32_t* seq_lens, int batch, int next_n, int num_ctas,
                 int32_t* schedule_meta, void* stream);

/*
 * pml_fp8_paged_mqa_logits ("flashinfer.attn_scores": math block, the two
 * bullets under it, the note on the output contract).
 *
 *   out[b*next_n + t, p] = s_p * sum_h weights[b*next_n + t, h]
 *                                     * relu( q[b*next_n + t, h, :] . k_p )
 *
 * for every request b with seq_lens[b] > 0, slot t < next_n and position
 * p < min(seq_lens[b], max_context); the rectifier acts per head, before the
 * weighted sum, and weights may be negative.  Key p of request b is row p%64
 * of physical block block_table[b*bt_stride + p/64]; s_p is that row's scale.
 * Row b*next_n+t is meaningful only for p <= seq_lens[b] - next_n + t; later
 * positions below seq_lens[b] are written but carry no meaning (callers mask).
 * Nothing else in `out` is written: not positions >= seq_lens[b], and not the
 * rows of requests with seq_lens[b] == 0 (pre-fill `out` to read them).
 *
 * q            e4m3 [batch*next_n, num_heads, 128], contiguous, 16-byte aligned
 * kv_fused     [num_blocks][8448] bytes, 16-byte aligned: per block 64 keys x
 *              128 e4m3 (row-major, 8192 B), then 64 little-endian fp32
 *              per-token scales (256 B)
 * weights      fp32 [batch*next_n, num_heads], contiguous, 16-byte aligned
 * seq_lens     int32 [batch]; contents are trusted (not checked)
 * block_table  int32 [batch, bt_stride]; entries below ceil(min(seq_lens[b],
 *              max_context)/64) must be in [0, num_blocks) (others are never
 *              read); an entry outside is replaced by 0 and flagged
 *              PML_STATUS_BAD_BLOCK
 * schedule_meta  NULL (each CTA computes its range on the GPU) or the output
 *              of pml_schedule for the same seq_lens and num_ctas
 * num_ctas     persistent grid size; 0 = pml_default_num_ctas (only allowed
 *              with schedule_meta == NULL)
 * out          fp32 [batch*next_n, out_stride], 4-byte aligned;
 *              out_stride >= max_context
 * max_context  >= 1, and ceil(max_context/64) <= bt_stride
 * next_n       1..4;  num_heads  8, 16, 32 or 64 (head dim fixed at 128)
 */
int pml_fp8_paged_mqa_logits(const uint8_t* q, const uint8_t* kv_fused, int64_t num_blocks,
                             const float* weights, const int32_t* seq_lens,
                             const int32_t* block_table, int64_t bt_stride,
                             const int32_t* schedule_meta, int num_ctas, float* out,
                             int64_t out_stride, int max_context, int batch, int next_n,
                             int num_heads, void* stream);

/* Output element types of pml_fp8_paged_mqa_logits_ex. */
#define PML_DTYPE_FLOAT32 0
#define PML_DTYPE_BFLOAT16 1

/*
 * pml_fp8_paged_mqa_logits_ex -- pml_fp8_paged_mqa_logits with the pages'
 * output_dtype option ("flashinfer.attn_scores": the paragraph comparing the
 * two variants -- the fp8 call exposes acc_dtype and output_dtype, output
 * float32 by default).
 *
 * output_dtype  PML_DTYPE_FLOAT32: `out` is fp32, exactly as
 *               pml_fp8_paged_mqa_logits (which is this call with that value);
 *               PML_DTYPE_BFLOAT16: `out` is bf16 [batch*next_n, out_stride]
 *               (2-byte aligned), each logit the fp32 result rounded to
 *               nearest even.  The accumulator is fp32 in both cases (the
 *               tensor cores' f32 accumulation; no other acc_dtype is
 *               offered).  Other values return PML_ERR_UNSUPPORTED.
 * All other arguments, the written region and the errors are those of
 * pml_fp8_paged_mqa_logits; out_stride counts elements of the output type.
 */
int pml_fp8_paged_mqa_logits_ex(const uint8_t* q, const uint8_t* kv_fused, int64_t num_blocks,
                                const float* weights, const int32_t* seq_lens,
                                const int32_t* block_table, int64_t bt_stride,
                                const int32_t* schedule_meta, int num_ctas, void* out,
                                int64_t out_stride, int output_dtype, int max_context, int batch,
                                int next_n, int num_heads, void* stream);

/*
 * pml_indexer_scores_bf16 ("flashinfer.sdsa.indexer_scores": body and the
 * query, key_cache, block_table, context_lengths, requests and scores
 * parameters).
 *
 *   scores[r, k] = query[r, :] . key_k      (one head: no weight, no ReLU)
 *
 * Query rows come in `groups` uniform groups of G = rows/groups consecutive
 * rows (1 <= G <= 8); group g owns rows [g*G, (g+1)*G), has
 * context_lengths[g] keys and reads the pages of block-table row
 * requests[g].  For k < min(context_lengths[g], max_context) the score is
 * written; later entries are not written, and a group of length <= 0 reads
 * nothing (its requests entry may hold any value).
 *
 * query          bf16 [rows, 128], contiguous, 16-byte aligned
 * key_cache      page P starts at byte P*page_stride_bytes and holds 64 keys x
 *                128 bf16 (row-major); base 16-byte aligned;
 *                page_stride_bytes a multiple of 16 and >= 16384
 * block_table    int32 [num_requests, bt_stride]; read entries must be in
 *                [0, num_pages) (else replaced by 0, PML_STATUS_BAD_BLOCK)
 * requests       int32 [groups]; read entries must be in [0, num_requests)
 *                (else replaced by 0, PML_STATUS_BAD_REQUEST)
 * scores         fp32 [rows, scores_stride], scores_stride >= max_context
 * max_context    >= 1, and ceil(max_context/64) <= bt_stride
 */
int pml_indexer_scores_bf16(const uint16_t* query, int rows, const uint16_t* key_cache,
                            int64_t page_stride_bytes, int64_t num_pages,
                            const int32_t* block_table, int64_t bt_stride, int num_requests,
                            const int32_t* context_lengths, const int32_t* requests, int groups,
                            float* scores, int64_t scores_stride, int max_context, void* stream);

/*
 * pml_indexer_scores_nvfp4 ("flashinfer.sdsa.indexer_scores": the NVFP4 forms
 * of query, key_cache, query_scales and key_scales).
 *
 *   scores[r, k] = q_r . k_k       (dequantised values; one head, no weight,
 *                                   no rectifier)
 *
 * A row of 128 values is 64 bytes of E2M1 codes, two to a byte (element d in
 * byte d/2; the low nibble holds the even element), and 8 E4M3 scale codes,
 * scale j applying to elements 16j .. 16j+15: value = E2M1(code) * E4M3(scale).
 * Every E4M3 code is accepted (negative scales negate their block; 0x7F and
 * 0xFF are NaN and make every score of their row or key NaN).  Groups,
 * lengths, requests, the written region and the status bits are those of
 * pml_indexer_scores_bf16.  Every product of two values is exact in fp32
 * (the block-scaled tensor cores take codes and scales as stored); only the
 * sums round.
 *
 * query           uint8 [rows, 64], 16-byte aligned
 * query_scales    uint8 [rows, 8] (E4M3), 8-byte aligned
 * key_cache       page P's 64 keys x 64 bytes start at byte P*page_stride_bytes;
 *                 base 16-byte aligned, page_stride_bytes a multiple of 16 and
 *                 >= 4096
 * key_scales      page P's 64 keys x 8 scale bytes start at byte
 *                 P*scale_page_stride_bytes; base 8-byte aligned,
 *                 scale_page_stride_bytes a multiple of 8 and >= 512 (the two
 *                 may be views of one cache holding each page's keys and then
 *                 its scales)
 * num_pages       pages in both (block_table entries must be below it)
 * scores          fp32 [rows, scores_stride], scores_stride >= max_context
 */
int pml_indexer_scores_nvfp4(const uint8_t* query, const uint8_t* query_scales, int rows,
                             const uint8_t* key_cache, int64_t page_stride_bytes,
                             const uint8_t* key_scales, int64_t scale_page_stride_bytes,
                             int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                             int num_requests, const int32_t* context_lengths,
                             const int32_t* requests, int groups, float* scores,
                             int64_t scores_stride, int max_context, void* stream);

/*
 * pml_fp8_paged_mqa_logits_wait_test -- test support; the pages have no
 * counterpart.  The fp32 fp8 logits call with the in-kernel schedule, in which
 * every CTA's producer leaves its stage number drop_stage (counted from 0
 * within the CTA) unpublished, and every wait inside the kernel gives up after
 * wait_limit_us microseconds instead of one second.  The roles waiting on the
 * missing stage run out of time: the CTA records PML_STATUS_WAIT_TIMEOUT,
 * raises its abort flag so that its other roles stop waiting, lets the copies
 * and MMAs it issued complete, frees its tensor memory and returns.  Logits of
 * the CTAs that stopped are incomplete.  It exists so that the tests can run
 * the kernel's timeout path on the GPU without a fault or a hang: the call
 * returns, the status word says what happened, and the device stays usable
 * for the next call.
 *
 * Arguments as pml_fp8_paged_mqa_logits (fp32 out, no schedule_meta, default
 * CTA count).  Returns PML_ERR_INVALID_ARG for drop_stage < 0 or
 * wait_limit_us outside 1 .. 1000000, else as pml_fp8_paged_mqa_logits.
 */
int pml_fp8_paged_mqa_logits_wait_test(const uint8_t* q, const uint8_t* kv_fused,
                                       int64_t num_blocks, const float* weights,
                                       const int32_t* seq_lens, const int32_t* block_table,
                                       int64_t bt_stride, float* out, int64_t out_stride,
                                       int max_context, int batch, int next_n, int num_heads,
                                       int drop_stage, int64_t wait_limit_us, void* stream);

/*
 * pml_fp4_paged_mqa_logits -- the MXFP4 variant ("flashinfer.attn_scores":
 * the math block, its two bullets and the paragraph after them: MXFP4 block
 * scales folded into the dequantised values, one per 32-element group on
 * both operands; two FP4 values per q byte; 64 heads of 128 only; no
 * per-position factor; default output bf16).
 *
 *   out[b*next_n + t, p] = sum_h w[t,h] * relu(q[t,h] . k_p)
 *
 * over values code * 2^(e - 127): code an E2M1 value (element d of a row in
 * byte d/2, low nibble for even d), e the row's E8M0 scale byte d/32.
 * Written region and schedule as pml_fp8_paged_mqa_logits.
 *
 * q          [batch*next_n, 64, 64] packed E2M1, 16-byte aligned
 * q_sf       [batch*next_n, 64, 4] E8M0, 16-byte aligned
 * kv_cache   [num_blocks][4352] bytes, 16-byte aligned: per block 64 keys x
 *            64 code bytes (4096 B), then 64 x 4 E8M0 scale bytes (256 B)
 * weights    fp32 [batch*next_n, 64], 16-byte aligned
 * out        output_dtype PML_DTYPE_BFLOAT16 (the pages' default) or
 *            PML_DTYPE_FLOAT32, [batch*next_n, out_stride], aligned to its
 *            element
 * batch      <= 65535; next_n 1..4; other arguments, the written region and
 *            the schedule as pml_fp8_paged_mqa_logits (next_n 3 and 4 run
 *            as two passes over the cache, slots 0-1 then the rest, each
 *            its own launch on `stream`)
 *
 * Method: every row (a key, or one head of one query slot) has a frame
 * 2^(E - 127), E its largest group exponent.  The block-scaled tensor cores
 * take the codes as stored and each group's scale relative to its row's
 * frame (2^(e - E), at most 1), so every product of a key group and a query
 * group is exact in fp32 and only the sums round; the key's and the query
 * rows' frames are applied afterwards, the rows' folded into the head weights
 * relative to the slot's largest one.  So each logit is its exact value up
 * to fp32 rounding of the sums -- a logit beyond the output type's range is
 * +-inf -- except where a key's and a query row's scale spreads together
 * exceed 124 binades, when products smaller than 2^-124 of the two rows'
 * frames may be rounded or dropped (a group more than 127 binades below its
 * row's frame is dropped), or a head's largest scale lies more than 100
 * binades below the slot's largest: both set PML_STATUS_FP4_INEXACT.  An
 * E8M0 NaN scale (0xFF) makes its group NaN, and a NaN dot product is
 * rectified to 0.
 */
int pml_fp4_paged_mqa_logits(const uint8_t* q, const uint8_t* q_sf, const uint8_t* kv_cache,
                             int64_t num_blocks, const float* weights, const int32_t* seq_lens,
                             const int32_t* block_table, int64_t bt_stride,
                             const int32_t* schedule_meta, int num_ctas, void* out,
                             int64_t out_stride, int output_dtype, int max_context, int batch,
                             int next_n, void* stream);

/*
 * pml_topk_logits -- the indexer's selection over the logits
 * ("flashinfer.attn_scores", intro: the logits are what a sparse-attention
 * indexer uses to choose which KV tokens to keep; note: row b*next_n+t is
 * meaningful for positions 0 .. seq_lens[b]-next_n+t).  The pages fix neither
 * k nor the order of equal values; this call's definition:
 *
 *   indices[r, 0..k) = the k positions p < min(seq_lens[b]-next_n+t+1,
 *   max_context) with the largest logits[r, p], r = b*next_n+t, in descending
 *   order of value -- the float32 bit order, -NaN < -inf < ... < -0 < +0 < ...
 *   < +inf < +NaN -- equal values in ascending position; slots past the
 *   number of candidates hold -1 (values: -inf).  Requests with
 *   seq_lens[b] <= 0 have no candidates.
 *
 * logits    fp32 [batch*next_n, logits_stride], logits_stride >= max_context
 *           (only candidate positions are read)
 * indices   int32 [batch*next_n, indices_stride], indices_stride >= k (written)
 * values    NULL, or fp32 [batch*next_n, values_stride] (written: the
 *           selected logits, bit for bit)
 * k         1 .. 4096 (else PML_ERR_UNSUPPORTED); next_n >= 1
 */
int pml_topk_logits(const float* logits, int64_t logits_stride, const int32_t* seq_lens, int batch,
                    int next_n, int max_context, int k, int32_t* indices, int64_t indices_stride,
                    float* values, int64_t values_stride, void* stream);

/*
 * pml_fp8_paged_mqa_logits_noalloc -- the two-step call (pml_schedule, then
 * pml_fp8_paged_mqa_logits with that schedule) for callers that cannot
 * allocate device memory.  The documentation pages have no counterpart: it
 * exists for this library's users.
 *
 * Who needs it: code that only receives the buffers it works on and has no
 * way to obtain more device memory -- a plugin inside a host runtime that owns
 * all allocations, a serving loop running under a memory pool that forbids
 * raw cudaMalloc (which also synchronises the device), or a C caller with no
 * allocator at hand.  The regular two-step path needs such a caller to find
 * room for the (num_ctas+1)*2 int32 schedule; here the schedule lives in a
 * fixed array inside the library's own device memory (8200 bytes, held on
 * every device that loads the library until the process exits).
 *
 * Arguments and results are those of pml_fp8_paged_mqa_logits without
 * schedule_meta.  num_ctas: 0 = pml_default_num_ctas (capped at the limit),
 * at most pml_noalloc_max_ctas() = 1024; larger values return
 * PML_ERR_INVALID_ARG and launch nothing.  Nothing is allocated or freed: no
 * cudaMalloc, no cudaFree, no allocating library routine.
 *
 * The first call on a device looks up the array's device address with that
 * device current (cudaGetSymbolAddress); make that first call before any
 * stream capture.  A failure there returns PML_ERR_CUDA.
 *
 * All calls share the one array, which keeps the last call's schedule; each
 * call rewrites every entry it reads, so nothing needs clearing.  Calls whose
 * work overlaps on the GPU (different streams, no ordering between them) race
 * on the array: order them, or use the regular entry points with separate
 * buffers.  If the logits launch is rejected after the schedule was written,
 * the only side effect is the rewritten array.
 */
int pml_fp8_paged_mqa_logits_noalloc(const uint8_t* q, const uint8_t* kv_fused,
                                     int64_t num_blocks, const float* weights,
                                     const int32_t* seq_lens, const int32_t* block_table,
                                     int64_t bt_stride, int num_ctas, float* out,
                                     int64_t out_stride, int max_context, int batch, int next_n,
                                     int num_heads, void* stream);

/* Largest num_ctas pml_fp8_paged_mqa_logits_noalloc accepts (1024). */
int pml_noalloc_max_ctas(void);

/* ------------------------------------------------------------------------
 * Serving operators: what feeds the logits above and what reads the positions
 * they select.  All of them work on pages of 64 tokens: token position p of a
 * request is slot p % 64 of page block_table[request * bt_stride + p / 64].
 * ------------------------------------------------------------------------ */

#define PML_DTYPE_FLOAT16 2   /* element type of the serving operators only */

#define PML_STATUS_NO_PAGES 16u  /* pml_pages_fork / _extend: the pool ran out of free pages */

/*
 * pml_rope -- rotary positions, and their gradient.
 *
 *   (a, b) -> mscale * (a cos t - b sin t, b cos t + a sin t),
 *   t = positions[token] * inv_freq[j]
 *
 * for the rot_dim / 2 pairs j of every head: elements rot_offset + j and
 * rot_offset + rot_dim/2 + j, or (interleaved != 0) rot_offset + 2j and
 * rot_offset + 2j + 1.  A head's other elements are copied.  gradient != 0
 * applies the transposed map (t negated): it takes the gradient of the
 * output to that of the input.  The angle is reduced exactly at any position
 * (64-bit fixed point); arithmetic is fp32, rounded once.
 *
 * x, out      dtype PML_DTYPE_FLOAT32, _BFLOAT16 or _FLOAT16; element (token,
 *             head, d) at token * token_stride + head * head_stride + d
 *             (strides in elements, any value; 16-byte aligned pointers and
 *             strides are fastest).  out may be x with the same strides;
 *             other overlaps are not allowed
 * positions   [tokens] int32, or int64 (positions_64 != 0); any sign
 * inv_freq    [rot_dim/2] fp32, or fp64 (freq_64 != 0), radians per position
 *             (long-context scalings are choices of inv_freq and mscale);
 *             infinities, NaN and subnormals count as 0
 * rot_dim     even, 0 .. head_dim - rot_offset;  head_dim  1 .. 512;  at most
 *             32768 heads
 */
int pml_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
             int64_t out_token_stride, int64_t out_head_stride, int dtype, const void* positions,
             int positions_64, const void* inv_freq, int freq_64, int rot_dim, int rot_offset,
             int interleaved, float mscale, int gradient, int tokens, int heads, int head_dim,
             void* stream);

/*
 * pml_rope_append -- a step's q, k and v on their way into attention: q
 * rotated into q_out, k rotated and v copied into the pages of their caches,
 * one launch.  The rotation is pml_rope's.
 *
 * q, q_out    [tokens, num_heads, head_dim] (num_heads may be 0); k, v
 *             [tokens, kv_heads, head_dim]: bf16 or fp16 with strides in
 *             elements as in pml_rope; q_out may be q
 * k_cache     element (page, slot, head, d) at page * k_page_stride + slot *
 *             k_slot_stride + head * k_cache_head_stride + d; v_cache alike
 * requests    int32 [tokens], the token's block-table row.  A negative
 *             request or position makes the token padding: nothing of it is
 *             written.  A request at or past num_requests sets
 *             PML_STATUS_BAD_REQUEST, a position at or past 64 * bt_width or
 *             a page outside [0, num_pages) PML_STATUS_BAD_BLOCK; that
 *             token's k and v are then not written
 * Two tokens of a call must not share a slot.
 */
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
                    int num_heads, int kv_heads, int head_dim, void* stream);

/*
 * pml_index_quant_append -- the inputs of pml_fp8_paged_mqa_logits from a
 * step's bf16 rows: r = rotated row, s = max(max |r|, 1e-12) / 448, codes
 * e4m3(r / s).  A q row's scale goes into its weight, w_out = weights * s *
 * weight_scale; a key's codes and scale go into its kv_fused block.
 *
 * q           bf16 [tokens, num_heads, 128], strides in elements, multiples of
 *             8, 16-byte aligned; k bf16 [tokens, 128] alike, or NULL (no
 *             keys are written; requests and kv_fused are not read)
 * weights     fp32 [tokens, num_heads], contiguous; w_out alike
 * q_out       e4m3 [tokens, num_heads, 128], contiguous, 16-byte aligned
 * kv_fused    [num_blocks][8448] as pml_fp8_paged_mqa_logits takes it
 * rot_dim a multiple of 16, rot_offset of 8; num_heads 1 .. 1024; padding
 * tokens and bad requests and pages as in pml_rope_append (without keys a
 * negative position alone makes the token padding).  A NaN in a row
 * makes its scale NaN, an infinity makes it infinite (the row's codes are
 * then 0 or NaN).
 */
int pml_index_quant_append(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                           const void* k, int64_t k_token_stride, const float* weights,
                           float weight_scale, const void* positions, int positions_64,
                           const int32_t* requests, int num_requests, const void* inv_freq,
                           int freq_64, int rot_dim, int rot_offset, int interleaved, float mscale,
                           uint8_t* q_out, float* w_out, uint8_t* kv_fused, int64_t num_blocks,
                           const int32_t* block_table, int64_t bt_stride, int bt_width, int tokens,
                           int num_heads, void* stream);

/*
 * pml_paged_attention -- attention of new tokens over a paged cache: one
 * token per request, chunks, or any mix.
 *
 *   out[t, h] = sum_p softmax_p(softmax_scale * q[t, h] . k_p) v_p,
 *   lse[t, h] = ln sum_p exp(softmax_scale * q[t, h] . k_p)
 *
 * Request b's new tokens are rows cu_q[b] .. cu_q[b+1]-1 of q (cu_q NULL:
 * tokens / batch rows each) and the last ones of its kv_lens[b] cached
 * tokens: row i of n stands at position kv_lens[b] - n + i.  It may see
 * positions p of its request up to its own (causal != 0; else all below
 * kv_lens[b]) and, for window > 0, past its own - window.  Query head h reads
 * kv head h / (num_heads / kv_heads).  A row that may see nothing (an empty
 * cache, a negative position) gives 0 and -inf.  Places a row may not see
 * never reach it, whatever they hold (infinities and NaN too), nor do slots
 * past kv_lens[b].
 *
 * Scores, softmax and sums are fp32; the probabilities are rounded to the
 * inputs' type for the second product (half a step each, averaged over the
 * keys: 2^-8 relative in bf16; 2^-11 in fp16, or 2^-32 of the row's largest
 * probability where that is more), the output once.
 *
 * q, out       bf16 or fp16 [tokens, num_heads, head_dim], strides in elements,
 *              multiples of 8 and (q) positive; 16-byte aligned pointers
 * k_cache      element (page, slot, head, d) at page * k_page_stride + slot *
 *              k_slot_stride + head * k_head_stride + d; strides positive
 *              multiples of 8, 16-byte aligned; v_cache alike
 * kv_lens      int32 [batch], contents trusted; positions at or past 64 *
 *              bt_width are not there
 * cu_q         int32 [batch+1], ascending from 0 to tokens, or NULL
 * head_dim     64 or 128;  num_heads a multiple of kv_heads, at most 128 times
 * softmax_scale  positive;  batch <= 16384
 * lse          fp32 [tokens, num_heads] or NULL
 * workspace    device, 16-byte aligned, pml_attention_workspace_bytes(SM count,
 *              head_dim) bytes or more; contents do not matter and nothing in
 *              it outlives the call, but calls that overlap need one each
 * A page outside [0, num_pages) is replaced by 0 (PML_STATUS_BAD_BLOCK).
 * Results do not depend on the order in which CTAs run.
 */
int pml_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                        const void* k_cache, int64_t k_page_stride, int64_t k_slot_stride,
                        int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                        int64_t v_slot_stride, int64_t v_head_stride, int dtype, int64_t num_pages,
                        const int32_t* block_table, int64_t bt_stride, int bt_width,
                        const int32_t* kv_lens, const int32_t* cu_q, int batch, int tokens,
                        int num_heads, int kv_heads, int head_dim, float softmax_scale, int causal,
                        int window, void* out, int64_t out_token_stride, int64_t out_head_stride,
                        float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * pml_sparse_attention -- the same over the positions that a list names, as
 * pml_topk_logits leaves them: token t looks at selected[t, 0..k) of request
 * requests[t].  Entries below 0 or at or past kv_lens[requests[t]] are not
 * there; the order does not matter; an entry that is there twice counts
 * twice.  No causal rule applies beyond the list.  A negative request makes
 * all of its token's entries absent (out 0, lse -inf), one at or past
 * num_requests does too and sets PML_STATUS_BAD_REQUEST.
 *
 * selected     int32 [tokens, selected_stride], k entries used (at most 2^31 -
 *              256)
 * The rest as in pml_paged_attention.
 */
int pml_sparse_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                         const void* k_cache, int64_t k_page_stride, int64_t k_slot_stride,
                         int64_t k_head_stride, const void* v_cache, int64_t v_page_stride,
                         int64_t v_slot_stride, int64_t v_head_stride, int dtype, int64_t num_pages,
                         const int32_t* block_table, int64_t bt_stride, int bt_width,
                         const int32_t* kv_lens, const int32_t* requests, int num_requests,
                         const int32_t* selected, int64_t selected_stride, int k, int tokens,
                         int num_heads, int kv_heads, int head_dim, float softmax_scale, void* out,
                         int64_t out_token_stride, int64_t out_head_stride, float* lse,
                         void* workspace, int64_t workspace_bytes, void* stream);

/*
 * K/V caches held in 4 bits: 9/32 of the memory and traffic of 16 bits.
 * A row (a token's head of head_dim values, 64 or 128) is head_dim / 2 bytes
 * of E2M1 codes, element d in byte d / 2, the low nibble the even one, and
 * head_dim / 16 E4M3 scales, each of sixteen values, as the rows of
 * pml_indexer_scores_nvfp4; all values of a cache are multiplied by one power
 * of two besides:
 *
 *   value = E2M1(code) * E4M3(scale) * cache.scale
 *
 * A NaN scale (0x7F, 0xFF) makes its sixteen values NaN; a negative one negates
 * them.
 *
 * codes    the row of (page, slot, head) at page * page_stride + slot *
 *          slot_stride + head * head_stride bytes; 16-byte aligned, strides
 *          positive multiples of 16
 * scales   alike with its own strides, all aligned to head_dim / 16 bytes
 * scale    2^-32 .. 2^32, a power of two (else PML_ERR_INVALID_ARG)
 */
typedef struct pml_nvfp4_cache {
    uint8_t* codes;
    uint8_t* scales;
    int64_t page_stride, slot_stride, head_stride;
    int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
    float scale;
} pml_nvfp4_cache;

/*
 * pml_append_nvfp4 -- a step's k and v rows quantised into their pages.  For
 * each sixteen values x of a row, g the cache's scale:
 *
 *   s = e4m3(max |x| / (6 g)), 448 at most, NaN if some x is not finite;
 *   code = the E2M1 value nearest to x / (s g), ties to the even code, 6 at
 *          most in magnitude, the sign that of x (0 of -0); 0 where s is 0 or
 *          NaN
 *
 * The codes are those of the exact quotient: equal rows give equal codes.  (k is
 * stored as it comes; pml_rope rotates it.)
 *
 * k, v        bf16 or fp16 [tokens, kv_heads, head_dim], strides in elements,
 *             multiples of 8, 16-byte aligned
 * positions, requests, block_table   as in pml_rope_append: padding tokens are
 *             not written, nor are those of a bad request or page (status)
 * Two tokens of a call must not share a slot.
 */
int pml_append_nvfp4(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                     int64_t v_token_stride, int64_t v_head_stride, int dtype, const void* positions,
                     int positions_64, const int32_t* requests, int num_requests,
                     const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache, int64_t num_pages,
                     const int32_t* block_table, int64_t bt_stride, int bt_width, int tokens,
                     int kv_heads, int head_dim, void* stream);

/*
 * pml_read_nvfp4 -- pages read back into 16-bit pages: slot p % 64 of page
 * out_table[b, p / 64] of k_out and v_out becomes the values of position p of
 * request b, p < kv_lens[b], rounded once to dtype (exact but where the type's
 * range ends).  Other slots stay as they were.  A prefill chunk reads its
 * contexts back once and attends to them with pml_paged_attention, whose
 * block_table is then out_table.
 *
 * k_out, v_out  bf16 or fp16, element (page, slot, head, d) at page *
 *               k_page_stride + slot * k_slot_stride + head * k_head_stride +
 *               d; strides positive multiples of 8, 16-byte aligned
 * width         columns of both tables; positions at or past 64 * width are
 *               not there
 * A page outside [0, num_pages) or [0, out_pages) is skipped
 * (PML_STATUS_BAD_BLOCK).  No two blocks of a call share a page of the outputs.
 */
int pml_read_nvfp4(const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache, int64_t num_pages,
                   const int32_t* block_table, int64_t bt_stride, const int32_t* kv_lens, int batch,
                   int width, void* k_out, int64_t k_page_stride, int64_t k_slot_stride,
                   int64_t k_head_stride, void* v_out, int64_t v_page_stride, int64_t v_slot_stride,
                   int64_t v_head_stride, int dtype, int64_t out_pages, const int32_t* out_table,
                   int64_t ot_stride, int kv_heads, int head_dim, void* stream);

/*
 * pml_paged_attention_nvfp4 -- pml_paged_attention over caches held in 4 bits:
 * single tokens and a few drafts per request, or any mix (long chunks are
 * faster through pml_read_nvfp4).  Arguments, masks, rows without keys, `lse`,
 * the workspace and the errors are as there, with these differences: the
 * products take q and the probabilities in fp16 (a bf16 row of q scaled by a
 * power of two, which keeps its 8 bits for elements down to 2^-17 of its
 * largest); kv_heads divides num_heads, whose number is at most 8192;
 * softmax_scale * k_cache->scale is in 1e-30 .. 1e30 (else
 * PML_ERR_INVALID_ARG); a row of q that is not finite, or whose scores fp32
 * does not hold, gives a row without meaning.
 * Which way a call goes, and with it its roundings, follows from its sizes.  A
 * request's rows of q to a kv head are its tokens (taken as tokens / batch each, one
 * more for tokens % batch of them) times num_heads / kv_heads; items are 16 of them:
 * whole tokens, or some of one's heads.  Calls of up to 32 rows to each request, or
 * of up to 19/8 items a request, or of fewer than 128 rows in all, and those of more
 * than 128 heads to a kv head are taken warp by warp, others in tiles of 128.
 */
int pml_paged_attention_nvfp4(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
                              const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache,
                              int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                              int bt_width, const int32_t* kv_lens, const int32_t* cu_q, int batch,
                              int tokens, int num_heads, int kv_heads, int head_dim,
                              float softmax_scale, int causal, int window, void* out,
                              int64_t out_token_stride, int64_t out_head_stride, float* lse,
                              void* workspace, int64_t workspace_bytes, void* stream);

/*
 * pml_sparse_attention_nvfp4 -- pml_sparse_attention over caches held in 4
 * bits, with the differences above.  Groups of 33 to 128 heads to a kv head go in
 * tiles once there is more to do than eight steps (32 positions for 16 heads) for
 * each of 12 warps an SM; all else goes warp by warp.
 */
int pml_sparse_attention_nvfp4(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
                               const pml_nvfp4_cache* k_cache, const pml_nvfp4_cache* v_cache,
                               int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                               int bt_width, const int32_t* kv_lens, const int32_t* requests,
                               int num_requests, const int32_t* selected, int64_t selected_stride,
                               int k, int tokens, int num_heads, int kv_heads, int head_dim,
                               float softmax_scale, void* out, int64_t out_token_stride,
                               int64_t out_head_stride, float* lse, void* workspace,
                               int64_t workspace_bytes, void* stream);

/* Bytes of workspace for any attention call; num_ctas is the device's SM
 * count (pml_default_num_ctas).  0 for a head_dim other than 64 and 128. */
int64_t pml_attention_workspace_bytes(int num_ctas, int head_dim);

/*
 * Page bookkeeping.  A pool is ref_counts [num_pages] (how many requests hold
 * each page; 0: free), block_table [rows, bt_stride] of which bt_width columns
 * are used, and seq_lens [rows]; a row's first ceil(seq_lens / 64) entries are
 * its pages.  Pages are taken lowest number first, so results depend on the
 * pool alone.  All arrays are device int32; rows * (bt_width + 1) < 2^31.
 *
 * pml_pages_fork: for i < n, row children[i] becomes a copy of row
 * parents[i]: full pages are shared (their count rises), a last page that is
 * part full is replaced by a free page, and (its page, the new page) is added
 * to copy_src / copy_dst (n entries each, in order of i, -1 past
 * *copy_count) for pml_pages_copy.  Forks are served in order; one that finds
 * no free page leaves the child with length 0 and sets PML_STATUS_NO_PAGES.
 * A row is not both a parent and a child of one call nor twice a child, and a
 * child holds no pages (free it first).  Rows outside [0, rows) or longer
 * than the table set PML_STATUS_BAD_REQUEST and are skipped.
 *
 * pml_pages_extend: grows every row to new_lens[row] tokens, taking pages in
 * (row, page) order; shorter lengths change nothing.  A row whose pages are
 * not all there keeps its length, as does every later row that needs one
 * (PML_STATUS_NO_PAGES); a length past the table's width is refused
 * (PML_STATUS_BAD_BLOCK).  new_pages [capacity] receives the pages taken, -1
 * past *new_count; at most `capacity` pages are taken.
 *
 * pml_pages_free: the rows in list (distinct) give back their pages and get
 * length 0; their table entries stay.
 *
 * pml_pages_compact: the L live pages move to numbers 0 .. L-1: the live pages
 * at or past L, ascending, to the free ones below it, ascending.  remap
 * [num_pages] says where each page went (-1: it was free), copy_src /
 * copy_dst [capacity >= num_pages / 2] list the moves for pml_pages_copy, -1
 * past *copy_count; ref_counts_out and block_table_out (which may be the
 * inputs) are the new state, entries past a row's length copied as they are.
 *
 * pml_pages_copy: for i < min(*copy_count, capacity), page copy_src[i] of
 * every layer is copied over page copy_dst[i]; layer l, page p starts at byte
 * l * layer_stride_bytes + p * page_stride_bytes.  No page is a source and a
 * target of one call, nor a target twice.  Page numbers outside the cache are
 * skipped (PML_STATUS_BAD_BLOCK).
 */
int pml_pages_fork(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                   int bt_width, int32_t* seq_lens, int rows, const int32_t* parents,
                   const int32_t* children, int n, int32_t* copy_src, int32_t* copy_dst,
                   int32_t* copy_count, void* stream);
int pml_pages_extend(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                     int bt_width, int32_t* seq_lens, int rows, const int32_t* new_lens,
                     int32_t* new_pages, int capacity, int32_t* new_count, void* stream);
int pml_pages_free(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                   int bt_width, int32_t* seq_lens, int rows, const int32_t* list, int n,
                   void* stream);
int pml_pages_compact(int32_t* ref_counts, int num_pages, int32_t* block_table, int64_t bt_stride,
                      int bt_width, const int32_t* seq_lens, int rows, int32_t* ref_counts_out,
                      int32_t* block_table_out, int64_t bt_out_stride, int32_t* remap,
                      int32_t* copy_src, int32_t* copy_dst, int capacity, int32_t* copy_count,
                      void* stream);
int pml_pages_copy(void* cache, int layers, int64_t layer_stride_bytes, int num_pages,
                   int64_t page_stride_bytes, int64_t page_bytes, const int32_t* copy_src,
                   const int32_t* copy_dst, const int32_t* copy_count, int capacity, void* stream);

/* Read (and, if clear != 0, reset) the current device's sticky status word.
 * Synchronises with the device (waits for all work queued so far). */
int pml_device_status(unsigned int* status, int clear);

#ifdef __cplusplus
}
#endif

#endif /* PML_H */
