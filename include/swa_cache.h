/*
 * swa_cache.h — C ABI of libswa.so, serving side: a paged key/value cache held in 8 bits, attention
 * over it for single tokens and short runs of tokens, and its eviction by accumulated attention
 * weight.  Hand-written for NVIDIA GB300 (sm_103a); the training side is swa_attn.h, whose status
 * codes, ownership and error rules hold here too: the caller allocates every buffer, arguments are
 * checked on the host before anything is launched, calls are asynchronous on `stream`, allocate
 * nothing and never synchronise, so they can be captured in a CUDA graph.
 *
 * The cache is a pool of pages.  A page holds `page` consecutive tokens of one sequence for every
 * kv head; the tokens of one page and head form a block and share one scale for their keys and one
 * for their values:
 *
 *     value = e4m3 code * scale,      scale = 2^e,  -48 <= e <= 40
 *
 * so a code keeps e4m3's relative precision (2^-4) down to 2^-6 scale, and changing a block's scale
 * changes its codes only where they become subnormal.  Slot s of sequence b (0 = its first cached
 * token) is row s % page of page table[b][s / page].  `lens` holds how many tokens each sequence
 * had cached before the step's new tokens, in every call of the step; the caller adds the new
 * tokens to it afterwards.  The table, lens and new_lens are read on the device, so a captured step
 * replays with whatever they hold then.  max_pages * page < 2^30, pages * Hkv < 2^31, B * Hkv < 2^31,
 * and B and Hkv at most 65535.
 *
 * Alignment: 16 bytes for codes, k, v, q, o, the cache's weight and workspaces; 4 bytes (an element) for
 * scales, lse, the weights of append and key_weights, tables and lengths.
 *
 * What the device reads is checked there: a page number outside the pool, a sequence longer than
 * its table or a negative length is not followed; the call skips that page or sequence (attention
 * treats its tokens as unseen) and sets the device error word: swa_check_device returns
 * SWA_ERR_DEVICE_INDEX.
 */
#ifndef SWA_CACHE_H
#define SWA_CACHE_H

#include "swa_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct swa_cache {
    void* k;        /* e4m3 [pages, Hkv, page, D], 16-byte aligned, like v                    */
    void* v;
    float* k_scale; /* fp32 [pages, Hkv]                                                      */
    float* v_scale;
    float* weight;  /* fp32 [pages, Hkv, page] accumulated attention weights; may be NULL for
                       a cache that is never evicted from                                     */
    int pages;      /* >= 1                                                                   */
    int Hkv;        /* >= 1                                                                   */
    int page;       /* tokens of a page: 32, 64 or 128                                        */
    int D;          /* 64, 128 or 256                                                         */
} swa_cache;

/* Element types of the calls below. */
#define SWA_BF16 0
#define SWA_FP16 1
#define SWA_FP32 2

/*
 * Append: quantises n_b new tokens of each sequence into slots lens[b] .. lens[b] + n_b - 1.
 *   table    : int32 [B, max_pages]; the entries of the pages written must name pages that no other
 *              sequence holds, each once.
 *   lens     : int32 [B], tokens cached before.
 *   new_lens : int32 [B], n_b in 0..T, or NULL: n_b = T.
 *   k, v     : [B, Hkv, T, D] in `dtype` (bf16, fp16 or fp32); tokens n_b.. of a row are not read
 *              into the cache.
 *   weight   : fp32 [B, Hkv, T], the accumulated weights the tokens start with (a prompt's:
 *              swa_attn_key_weights), or NULL: zero.  Given with a cache without weights:
 *              SWA_ERR_INVALID_ARG.
 * A block's scale becomes max(its old scale if it holds older tokens, the least 2^e with
 * |x| <= 448 2^e for all its new elements); when that raises it, the older codes are rounded to the
 * new scale.  New codes are x / scale rounded to nearest even.  Slots of a page behind the last new
 * token are left as they were.
 * A token with an element that is NaN, infinite or above 448 * 2^40 in k or v is stored so that
 * attention gives NaN to every query that sees it and is unchanged for the others: its key is all
 * NaN codes, its value zeros, and it takes no part in the scales.
 */
swa_status swa_cache_append(const swa_cache* cache, const int* table, int max_pages,
                            const int* lens, const int* new_lens, const void* k, const void* v,
                            const float* weight, int B, int T, int dtype, cudaStream_t stream);

/*
 * Attention of T tokens of each sequence over its cache, the tokens themselves included (append
 * them first).  Query t of sequence b sits at slot lens[b] + t and sees slots s with
 * 0 <= lens[b] + t - s < window, for t < n_b (new_lens; NULL: n_b = T):
 *     x = scale <q, k_s>,  lse = ln sum exp(x),  p = exp(x - lse),  o = sum p v_s.
 *   q, o  : [B, Hq, T, D], bf16 or fp16 (`dtype`); Hq % Hkv == 0; 1 <= T <= 64; o may be q.
 *   lse   : fp32 [B, Hq, T].
 * Rows t >= n_b, and rows of skipped sequences, get o = 0, lse = -inf.  Pages wholly before every
 * window, and table entries behind the last token, are not read: a sliding layer's caller may reuse
 * them.
 *   accumulate : 1 -> weight of every cached token += the sum of its p over the T queries and the
 *                Hq / Hkv query heads of its kv head (needs cache->weight; the tables must then name
 *                each page once: two sequences that share one would add to the same weights at the
 *                same time); 0 -> weights untouched, and pages may be shared.
 *   workspace  : at least swa_cache_attn_window_workspace_bytes bytes for this window, 16-byte
 *                aligned (swa_cache_attn_workspace_bytes is enough for any); nothing is kept there
 *                between calls.  Calls that may overlap (other streams, graphs replayed at once)
 *                need workspaces of their own.  Accumulating takes 4 bytes for each row (T Hq) and
 *                slot that a sequence can see, min(max_pages page, window + T + 62), of up to 1024
 *                sequences, in units of 2 MB; up to twice that where a kv head has more than 64 rows.
 *                The size holds for the GPU that is current when it is asked for; 0 for sizes that
 *                the call refuses.
 * A key that a query does not see changes nothing for it, NaN included; where some queries of a call
 * see a token and others do not, this takes values that are finite, as append stores them.
 * A query with an element that is NaN or infinite gets o, lse and the weights that it adds as NaN.
 * Scores, softmax statistics and sums are fp32.  q is taken as fp16 operands after scaling each row
 * by a power of two (exact for bf16 and fp16 values down to 2^-28 of the row's largest, and below
 * that within 2^-39 of the largest), codes are exact in fp16, and p is rounded to fp16 as the second
 * product's operand (relative 2^-11, half the step of an fp16 result).  The same call on one GPU gives the
 * same bits (another max_pages may divide the work otherwise).  Accumulated weights are exp(x - lse) of
 * both in fp32: beside the score's own error, relative to within |x| 2^-22.
 */
size_t swa_cache_attn_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages,
                                      int page, int accumulate);
size_t swa_cache_attn_window_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int max_pages,
                                             int page, int window, int accumulate);
swa_status swa_cache_attn(const swa_cache* cache, const int* table, int max_pages,
                          const int* lens, const int* new_lens, const void* q, void* o, float* lse,
                          int B, int Hq, int T, int window, float scale, int accumulate, int dtype,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Eviction: cuts each sequence and kv head to min(lens[b], budget) tokens.  When lens[b] > budget
 * the last `recent` slots stay, and of the others the budget - recent with the largest accumulated
 * weight (equal weights: the lower slot; NaN above every number); the survivors keep their order.
 * They are written to slots 0, 1, .. of the pages of dst_table, with their weights; the pages of
 * `table` are only read, so they may be shared, and the caller frees them.
 *   dst_table : int32 [B, dst_pages] with dst_pages * page >= budget; its pages must not occur in
 *               `table`, nor twice (dst_table == table is refused).
 *   budget    : >= 1;  0 <= recent <= budget.
 *   kept      : int32 [B, Hkv, budget], the surviving slots in order, -1 behind the last.
 *   lens_out  : int32 [B], min(lens[b], budget); may be lens.
 * A sequence that is skipped (its length negative or longer than its table) keeps nothing: kept -1,
 * lens_out 0, no page written.  Whoever goes on with lens_out has dropped it, so swa_check_device, or
 * the lengths, come first where they can be wrong.  Tokens on a skipped page of `table` count as the
 * lightest; those that stay all the same are in kept, and their destination slots are left as they were,
 * like every slot of a skipped page of dst_table.
 * A destination block's scale is the largest of its tokens' old scales; slots behind the last
 * survivor are left as they were.  Window rules count cached tokens, so under a window evicted
 * tokens no longer count.  Needs cache->weight.
 */
swa_status swa_cache_evict(const swa_cache* cache, const int* table, int max_pages,
                           const int* lens, const int* dst_table, int dst_pages, int budget,
                           int recent, int* kept, int* lens_out, int B, cudaStream_t stream);

/*
 * The weight each key of a prompt received: after swa_attn_fwd / swa_attn_fwd_ex gave lse,
 *     w[b, hk, j] = sum over the query heads of kv head hk and the queries i that see key j of
 *                   exp(scale <q_i, k_j> - lse_i).
 *   q [B, Hq, Lq, D], k [B, Hkv, Lk, D] in bf16 or fp16 (`dtype`), lse fp32 [B, Hq, Lq],
 *   w fp32 [B, Hkv, Lk], fully written; shapes, window and causal as in swa_attn_fwd_ex.
 *   workspace : at least swa_attn_key_weights_workspace_bytes bytes (0 for many keys: it may then be
 *               NULL), 16-byte aligned; nothing is kept there between calls.  Calls that may overlap
 *               need workspaces of their own.  The size holds for the GPU that is current when it is
 *               asked for.
 * B Hkv ceil(Lk / 256) must stay below 2^30.  The N x N weights are never stored; scores, exponentials
 * and sums are fp32.  Bit-reproducible on one GPU.
 */
size_t swa_attn_key_weights_workspace_bytes(int B, int Hq, int Hkv, int Lq, int Lk, int D,
                                            int window, int causal);
swa_status swa_attn_key_weights(const void* q, const void* k, const float* lse, float* w, int B,
                                int Hq, int Hkv, int Lq, int Lk, int D, int window, int causal,
                                float scale, int dtype, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SWA_CACHE_H */
