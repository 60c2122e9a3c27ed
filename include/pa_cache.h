/*
 * pa_cache.h -- C ABI of the cache operators: writing a paged K/V cache,
 * keeping it in 4 bits, and evicting keys from it.  They work on the caches,
 * block tables and lengths of pa.h, whose conventions (device pointers,
 * streams, 16-byte alignment, no allocation, status codes) hold here too.
 *
 * PA_MX4 cache
 *   Microscaled 4-bit floating point (the OCP MX format MXFP4): a K or V row
 *   of D elements is D/2 bytes of E2M1 codes (sign, 2 exponent bits, 1
 *   mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; element 2i
 *   in the low four bits of byte i) and D/32 E8M0 scale bytes e, one per block
 *   of 32 elements: value = code * 2^(e - 127); e = 255 makes the block NaN.
 *   Codes:  uint8 [pages, page_size, Hkv, D/2]  (NHD) or [pages, Hkv, page_size, D/2]  (HND).
 *   Scales: uint8 [pages, page_size, Hkv, D/32] (NHD) or [pages, Hkv, page_size, D/32] (HND).
 *   A row carries all it needs, so rows can move between pages.
 *
 * Key weights
 *   fp32 [pages][Hkv][page_size], in either layout: per cached key, the
 *   attention weight that pa_key_weights added up.  They belong to one
 *   sequence's keys: a page that several sequences share has no defined weights.
 *
 * device_error: int32 on the device, or NULL.  The kernels OR PA_DEV_* bits
 *   into it (they never clear it): PA_DEV_BAD_LENGTHS for q_lens or
 *   context_lens that are negative, above the declared maxima, q_lens[b] >
 *   context_lens[b], or a sum of q_lens that is not total_q_tokens;
 *   PA_DEV_BAD_PAGE for a block-table entry outside [0, num_pages) that the
 *   call has to look up.  The rows concerned are skipped, the rest is done: a
 *   key on such a page is not written, not read, seen by no query, given no
 *   weight, and the first to be evicted.  PA_DEV_WAIT_TIMEOUT (only
 *   pa_key_weights, with more than 16 rows of queries and heads): a pipeline
 *   wait ran out; the weights are then unspecified.
 *
 * total_q_tokens = 0 (all but pa_kv_evict): there is nothing to do.  The call
 *   returns PA_OK after its checks of the problem (and of the workspace), takes
 *   NULL for every other pointer, and launches nothing: lengths are not read, so
 *   q_lens that add up to more are not reported.
 *
 * Shapes: head_dim 64 or 128; page_size 16, 32, 64, 128 or 256; any number of
 * KV heads.  pa_problem's mask_q_tiles / mask_kv_tiles must be 0 and q_dtype
 * PA_BF16; fields an operator does not mention are not read by it, but must
 * hold valid values.
 */
#ifndef PA_CACHE_H
#define PA_CACHE_H

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* pa_decode_mx4 only, beside the PA_DEV_* codes of pa.h: a counter of the workspace
 * is none that a call leaves behind; rows of out and lse were not written. */
enum { PA_DEV_BAD_WORKSPACE = 8 };

/* pa_problem.kv_dtype of the operators below (the entry points of pa.h refuse it). */
enum { PA_MX4 = 2 };

/*
 * Write the K and V rows of the new tokens into the cache.  Row i of sequence
 * b (row sum(q_lens[0..b)) + i of k_new / v_new) is the token at position
 * context_lens[b] - q_lens[b] + i: context_lens already counts the new tokens,
 * as in attention.
 *   kv_dtype PA_BF16: rows are copied; k_scale and v_scale are not used.
 *   kv_dtype PA_MX4: rows are quantised.  Per block, e - 127 =
 *     floor(log2(largest magnitude)) - 2, at least -127; elements divided by
 *     2^(e - 127) round to the nearest E2M1 value, ties to the even code,
 *     saturating at 6.  A block with a NaN or an infinity gets e = 255 and
 *     zero codes, a block of zeros e = 0.
 *   E4M3 caches carry one scale per page, which new rows cannot join:
 *   PA_ERR_UNSUPPORTED.
 *   k_new, v_new: bf16 [total_q_tokens][Hkv][D], tokens k_stride / v_stride
 *     elements apart (multiples of 8, at least Hkv * D): they may be slices of
 *     a fused projection's output.
 *   key_weights: NULL, or the running weights, set to 0 for the new tokens.
 */
PA_API pa_status pa_kv_append(const pa_problem* problem, const void* k_new, const void* v_new,
                              int64_t k_stride, int64_t v_stride, const int32_t* block_table,
                              const int32_t* context_lens, const int32_t* q_lens, void* k_cache,
                              void* k_scale, void* v_cache, void* v_scale, float* key_weights,
                              int32_t* device_error, void* stream);

/*
 * Read the last q_lens[b] tokens of every sequence of a PA_MX4 cache back
 * into bf16 pages of the same layout and page size, at the same positions of
 * the page lists in dst_block_table (int32 [B][dst_max_pages_per_seq]); with
 * q_lens = context_lens the whole cache.  This is how pa_prefill, which takes
 * bf16 caches, attends to a prefix that is kept in 4 bits.  Values round to
 * bf16 only where they leave its range.
 *   k_out, v_out: bf16 caches of dst_num_pages pages; other slots are left alone.
 */
PA_API pa_status pa_kv_expand(const pa_problem* problem, const void* k_cache, const void* k_scale,
                              const void* v_cache, const void* v_scale,
                              const int32_t* block_table, const int32_t* context_lens,
                              const int32_t* q_lens, const int32_t* dst_block_table,
                              int32_t dst_max_pages_per_seq, int32_t dst_num_pages, void* k_out,
                              void* v_out, int32_t* device_error, void* stream);

/*
 * Decode attention over a PA_MX4 cache: the semantics of pa_decode_splitk
 * (causal, sliding window, GQA; at most 32 rows (Hq/Hkv) * max_q_len for
 * head_dim 128, 64 for head_dim 64) in one kernel launch.  The cache's length
 * is split over the GPU inside the kernel, and the parts of a split unit are
 * joined by the last CTA to finish one: no task map is built or read.
 * num_ctas and unit_cost have their pa.h meaning (num_ctas at most 1024);
 * balance_rows is not used.
 * The scores and the products with V are taken in f16 by the tensor cores with
 * fp32 sums; the block scales of K are applied in fp32.  What f16 rounds:
 *   - a probability by 2^-11 of itself, or 2^-32 of its row's largest where that
 *     is more (so that keys up to 22 nats below one that outweighs them all
 *     still count), in the product with V only: lse and the normalisation take
 *     it in fp32;
 *   - an element of q by 2^-25 of its row's largest, below 2^-14 of that (above,
 *     bf16's eight bits are exact);
 *   - a V block relative to the largest scale that its 32 columns met so far:
 *     what lies more than a factor 2^24 below that is lost.
 * Scores are summed before a query's power of two is put back (here, and in
 * pa_key_weights over PA_MX4 up to 16 rows): keys of 2^119 and more may
 * overflow to infinite scores, whatever the query.
 *   ws: >= pa_mx4_workspace_size bytes, 256-byte aligned, zero-filled by the
 *     caller before its first use.  Every call that runs to its end leaves it
 *     ready for the next one, of the same or another problem (a second launch to
 *     clear it would cost a small call more than its attention); its first 256
 *     bytes hold the error word that pa_last_device_error reads, which stays
 *     set until the caller clears them.  Calls that may run at the same time
 *     need a workspace each.  A workspace that was never filled, or that two
 *     calls used at once, is reported (PA_DEV_BAD_WORKSPACE) where its counters
 *     can no longer come out; it serves again once it is filled with zeros.
 *   Other arguments as pa_decode_splitk.
 */
PA_API size_t pa_mx4_workspace_size(const pa_problem* problem);
PA_API pa_status pa_decode_mx4(const pa_problem* problem, const void* q, const void* k_cache,
                               const void* k_scale, const void* v_cache, const void* v_scale,
                               const int32_t* block_table, const int32_t* context_lens,
                               const int32_t* q_lens, void* ws, size_t ws_bytes, void* out,
                               float* lse, void* stream);

/*
 * Add to every cached key's running weight the softmax weight that the given
 * queries give it:
 *   key_weights[j] += sum over queries i and the q heads of j's KV head of
 *                     exp(sm_scale * q_i . k_j - lse_i),
 * where query i sees key j as in attention (positions, sliding window).  lse
 * is what the attention call over the same queries wrote.  A query with lse =
 * -inf (no visible key) adds nothing.  The queries are the last q_lens[b]
 * tokens of each sequence, any number of them: a decode step's, or the last
 * few of a prompt.  kv_dtype PA_BF16 or PA_MX4 (k_scale for PA_MX4 only; E4M3
 * is PA_ERR_UNSUPPORTED).  Sums are in a fixed order: equal inputs give equal
 * bits.  (Hq / Hkv) * max_q_len decides between two kernels, whose sums differ
 * in order; pa_test_inject_wait_timeout reaches the one for more than 16 rows,
 * where skip_entry counts tiles of 256 keys.
 */
PA_API pa_status pa_key_weights(const pa_problem* problem, const void* q, const void* k_cache,
                                const void* k_scale, const int32_t* block_table,
                                const int32_t* context_lens, const int32_t* q_lens,
                                const float* lse, float* key_weights, int32_t* device_error,
                                void* stream);

/*
 * Evict: of every sequence longer than budget keep, per KV head, budget keys:
 * the first num_first, the last num_recent, and of the others those with the
 * largest weights (equal weights: the lower position; a NaN counts as less
 * than every number, and so does what a page outside the pool would hold:
 * where such a key is kept, its row is not copied).  The kept rows of K, V
 * (with their scales) and their weights are copied in ascending order to the
 * slots 0 .. budget-1 of the pages listed in dst_block_table (int32
 * [B][dst_max_pages_per_seq]), pages of the same pool that no sequence of the
 * call uses; the old pages are left as they are.  A sequence of at most budget
 * tokens is not touched, and its row of dst_block_table is not read.  After the
 * call attention reads the evicted sequences through their new pages with
 * new_context_lens; the relative order of their keys is kept, so causal
 * attention of tokens appended later is exact over what is left, while a
 * sliding window counts kept keys.
 *   budget >= 1; num_first, num_recent >= 0 and num_first + num_recent <= budget.
 *   kept: int32 [B][Hkv][budget]: the positions that were kept, ascending;
 *     rows of sequences that were not evicted are left alone.
 *   new_context_lens: int32 [B], min(context_lens[b], budget) (0 for a
 *     sequence with bad lengths); must not overlap context_lens.
 *   kv_dtype PA_BF16 or PA_MX4.  q_lens is not used: pa_problem's
 *   total_q_tokens and max_q_len may be 0.
 */
PA_API pa_status pa_kv_evict(const pa_problem* problem, int32_t budget, int32_t num_first,
                             int32_t num_recent, void* k_cache, void* k_scale, void* v_cache,
                             void* v_scale, float* key_weights, const int32_t* block_table,
                             const int32_t* dst_block_table, int32_t dst_max_pages_per_seq,
                             const int32_t* context_lens, int32_t* kept,
                             int32_t* new_context_lens, int32_t* device_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_CACHE_H */
