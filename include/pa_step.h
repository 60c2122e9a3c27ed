/*
 * pa_step.h -- C ABI of the operators of a serving step around attention:
 * pages and slot maps for the new tokens, rotary positions on their way into
 * the cache, and attention over the few pages that a cheap score selects.
 * They work on the caches, block tables and lengths of pa.h and pa_cache.h,
 * whose conventions (device pointers, streams, 16-byte alignment, no
 * allocation, status codes, shapes, device_error) hold here too.
 *
 * Row maps
 *   A step's new tokens are the rows 0 .. total_q_tokens-1, those of a sequence
 *   together, in order.  pa_pages_take writes, and the others read, int32
 *   [total_q_tokens] each:
 *     row_seq    the row's sequence, or -1: a row of padding (behind the last
 *                sequence's rows, and where a sequence's would be that got no
 *                pages).  Every operator leaves its outputs as they are.
 *     positions  its position in the sequence.  The row's query sees the keys
 *                j <= position (and > position - window), so no lengths are needed.
 *     slots      page * page_size + slot of its K and V rows in the cache, or -1:
 *                not in the cache.
 *   Any program may write them.  So that a step can be captured once for a
 *   number of rows, q_lens may add up to less than total_q_tokens.
 *
 * device_error: PA_DEV_BAD_LENGTHS for a row_seq >= num_seqs, a position
 *   outside [0, max_context_len), or bad lengths; PA_DEV_BAD_PAGE for a page
 *   number, block-table entry or slot outside the pool; PA_DEV_NO_PAGES.  The
 *   rows, pages or sequences concerned are skipped, the rest is done.
 *
 * total_q_tokens: at most 2^30 (more: PA_ERR_UNSUPPORTED).
 * total_q_tokens = 0 (all but pa_pages_*): returns PA_OK after the checks of the
 *   problem (and of the workspace) and launches nothing; the other pointers may
 *   be NULL.
 */
#ifndef PA_STEP_H
#define PA_STEP_H

#include "pa_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* pa_pages_take only, beside the PA_DEV_* codes of pa.h and pa_cache.h: the free
 * stack held too few pages. */
enum { PA_DEV_NO_PAGES = 16 };

/*
 * Give the new tokens of a step their pages, and map its rows.  Sequence b holds
 * seq_lens[b] tokens, whose pages block_table lists, and gets q_lens[b] more.
 * The pages that these need beyond those it has are taken from the top of the
 * stack free_pages[0 .. *free_count): sequences in order, a sequence's pages in
 * order, the first from free_pages[*free_count - 1] down.
 *   block_table: the entries of the new pages are written, others left alone.
 *   context_lens: int32 [B], written: seq_lens[b] + q_lens[b].
 *   row_seq, positions, slots: written, all total_q_tokens rows (-1, 0, -1 behind
 *     the last sequence's).  A token whose page the table already listed has
 *     its slot there (-1, and PA_DEV_BAD_PAGE, where that is none).
 *   free_left: int32 [1], written: *free_count less the pages taken; the stack
 *     itself is only read, so calls with equal inputs give equal results.
 *   *free_count outside [0, num_pages] is cut to that, with PA_DEV_BAD_LENGTHS.
 *   Where the stack runs out (PA_DEV_NO_PAGES), the sequence concerned and all
 *   after it that need pages get none: context_lens[b] = seq_lens[b], no entry of
 *   the table is written, and its rows become padding.
 *   A sequence with bad lengths (negative, q_lens[b] > max_q_len, or more than
 *   max_context_len together), or whose rows would pass total_q_tokens, is treated
 *   so too, with PA_DEV_BAD_LENGTHS (context_lens[b] is then cut to [0,
 *   max_context_len]).  Its q_lens, cut to [0, max_q_len], still count in where the
 *   rows of the sequences after it are.
 *   kv_dtype may be any.  num_pages * page_size at most 2^31 - 1.
 *   free_pages: int32 [num_pages].  Page numbers outside the pool on it are passed on as
 *   they are, with PA_DEV_BAD_PAGE, and slots of -1.
 *   What is written (block_table, context_lens, row_seq, positions, slots, free_left) must
 *   overlap neither an input nor each other: PA_ERR_INVALID_ARG.
 */
PA_API pa_status pa_pages_take(const pa_problem* problem, const int32_t* seq_lens,
                               const int32_t* q_lens, int32_t* block_table,
                               const int32_t* free_pages, const int32_t* free_count,
                               int32_t* context_lens, int32_t* row_seq, int32_t* positions,
                               int32_t* slots, int32_t* free_left, int32_t* device_error,
                               void* stream);

/*
 * Put pages back: sequence b held seq_lens[b] tokens and keeps the first
 * keep_lens[b] of them (0: it has finished; a few less: drafts that were not
 * accepted).  The pages that hold none of those go on top of the stack, sequences
 * in order, a sequence's pages in order: from free_pages[*free_count] up.
 *   free_pages: int32 [num_pages]; what is below *free_count (cut to [0, num_pages],
 *     with PA_DEV_BAD_LENGTHS, where it is outside) is left alone.  A push past its
 *     end is not done (PA_DEV_BAD_LENGTHS).
 *   free_left: int32 [1], written: the new number of pages on the stack.
 *   free_pages and free_left must overlap neither an input nor each other:
 *     PA_ERR_INVALID_ARG.
 *   block_table is only read; an entry outside the pool is put back as -1
 *     (PA_DEV_BAD_PAGE).  A page that several sequences share goes back once for
 *     each of them: keep such pages out of the call.
 *   Lengths that are negative, above max_context_len, or keep_lens[b] >
 *   seq_lens[b]: PA_DEV_BAD_LENGTHS, nothing of that sequence goes back.
 */
PA_API pa_status pa_pages_return(const pa_problem* problem, const int32_t* seq_lens,
                                 const int32_t* keep_lens, const int32_t* block_table,
                                 int32_t* free_pages, const int32_t* free_count,
                                 int32_t* free_left, int32_t* device_error, void* stream);

/* ------------------------------------------------------- rotary positions */

/* Frequencies of rotary positions scaled for contexts longer than the ones a
 * model was first trained on, from base^(-2i / rotary_dim):
 *   LINEAR  divided by factor;
 *   NTK     the base times factor^(rotary_dim / (rotary_dim - 2));
 *   YARN    pairs that make more than high_turns turns over original_context
 *           tokens as they are, fewer than low_turns divided by factor, between
 *           them a line over the pair's index (from the whole index at or before the
 *           first end, at least 0, to that at or behind the second, at most
 *           rotary_dim - 1); cos and sin times 0.1 ln(factor) + 1;
 *   BANDS   the same two ends, between them a line over the number of turns. */
enum { PA_ROPE_NONE = 0, PA_ROPE_LINEAR = 1, PA_ROPE_NTK = 2, PA_ROPE_YARN = 3, PA_ROPE_BANDS = 4 };

typedef struct pa_rope_scaling {
    int32_t kind;             /* PA_ROPE_*                                             */
    int32_t rotary_dim;       /* even, 2 .. 128                                        */
    double base;              /* > 1                                                   */
    double factor;            /* >= 1; all but NONE                                    */
    double original_context;  /* tokens, >= 1; YARN and BANDS                          */
    double high_turns;        /* > low_turns > 0; YARN and BANDS                       */
    double low_turns;
} pa_rope_scaling;

/* inv_freq: host, double [rotary_dim / 2], radians a position; cos_sin_scale: host,
 * double [1].  No CUDA call. */
PA_API pa_status pa_rope_inv_freq(const pa_rope_scaling* scaling, double* inv_freq,
                                  double* cos_sin_scale);

/* The form in which pa_rope_append takes frequencies (any, not only those of
 * pa_rope_inv_freq): steps[i] = inv_freq[i] / (2 pi), the turns a position, as a
 * fraction of 2^64.  Times a position it wraps where the angle does, so the angle
 * of a far position is as good as that of a near one: inv_freq's own 53 bits.
 * Host pointers, count entries each; inv_freq finite.  No CUDA call. */
PA_API pa_status pa_rope_steps(const double* inv_freq, int32_t count, uint64_t* steps);

typedef struct pa_rope {
    int32_t rotary_dim;     /* the first elements of a head, which turn: a multiple of 16,
                               16 .. head_dim; the rest stay as they are                */
    int32_t interleaved;    /* 0: element i turns with i + rotary_dim / 2; 1: 2i with 2i + 1 */
    float cos_sin_scale;    /* factor on cos and sin, finite; 1 for none                */
} pa_rope;

/*
 * Turn the new tokens' queries and keys to their positions and write the keys,
 * and the values as they are, into the cache: pair i of a head turns by
 * positions[t] * inv_freq[i],
 *   (x, y) -> cos_sin_scale * (x cos - y sin, y cos + x sin),
 * in fp32, rounded to bf16.  What is cached is what pa_kv_append caches of the
 * turned keys: kv_dtype PA_BF16, or PA_MX4 (quantised from the bf16 values; E4M3:
 * PA_ERR_UNSUPPORTED).
 *   rope: host.  steps: device, uint64 [rotary_dim / 2].
 *   q: bf16 [total_q_tokens][Hq][D], tokens q_stride elements apart, or NULL with
 *     q_out NULL; k_new, v_new as pa_kv_append's.  Strides: multiples of 8, at
 *     least a token's rows: the three may be slices of a fused projection's output.
 *   q_out: bf16 [total_q_tokens][Hq][D], dense; may be q itself where q is dense.  Any other
 *     overlap with the memory from the first to the last of q, k_new or v_new:
 *     PA_ERR_INVALID_ARG.
 *   positions: any int32 >= 0 (max_context_len does not bound them).
 *   A row whose slot is -1 is not cached and its q not written; other slots outside
 *   the pool: neither, and PA_DEV_BAD_PAGE; a negative position: neither, and
 *   PA_DEV_BAD_LENGTHS.  Two rows with one slot leave either's values in it.
 *   num_pages * page_size at most 2^31 - 1.
 */
PA_API pa_status pa_rope_append(const pa_problem* problem, const pa_rope* rope,
                                const uint64_t* steps, const void* q, const void* k_new,
                                const void* v_new, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, const int32_t* positions, const int32_t* slots,
                                void* q_out, void* k_cache, void* k_scale, void* v_cache,
                                void* v_scale, int32_t* device_error, void* stream);

/* ------------------------------------- attention over selected pages */

/*
 * Page bounds: per page and KV head, each channel's largest and smallest key, in
 * 8 bits.  With e the least exponent in [-50, 50] for which the largest magnitude
 * of all channels is at most 127 * 2^e (-50 for zeros),
 *   bounds      int8 [pages][Hkv][2][D]: ceil(largest / 2^e), then
 *               floor(smallest / 2^e), within [-127, 127];
 *   bound_scale fp32 [pages][Hkv]: 2^e.
 * Rounded outward they still bound the keys (below 127 * 2^50 in magnitude).  A
 * channel with a NaN has the bounds 127 and -127, a page with a NaN or an
 * infinity e = 50, so that such a page is looked at rather than lost.
 *
 * The call rewrites the bounds of every page in which the given rows have slots:
 * over the page's slots up to that of its last row in the call.  Rows of a page
 * stand together, in order, with none of another page or of -1 among them (as
 * pa_pages_take maps them); else which of its rows is the last is not said.  slots of
 * -1 are passed over.  k_cache: PA_BF16 (other kv_dtype: PA_ERR_UNSUPPORTED), with the new rows.
 * num_pages * page_size at most 2^31 - 1.
 */
PA_API pa_status pa_page_bounds(const pa_problem* problem, const void* k_cache,
                                const int32_t* slots, int8_t* bounds, float* bound_scale,
                                int32_t* device_error, void* stream);

/*
 * Select, for every row and KV head, budget pages of those its query sees keys of:
 * the num_first first and the num_recent last of them, and of the others those
 * with the highest score (equal scores: the lower position).  The score of a
 * page is an upper bound on the logits that the group's heads get from its keys,
 * with the query in 8 bits too: with e_h the least exponent in [-50, 50] for which
 * head h's largest magnitude is at most 127 * 2^e_h, and q8 = q_h / 2^e_h rounded
 * to the nearest whole number, ties to even (NaN: 0; within [-127, 127]),
 *   score = bound_scale * max over h of 2^e_h * sum over channels of
 *           q8 * (the channel's largest where q8 > 0, its smallest where q8 < 0).
 * Every sum is a whole number below 2^24, so scores, and lists, are exact.
 *   q: bf16 [total_q_tokens][Hq][D], dense, as pa_decode_selected takes it.
 *   selected: int32 [total_q_tokens][Hkv][budget], written: page indices in the
 *     sequence (positions / page_size), ascending, then -1: all pages where no
 *     more than budget are seen.  Rows that are skipped are left as they are.
 *   A page whose block-table entry is outside the pool has the lowest score
 *   (PA_DEV_BAD_PAGE, where scores are needed at all), and so has one whose
 *   bound_scale is negative or NaN: no bounds were written for it.
 *   budget >= 1; num_first, num_recent >= 0, together at most budget.  At most 64
 *   q heads a KV head; a context of at most PA_MAX_SELECT_PAGES pages
 *   (max_context_len / page_size): 720,896 tokens in pages of 16, 2.9 million of 64;
 *   num_ctas, kv_dtype and sm_scale have no part in it.
 */
#define PA_MAX_SELECT_PAGES 45056
PA_API pa_status pa_select_pages(const pa_problem* problem, int32_t budget, int32_t num_first,
                                 int32_t num_recent, const void* q, const int8_t* bounds,
                                 const float* bound_scale, const int32_t* block_table,
                                 const int32_t* row_seq, const int32_t* positions,
                                 int32_t* selected, int32_t* device_error, void* stream);

/*
 * Attention of every row over the pages listed for it (as pa_select_pages lists
 * them, or any other way): the semantics of pa_decode_splitk with the keys of
 * unlisted pages hidden.  The lists' lengths are split over the GPU inside the
 * kernel, and the parts of a split list joined by the last to finish one of them.
 *   selected: of row t and KV head h the entries 0 .. n-1, n = min(budget, pages
 *     that the row sees keys of); an entry of -1 among them is passed over, and so
 *     is one outside the row's pages [0, positions[t] / page_size] (PA_DEV_BAD_LENGTHS) or
 *     with a block-table entry outside the pool (PA_DEV_BAD_PAGE).  Order does not
 *     matter but for rounding.  No page should be listed twice for a row: whether it
 *     then counts once or twice is not said.
 *   With max_q_len > 1 up to six rows that stand together and are of one sequence
 *   (drafts, a chunk's tokens) are taken together, by a first launch that joins their
 *   lists: a page that several of them list is read once.  Nothing a row does not
 *   list, or sees, reaches its result, infinities and NaN included.
 *   A row with no visible key listed: out = 0, lse = -inf.
 *   kv_dtype PA_BF16 (other: PA_ERR_UNSUPPORTED); at most 32 q heads a KV head for
 *   head_dim 128, 64 for 64.
 *   The products are bf16 with fp32 sums, probabilities rounded to bf16 for the
 *   product with V (2^-8 of each); num_ctas and unit_cost have their pa.h meaning
 *   (num_ctas at most 1024; a unit_cost that, added to a unit's 64-token tiles, is 2^31 or
 *   more, or over all rows and KV heads more than 2^52: PA_ERR_UNSUPPORTED).
 *   With max_q_len > 1 rows * KV heads * budget is at most 2^56 (more: PA_ERR_UNSUPPORTED).
 *   ws: >= pa_selected_workspace_size bytes, 256-byte aligned, zero-filled before
 *     its first use; the rules of pa_decode_mx4's, whose workspace it must not be
 *     while either runs.  device errors: pa_last_device_error(ws).
 *   lse: fp32 [total_q_tokens][Hq], or NULL.
 */
PA_API size_t pa_selected_workspace_size(const pa_problem* problem, int32_t budget);
PA_API pa_status pa_decode_selected(const pa_problem* problem, int32_t budget, const void* q,
                                    const void* k_cache, const void* v_cache,
                                    const int32_t* block_table, const int32_t* row_seq,
                                    const int32_t* positions, const int32_t* selected, void* ws,
                                    size_t ws_bytes, void* out, float* lse, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_STEP_H */
