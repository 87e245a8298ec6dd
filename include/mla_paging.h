/*
 * mla_paging.h -- C ABI of the operators around the paged MLA decode
 * (mla_decode.h): what a serving step does to the cache before the decode,
 * and the choice of the pages that a sparse decode reads.
 *
 *   mla_build_tables     pages handed out and taken back, page lists and slot
 *                        maps, all on the device from the request lengths
 *   mla_rope_append      rotary embedding (one or several position axes) of
 *                        queries and rope keys, RMS norm of the latent row,
 *                        both written into the paged cache
 *   mla_summarize_pages  one mean row for every page just completed
 *   mla_page_scores      a page's best score over the heads of a query
 *   mla_select_pages     the pages of the best scores, as a page list that
 *                        mla_decode_plan takes
 *
 * Conventions, as in mla_decode.h: device pointers of the current device
 * owned by the caller; every call queues its work on `stream`, allocates
 * nothing and does not synchronise (unless check_status is nonzero, where a
 * call has it), so it can be captured in a CUDA graph; the kernels are
 * programmatic dependent launches that wait for the kernel before them.  No
 * call throws, exits or traps.  Calls on different streams may overlap as
 * long as none writes what another reads or writes.
 *
 * The lengths that a step makes on the device are not read back: a decode is
 * planned from HOST offsets and lengths (mla_decode_plan), so the caller keeps
 * the lengths of its requests as well, and adds to them what it asks
 * mla_build_tables for.  A step that mla_build_tables refuses shows in its
 * status word alone.  Nothing of its tokens is written then (their slots are
 * -1), and a decode planned for the lengths it asked for reads page lists that
 * were not made: read the status before such a step's results are used.
 *
 * check_status != 0 waits for the stream and returns the first device error
 * recorded on this device since the last such call (MLA_ERR_DEVICE_BOUNDS: an
 * index outside its array, whose access was skipped; MLA_ERR_DEVICE_TIMEOUT: a
 * bounded wait ran out), and clears it.  All calls of this file that take
 * check_status share one word, whichever of them recorded the error and on
 * whichever stream: a step may check once, through its last call, and callers
 * that are to tell their errors apart check after each of their calls.  A call
 * of no tokens or rows checks without a kernel of its own.  It cannot be
 * captured.
 */
#ifndef MLA_PAGING_H
#define MLA_PAGING_H

#include <stdint.h>

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One step of the page tables of a batch of requests, on the device.
 *   Request b holds kv_len[b] tokens in the pages block_table[b, 0 ..
 *   ceil(kv_len[b] / page_size)).  new_len[b] >= 0 appends that many tokens;
 *   new_len[b] = -1 ends the request: its pages return to the free pages and
 *   its length becomes 0.
 *   Free pages are a stack: free_pages[0 .. free_count[0]), its top last.
 *   First the pages of ended requests are pushed (in request order, each
 *   request's in position order), then the new pages are popped one by one
 *   (in the same order).  New pages are written to block_table; entries past
 *   a request's pages keep what they held.
 *
 *   kv_len          [batch] int32
 *   new_len         [batch] int32
 *   kv_len_out      [batch] int32: the lengths after the step; may be kv_len
 *   block_table     [batch, table_stride] int32, max_pages entries of a row
 *                   used; updated in place
 *   free_pages      [num_pages] int32, updated in place
 *   free_count      [1] int32; free_count_out [1]: may be free_count
 *   kv_indptr       [batch + 1] int32: offsets into kv_indices after the step
 *   kv_indices      [indices_cap] int32: the page lists of all requests; what
 *                   lies past kv_indptr[batch] is left as it was
 *   q_indptr        [batch + 1] int32: offsets of each request's new tokens
 *   slots           [max_tokens] int64: page * page_size + offset of each new
 *                   token, requests in order; -1 past the last one
 *   positions       [max_tokens] int32: its position; 0 past the last one
 *   status          [1] int32, written by every call:
 *     MLA_OK                 the step was made;
 *     MLA_ERR_CAPACITY       too few free pages, or a request would exceed
 *                            max_pages (or 2^31 - 1 tokens), or the new
 *                            tokens max_tokens, or the page lists
 *                            indices_cap;
 *     MLA_ERR_INVALID_ARG    kv_len < 0 or past max_pages, new_len < -1,
 *                            free_count outside [0, num_pages], or more pages
 *                            coming back than the stack has room for;
 *     MLA_ERR_DEVICE_BOUNDS  the step was made, but a page id in use lies
 *                            outside [0, num_pages); slots in such a page
 *                            are -1.
 *     After CAPACITY or INVALID_ARG nothing has changed: kv_len_out and
 *     free_count_out hold the old values, every slot is -1 and every position
 *     0, and the other arrays are as they were.
 *   The arrays must not overlap, but for the two pairs named above.
 * Returns MLA_ERR_INVALID_ARG for sizes < 1 (num_pages, max_pages,
 * page_size), batch < 0, table_stride < max_pages or NULL pointers;
 * MLA_ERR_UNSUPPORTED for a page_size other than 16, 32 or 64;
 * MLA_ERR_CAPACITY for batch > 4096 or batch * max_pages, num_pages or
 * max_tokens past 2^31 - 1.  max_tokens = 0 (only ends) is allowed.
 */
mla_status_t mla_build_tables(const int32_t* kv_len, const int32_t* new_len, int32_t* kv_len_out,
                              int32_t* block_table, int64_t table_stride, int max_pages,
                              int32_t* free_pages, const int32_t* free_count,
                              int32_t* free_count_out, int num_pages, int batch, int page_size,
                              int32_t* kv_indptr, int32_t* kv_indices, int64_t indices_cap,
                              int32_t* q_indptr, int64_t* slots, int32_t* positions,
                              int64_t max_tokens, int32_t* status, void* stream);

/*
 * The rotary embedding: pair i of the 64 rope dims is turned by the angle
 *   positions[axis_of_pair[i], t] * inv_freq[i]   (radians)
 * and scaled by `scale`.  With several axes (time, height and width of an
 * image or video patch) each pair follows the axis named for it; text uses
 * one axis, or equal positions on all of them.
 */
typedef struct {
  int32_t n_axes;             /* rows of `positions`, 1 .. 8 */
  int32_t interleaved;        /* pair i: dims (2i, 2i+1) if nonzero, (i, i+32) if 0 */
  float scale;                /* factor on cos and sin (1 unless the context was extended) */
  int32_t axis_of_pair[32];   /* 0 .. n_axes - 1 */
  double inv_freq[32];        /* finite */
} mla_rope_t;

/*
 * The new tokens of a step: queries and rope keys rotated, the latent rows
 * normed, and both key parts written into the paged cache.
 * For each token t with slots[t] >= 0:
 *   q_pe_out[t, h]           = bf16(scale * rotate(q_pe[t, h]))
 *   ckv_cache[slots[t]]      = round(ckv[t] * norm_weight / sqrt(mean(ckv[t]^2) + eps) / kv_scale)
 *   kpe_cache[slots[t]]      = round(scale * rotate(kpe[t]) / kv_scale)
 * computed in fp32 and rounded once to the cache's type; an e4m3 cache
 * saturates at +-448 and keeps NaN.  Angles are first reduced to one turn, to
 * within 2^-31 turns at any position for frequencies up to 2^40 in magnitude
 * (larger ones lose up to a bit for each doubling).
 * A token with slots[t] < 0 is padding: nothing of it is written.  A slot
 * past the cache is reported (MLA_ERR_DEVICE_BOUNDS) and nothing of its token
 * is written either.  No two tokens may have the same slot.
 *   rope         HOST, read before the call returns
 *   positions    [n_axes, tokens] int32, axes axis_stride entries apart (0:
 *                the same positions for all axes)
 *   slots        [tokens] int64
 *   q_pe         bf16, element (t, h, d) at t * q_token_stride + h *
 *                q_head_stride + d; NULL (with num_heads 0): keys only
 *   q_pe_out     [tokens, num_heads, 64] bf16; may be q_pe where that is
 *                contiguous
 *   ckv          bf16, element (t, d) at t * ckv_stride + d, d < 512
 *   kpe          bf16, element (t, d) at t * kpe_stride + d, d < 64
 *   norm_weight  [512] bf16, or NULL: the latent rows are stored as they are
 *   eps          >= 0, finite
 *   ckv_cache    [num_pages, page_size, 512], kpe_cache [num_pages, page_size,
 *                64] of kv_dtype (BF16 or FP8_E4M3); kv_scale as in
 *                mla_decode_run
 * Strides count elements.  q_pe, ckv, kpe, norm_weight, the outputs and the
 * caches are 16-byte aligned, and the strides of q_pe, ckv and kpe multiples
 * of 8 (else MLA_ERR_INVALID_ARG).  num_heads 0 .. 1024; tokens <= 2^24
 * (else MLA_ERR_CAPACITY).
 */
mla_status_t mla_rope_append(const mla_rope_t* rope, const int32_t* positions,
                             int64_t axis_stride, const int64_t* slots, const void* q_pe,
                             int64_t q_token_stride, int64_t q_head_stride, void* q_pe_out,
                             const void* ckv, int64_t ckv_stride, const void* kpe,
                             int64_t kpe_stride, const void* norm_weight, float eps,
                             void* ckv_cache, void* kpe_cache, int kv_dtype, float kv_scale,
                             int num_pages, int page_size, int64_t tokens, int num_heads,
                             int check_status, void* stream);

/*
 * Summary rows of the pages that the tokens of a step completed: for every
 * token whose slot is the last of its page,
 *   summaries[page, d] = bf16(mean over the page's tokens of the cached row,
 *                             ckv dims then kpe dims, times kv_scale)
 * summed in fp32.  Other pages keep their summaries, so one call after each
 * mla_rope_append keeps those of all full pages current; the last, partly
 * filled page of a request has none (mla_select_pages keeps it unseen).
 *   slots        [tokens] int64, as for mla_rope_append: negative entries are
 *                skipped, entries past the cache reported and skipped
 *   ckv_cache, kpe_cache, kv_dtype, kv_scale  as for mla_rope_append
 *   summaries    [num_pages, 576] bf16, 16-byte aligned
 * tokens <= 2^24 (else MLA_ERR_CAPACITY).
 */
mla_status_t mla_summarize_pages(const int64_t* slots, int64_t tokens, const void* ckv_cache,
                                 const void* kpe_cache, int kv_dtype, float kv_scale,
                                 int num_pages, int page_size, void* summaries,
                                 int check_status, void* stream);

/*
 * scores[r, p] = max over the heads h of
 *     q_nope[r, h] . summaries[page, 0:512] + q_pe[r, h] . summaries[page, 512:576]
 * for the p-th page of row r's list, page = kv_indices[kv_indptr[r] + p]: how
 * much some head of the query wants the page's mean key.  All heads of a row
 * share one choice because they share the latent cache.  Products accumulate
 * in fp32.  A NaN product counts as -inf.
 *   q_nope     [rows, num_heads, 512] bf16;  q_pe [rows, num_heads, 64] bf16.
 *              Several query tokens of a request that are to share a choice
 *              are rows of one: num_heads = tokens x heads.
 *   summaries  [num_pages, 576] bf16
 *   kv_indptr  [rows + 1] int32 and kv_indices [n_indices] int32, DEVICE
 *   scores     fp32, max_pages entries of a row, rows score_stride apart;
 *              entries past a row's list are left as they were
 * num_heads 1 .. 128; q_nope, q_pe and summaries 16-byte aligned.  A page id
 * outside [0, num_pages) scores -inf and is reported; a row whose list leaves
 * kv_indices or is longer than max_pages (or 2^30 pages) is reported and
 * skipped.
 * 0 <= max_pages <= score_stride (else MLA_ERR_INVALID_ARG); rows <= 4096 (else
 * MLA_ERR_CAPACITY).
 */
mla_status_t mla_page_scores(const void* q_nope, const void* q_pe, const void* summaries,
                             int num_pages, const int32_t* kv_indptr, const int32_t* kv_indices,
                             int64_t n_indices, int rows, int num_heads, float* scores,
                             int64_t score_stride, int64_t max_pages, int check_status,
                             void* stream);

/*
 * The page lists of a sparse decode: of the n pages of row r, the first
 * keep_first, the last keep_last and the highest scoring of the others, in
 * all min(top_k, n), in their order.  Equal scores go to the lower position;
 * NaN counts as -inf; the scores of the kept ends are not looked at.
 *   scores, score_stride, max_pages, kv_indptr, kv_indices, n_indices  as above
 *   sel_indptr   [rows + 1] int32: offsets of each row's pages
 *   sel_indices  [sel_cap] int32: page ids, sel_cap >= rows * top_k; what lies
 *                past sel_indptr[rows] is left as it was
 * The last page is always kept, so a row's selected pages hold
 * (min(top_k, n) - 1) * page_size + (tokens of the last page) tokens: the
 * kv_len that mla_decode_plan takes with sel_indptr and sel_indices.
 * top_k >= 1, keep_first >= 0, keep_last >= 1 and keep_first + keep_last <=
 * top_k (else MLA_ERR_INVALID_ARG).  A row whose list leaves kv_indices or is
 * longer than max_pages is reported and counts as empty.  rows <= 4096,
 * rows * top_k <= 2^31 - 1 and sel_cap as above (else MLA_ERR_CAPACITY).
 */
mla_status_t mla_select_pages(const float* scores, int64_t score_stride, int64_t max_pages,
                              const int32_t* kv_indptr, const int32_t* kv_indices,
                              int64_t n_indices, int rows, int top_k, int keep_first,
                              int keep_last, int32_t* sel_indptr, int32_t* sel_indices,
                              int64_t sel_cap, int check_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PAGING_H */
