/*
 * spec_cache.h -- C ABI of the cache side of a verify step on GB300 (sm_103a): what the target
 * model's forward over each request's k_b + 1 new tokens needs around its paged KV cache, and
 * what the cache needs around the verdict of spec_verify.
 *
 * Sources (the same pages as spec_verify.h):
 *  - "Speculative Decoding in Custom LLM Servicing: Implementing Draft Models in Rust": the
 *    append with its overflow error and the rollback ("KV Cache Rollback Mechanics"), the mask
 *    by which draft row i sees the L cached tokens and the rows up to itself (section on the
 *    speculative attention mask), freeing paged blocks after a rollback.
 *  - "Adding Speculative Decoding": k + 1 rows per request, requests with different k, the KV
 *    reservation of a speculative step.
 *
 * One step of a server, for B requests:
 *     spec_page_reserve          kv_seq_len[b] += k_b + 1, with pages to hold them
 *     per layer: spec_append     norm and rotate q and k, append k and v to the layer's cache
 *                spec_attention  the rows attend over the layer's cache
 *     spec_verify                (spec_verify.h) the logits' verdict: accept_len
 *     spec_cache_rollback        kv_seq_len[b] <- kv_seq_len[b] - k_b + a_b, the accepted drafts kept
 *     spec_page_release          pages past the new length, or out of the window, go back
 * and between steps spec_page_fork (a new request continues from another's tokens) and
 * spec_page_compact, each followed by spec_page_copy.
 *
 * Shared conventions are those of spec_verify.h: device pointers, no allocation, no host copy,
 * no synchronisation, host-visible errors returned with nothing enqueued, device-data errors
 * in the workspace's sticky error word (sv_read_device_error), no trap or assert.  Every kernel
 * is a programmatic dependent of the work before it on its stream and waits for that work before
 * it touches a caller's buffer; a kernel of the caller's that is launched with programmatic stream
 * serialization behind one of these must wait for its prerequisite grid likewise.  A call may be
 * captured into a graph.  Calls on several streams need a workspace each.
 *
 *  - The workspace's first 256 bytes are its header.  These calls add to the error word and do
 *    not clear it (spec_verify does): zero the header once before the first call.
 *  - Rows.  Request b owns rows [row_offsets[b], row_offsets[b+1]) (row_offsets == NULL:
 *    [b (k_max+1), (b+1) (k_max+1))) and uses its first num_drafts[b] + 1, as in spec_verify.
 *    num_drafts[b] == -1 marks an idle request: it has no new tokens, and every call here leaves
 *    it as it is.  (spec_verify knows no idle requests: give it 0 drafts for one and ignore its
 *    token.)  Rows that no request uses get zero outputs.
 *  - Lengths.  kv_seq_len[b] counts the new tokens: used row i of request b is the token at
 *    position kv_seq_len[b] - (num_drafts[b] + 1) + i.  A negative length marks a request whose
 *    reservation or fork failed; spec_append and spec_attention treat it as a layout error.
 *  - Pages.  Token position t of request b is slot t % page_size of page
 *    block_table[b, t / page_size]; -1 is no page.  Pages out of a sliding window may be -1.
 *  - A request with a device-data error (SV_DEV_BAD_LAYOUT: num_drafts, offsets or length out of
 *    range; SV_DEV_BAD_PAGE: a page it needs is not in [0, num_pages)) has NaN outputs, and
 *    nothing of it is written to the cache by the rows in error.
 *    row_offsets that do not ascend are reported too, but leave open which rows are whose: outputs
 *    and appended rows of any request are then unspecified, within the arrays.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device-data error codes of these calls, beside SV_DEV_BAD_LAYOUT. */
enum {
    SV_DEV_BAD_PAGE = 9,      /* a needed page id outside [0, num_pages), or a use count that
                                 does not fit what the call found                            */
    SV_DEV_NO_PAGES = 10,     /* the pool ran out                                            */
    SV_DEV_SHARED_PAGE = 11   /* the new tokens would be written into a page of two requests */
};

/* One layer's paged keys and values.  Element [page, slot, head, d] of k and of v is at
 * page * page_stride + slot * token_stride + head * head_stride + d: both the order
 * [page, slot, head, d] and [page, head, slot, d] are strides. */
typedef struct sv_kv_cache {
    void *k, *v;                    /* device, 16-byte aligned                                 */
    int64_t page_stride, token_stride, head_stride;   /* elements; positive multiples of 8    */
    int32_t num_pages;              /* pages in the pool                                       */
    int32_t page_size;              /* tokens per page: a power of two in [8, 256]             */
    int32_t num_heads;              /* key/value heads                                         */
    int32_t head_dim;               /* a multiple of 8: up to 256 (append), 128 (attention)    */
    sv_dtype dtype;                 /* SV_BF16 or SV_F16                                       */
    int32_t max_pages;              /* entries per request in block_table                      */
    const int32_t *block_table;     /* device int32 [B, max_pages]                             */
} sv_kv_cache;

/*
 * spec_append -- per-head norm and rotation of the new tokens' queries and keys, and the append
 * of keys and values to the cache, in one pass.
 *
 * For the token at position t and each query and key head x in R^head_dim:
 *     y = x / sqrt(mean(x^2) + eps) * weight            (weight NULL: y = x)
 *     for j < rotary_dim / 2, with (a, z) the j-th pair of y and angle = t * inv_freq[j]:
 *         (a, z) <- rope_scale * (a cos - z sin, a sin + z cos)
 * The j-th pair is (y[j], y[j + rotary_dim/2]), or (y[2j], y[2j+1]) with interleaved != 0;
 * elements from rotary_dim on are only normalised.  The query goes to out_q, the key and the
 * unchanged value to the token's slot of the cache.  Arithmetic is fp32, rounded once; the
 * angle is reduced exactly in fixed point, so far positions lose nothing.
 *
 *   q, k, v      device [total_rows, heads, head_dim], cache.dtype, 16-byte aligned; heads and
 *                elements contiguous, rows q_stride, k_stride, v_stride elements apart
 *                (multiples of 8): slices of one projection's output are fine.
 *   q_weight,    device [head_dim], cache.dtype; NULL: no norm of the queries / of the keys.
 *   k_weight
 *   inv_freq     device fp32 [rotary_dim / 2] (scaled variants: scale it); may be NULL with
 *                rotary_dim == 0.
 *   rotary_dim   even, 0 .. head_dim.
 *   out_q        device [total_rows, num_q_heads, head_dim], rows out_q_stride apart; may be q
 *                itself (with q's stride).
 * Sizes: 1 <= B < 2^25, 0 <= k_max <= 64, total_rows >= 1, num_q_heads a multiple of
 * cache.num_heads, both up to 1024.  Rows of a request in error: out_q NaN, cache untouched.
 */
sv_status spec_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, int32_t num_q_heads, const void *q_weight, const void *k_weight, float eps,
                      const float *inv_freq, int32_t rotary_dim, int32_t interleaved, float rope_scale,
                      const int32_t *num_drafts, const int32_t *row_offsets, const int32_t *kv_seq_len, int32_t B,
                      int32_t k_max, int32_t total_rows, sv_kv_cache cache, void *out_q, int64_t out_q_stride,
                      void *workspace, void *stream);

/*
 * spec_attention -- the new tokens' rows attend over the paged cache, which already holds them.
 *
 * Row i of request b, at position p, sees key j iff
 *     j <= p  and  (window == 0  or  j > p - window  or  j < sinks):
 * a causal mask with an optional sliding window and a few first tokens that stay visible.  With
 * S = the keys it sees, for each query head (its key/value head is head / (Hq / num_heads)):
 *     out = sum_{j in S} softmax_{j in S}(scale * q . k_j) v_j,   lse = log sum_{j in S} e^(scale q . k_j)
 * Every row sees at least its own token.  Scores, softmax and sums are fp32; the weights are
 * rounded to cache.dtype for the product with v (off by up to eps / 2 of sum_j p_j |v_j|, as much
 * again as the output's own rounding), and the output once.  The lse is good to
 * (T + 16) 2^-23 + 2^-22 |lse| over T keys, beside the rounding of the fp32 scores.
 * A masked key has no influence, whatever its slot holds (an unwritten slot may hold NaN).
 *
 *   q            device [total_rows, num_q_heads, head_dim], cache.dtype, rows q_stride elements
 *                apart (a multiple of 8), 16-byte aligned.
 *   window       >= 0; 0: no window.   sinks  >= 0 (no effect without a window).
 *   out          device [total_rows, num_q_heads, head_dim], contiguous, 16-byte aligned.
 *   out_lse      optional device fp32 [total_rows, num_q_heads] (unused rows: 0).
 *   workspace    sv_attention_workspace_bytes() bytes, 256-byte aligned.
 * Every wait inside the kernel is bounded (2 s): one that runs out ends the call with
 * SV_DEV_TIMEOUT in the error word and unspecified outputs, and the device stays usable.
 * Sizes as spec_append, and head_dim <= 128.  Results are the same from call to call: the split
 * of the work over the chip depends on the lengths alone, and parts are joined in a fixed order.
 */
sv_status spec_attention(const void *q, int64_t q_stride, int32_t num_q_heads, const int32_t *num_drafts,
                         const int32_t *row_offsets, const int32_t *kv_seq_len, int32_t B, int32_t k_max,
                         int32_t total_rows, sv_kv_cache cache, float scale, int32_t window, int32_t sinks, void *out,
                         float *out_lse, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of spec_attention for heads of head_dim, whatever the batch: the parts of rows whose
 * keys are split over the chip (0 for a head_dim that spec_attention does not take). */
size_t sv_attention_workspace_bytes(int32_t head_dim);

/*
 * Page bookkeeping.  The state is three device arrays that the caller owns: kv_seq_len [B],
 * block_table [B, max_pages] and ref_count [num_pages], the requests that hold each page.  A
 * page with count 0 is free.  Pages are always taken lowest id first, in request order, so the
 * result of every call is a function of its inputs alone.  An empty request has length 0 and a
 * table row of -1.  A page shared by several requests is always full, so no request writes to it.
 *
 * spec_page_reserve -- room for the new tokens of a step.
 * kv_seq_len[b] grows by num_drafts[b] + 1 (idle requests, -1: unchanged) and its table row gets
 * the pages that this needs.  Requests are served in order; one for which the free pages do not
 * suffice, counting those asked for before it, is SV_DEV_NO_PAGES.  Also SV_DEV_BAD_LAYOUT
 * (num_drafts < -1, a negative length, more than max_pages), SV_DEV_SHARED_PAGE and
 * SV_DEV_BAD_PAGE (the partly filled last page is shared, or not a page in use before the call).
 * Table entries past a request's length are overwritten, not given back: release them first.
 * A request that fails takes no page, and its length becomes -1 - length until the caller repairs
 * it, so that the step's other calls leave it alone.
 *   workspace  sv_page_workspace_bytes(B, num_pages) bytes, 256-byte aligned.
 *   B < 2^25, max_pages <= 2^20, num_pages < 2^28, B * max_pages < 2^40.
 */
sv_status spec_page_reserve(const int32_t *num_drafts, int32_t *kv_seq_len, int32_t B, int32_t *block_table,
                            int32_t max_pages, int32_t *ref_count, int32_t num_pages, int32_t page_size,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * spec_cache_rollback -- commits the verdict to the lengths: spec_rollback (spec_verify.h) for a
 * batch with idle requests.  kv_seq_len[b] <- kv_seq_len[b] - num_drafts[b] + accept_len[b]; an idle
 * request (num_drafts -1) keeps its length, and its accept_len is not looked at.  num_drafts < -1, an
 * accept_len outside [0, num_drafts], a negative length or a result outside [0, kv_seq_len]: the
 * request keeps its length, SV_DEV_BAD_LAYOUT.
 *   workspace  its header only (256 bytes).
 */
sv_status spec_cache_rollback(int32_t *kv_seq_len, const int32_t *accept_len, const int32_t *num_drafts, int32_t B,
                              void *workspace, void *stream);

/*
 * spec_page_fork -- requests children[f] (empty) continue from the first fork_len[f] tokens of
 * requests parents[f] (fork_len NULL: from all).  The parent's full pages are shared; a partly
 * filled last page becomes a fresh page of the child, and (copy_src[f], copy_dst[f]) is the pair
 * to copy in every layer (spec_page_copy), or (-1, -1).  Entries of -1 (out of a window) stay -1.
 * Lengths, tables and counts are read as they were before the call.  SV_DEV_BAD_LAYOUT: an index
 * outside [0, B), a child that is not empty or already taken by a lower f, fork_len outside
 * [1, kv_seq_len[parent]]; SV_DEV_BAD_PAGE: the partly filled page is not a page in use, or a
 * shared one is not (its entry becomes -1); SV_DEV_NO_PAGES as above, in order of f.  The error's
 * request is f.  A fork that fails shares nothing, its pair is (-1, -1), and a child that was empty
 * gets length -1 unless a lower f took it.
 */
sv_status spec_page_fork(const int32_t *parents, const int32_t *children, const int32_t *fork_len, int32_t num_forks,
                         int32_t *kv_seq_len, int32_t B, int32_t *block_table, int32_t max_pages, int32_t *ref_count,
                         int32_t num_pages, int32_t page_size, int32_t *copy_src, int32_t *copy_dst, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * spec_page_release -- pages past each request's length go back, and with window > 0 those that
 * no later row can see: pages whose tokens all lie at or before kv_seq_len[b] - window and at or
 * after `sinks`.  A released entry becomes -1 and its page's count falls by one.  A request that
 * ends has its length set to 0 before the call: all that it holds goes back, whatever a window left
 * of it.  Negative lengths are left alone.
 * SV_DEV_BAD_LAYOUT: a length past max_pages; SV_DEV_BAD_PAGE: an entry that is not a page in use
 * (it becomes -1).
 *   workspace  its header only (256 bytes).
 */
sv_status spec_page_release(const int32_t *kv_seq_len, int32_t B, int32_t *block_table, int32_t max_pages,
                            int32_t *ref_count, int32_t num_pages, int32_t page_size, int32_t window, int32_t sinks,
                            void *workspace, void *stream);

/*
 * spec_page_compact -- moves used pages down so that the pool's upper part is free.  With U pages
 * in use, the r-th used page at or above U goes to the r-th free page below U, for r < capacity.
 * Counts and tables are updated, and copy_src / copy_dst [capacity] receive the pairs to copy
 * (-1 past the last).  SV_DEV_BAD_PAGE: a table entry that is not a page in use, from U on (left as
 * it is; the error's request is its row).
 */
sv_status spec_page_compact(int32_t B, int32_t *block_table, int32_t max_pages, int32_t *ref_count,
                            int32_t num_pages, int32_t *copy_src, int32_t *copy_dst, int32_t capacity,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of spec_page_reserve, spec_page_fork (with num_forks <= B) and spec_page_compact.
 * 0 for invalid sizes. */
size_t sv_page_workspace_bytes(int32_t B, int32_t num_pages);

/*
 * spec_page_copy -- copies page copy_src[i] to page copy_dst[i], for each i < n with both >= 0, in
 * the keys and the values of num_layers layers.  A page is page_bytes contiguous bytes; page p of
 * layer l begins layer_stride * l + page_stride * p bytes into k and into v.  Everything is a
 * multiple of 16 bytes.  No page may be in two pairs, except as the source of both.
 * SV_DEV_BAD_PAGE: an id of num_pages or more (the pair is skipped; the error's request is i).
 *   v          may be NULL (keys only).     workspace  its header only (256 bytes).
 */
sv_status spec_page_copy(void *k, void *v, int64_t page_bytes, int64_t page_stride, int32_t num_layers,
                         int64_t layer_stride, int32_t num_pages, const int32_t *copy_src, const int32_t *copy_dst,
                         int32_t n, void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
