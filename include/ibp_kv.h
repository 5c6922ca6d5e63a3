/*
 * ibp_kv.h -- the part of the C ABI of libibp.so that works on the dense K/V
 * rows the rest of the library (ibp.h) compresses and gathers: a paged K/V
 * cache of one layer in GPU memory, the placement of new keys and values in
 * it, attention over it, and the choice of the pages each query reads.
 *
 * A page is page_tokens token rows; a token's row is n_heads x head_dim
 * 16-bit values, the (layer, K|V, sequence, token) tensor that
 * ibp_compress_segments takes and ibp_gather_decompress_segments gives back.
 * With token_stride = n_heads * head_dim and page_stride = page_tokens *
 * token_stride a pool of pages is an array of such rows: row
 * page * page_tokens + slot of the pool is tensor `row` of a compressor call,
 * and a gather whose ids list the rows of pages writes whole pages.
 *
 * -------------------------------------------------------------- CONVENTIONS
 * Those of ibp.h: an ibp_status is returned, ibp_last_error() says why a call
 * was refused, nothing is enqueued on failure, work is enqueued on `stream` of
 * the current HIP device, the caller owns every buffer, the library keeps no
 * allocation and no state between calls, output is deterministic.  Calls allocate
 * nothing and synchronise nothing: they can be captured in a HIP graph.
 *   - Structs are host memory, read during the call.  Arrays in them, and
 *     every other pointer, are device memory.
 *   - Strides count elements.  Every data pointer is 16 B aligned, every
 *     stride and head_dim a multiple of 8 elements (16 B); channels are
 *     contiguous.  Index arrays are aligned to their type.
 *   - Lengths, page ids, slots and positions are read on the GPU and are not
 *     trusted: a value outside its range never leads to an access outside the
 *     buffers described (what it means is said at each call).
 *   - A workspace is written by the call that it is given to; calls that may
 *     run at the same time (two streams, two graphs) need one each.
 *   - What a call writes must not overlap what it reads, but where a call says
 *     that it may.
 */
#ifndef IBP_KV_H
#define IBP_KV_H

#include "ibp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IBP_KV_F16 0u
#define IBP_KV_BF16 1u
#define IBP_KV_MAX_HEAD_DIM 256u
#define IBP_KV_MAX_PAGE_TOKENS 65536u
#define IBP_KV_MAX_SELECT 4096u
#define IBP_KV_MAX_TOKENS (1u << 30)  /* of one sequence */

/* A paged cache: key token `slot` of page p, head h, starts at
 * k + p*page_stride + slot*token_stride + h*head_stride, values likewise.
 *   page_tokens in [1, IBP_KV_MAX_PAGE_TOKENS]; n_heads in [1, 65535];
 *   head_dim % 8 == 0 in [8, IBP_KV_MAX_HEAD_DIM]; dtype IBP_KV_F16 or
 *   IBP_KV_BF16; n_pages < 2^31.  No two rows may overlap (IBP_ERR_SIZE). */
typedef struct {
    void *k, *v;
    uint64_t n_pages;
    uint64_t page_stride, token_stride, head_stride;
    uint32_t page_tokens, n_heads, head_dim, dtype;
} ibp_kv_cache;

/* Rows of a batch of tokens, of the cache's dtype and head_dim: token t, head
 * h starts at data + t*token_stride + h*head_stride. */
typedef struct {
    void *data;
    uint64_t token_stride, head_stride;
    uint32_t n_heads;
} ibp_kv_rows;

/* Sequences of a call.  Sequence s holds kv_len[s] tokens in the cache; its
 * token at position j is slot j % page_tokens of page
 * page_table[s*table_stride + j / page_tokens].  Its new tokens are the last
 * ones: rows q_start[s] .. q_start[s+1]-1 of the batch's rows, row r being
 * position kv_len[s] - (q_start[s+1] - r).
 *   q_start     int32[n_seqs + 1], non-decreasing.
 *   kv_len      int32[n_seqs], new tokens included.  A negative one counts as 0.
 *   page_table  int32, n_seqs rows of table_stride entries, of which the
 *               first ceil(max_kv / page_tokens) are read where kv_len needs
 *               them; an entry outside [0, n_pages) is a page that is not
 *               there: its tokens are seen by no query.
 *   n_rows      rows of the batch (of q and out); rows x query heads below 2^24.
 *               Rows that belong to no sequence are left as they were.
 *   max_q       at least every q_start[s+1] - q_start[s]; new tokens of a
 *               sequence past the first max_q are left as they were.
 *   max_kv      at least every kv_len[s]; tokens at positions >= max_kv are
 *               not read.  At most IBP_KV_MAX_TOKENS. */
typedef struct {
    const int32_t *q_start, *kv_len, *page_table;
    uint64_t table_stride, n_rows;
    uint32_t n_seqs, max_q, max_kv;
} ibp_kv_batch;

/*
 * ibp_kv_append -- places the keys and values of n_tokens new tokens in the
 * cache; on the way each head of a key is normalised and rotated, and so are
 * the queries of the same tokens (written to q_out).
 *   slots      int64[n_tokens]: token t goes to slot slots[t] % page_tokens of
 *              page slots[t] / page_tokens (the pool's row slots[t]).  A token
 *              whose slot is outside [0, n_pages * page_tokens) (-1 pads a
 *              batch), or whose position is outside [0, n_positions), is not
 *              placed, and its q_out row is zeros.  Two tokens with one slot
 *              race.  Other rows of the cache are left as they were.
 *   k, v       n_heads = the cache's.  Values are copied as they are.
 *   q, q_out   NULL, or queries in and out (n_heads = q_out's); q_out may be q
 *              itself.
 *   rope       NULL, or float[n_positions][rope_dim]: row p holds rope_dim/2
 *              cosines, then rope_dim/2 sines.  Channel pair i < rope_dim/2 of
 *              position p turns as (a, b) -> (a cos - b sin, b cos + a sin)
 *              with (a, b) channels (i, i + rope_dim/2), or (2i, 2i + 1) under
 *              IBP_KV_ROPE_INTERLEAVED; channels >= rope_dim are not turned.
 *   positions  int64[n_tokens], required with rope.
 *   q_norm, k_norm  NULL, or head_dim weights of the cache's dtype: before the
 *              rotation x -> x * w / sqrt(mean(x^2) + eps), the mean over the
 *              head's channels.  eps >= 0, finite.
 * The arithmetic is in 32 bits and is rounded once, at the end.
 * Errors: NULL pointer; sizes (rope_dim not a multiple of 16 or > head_dim,
 * head counts, n_tokens >= 2^31, rows of q_out that overlap, q_out in part over
 * q, k and v of the cache the same memory); alignment; flags.
 */
#define IBP_KV_ROPE_INTERLEAVED 1u
int ibp_kv_append(const ibp_kv_cache *cache, const ibp_kv_rows *k, const ibp_kv_rows *v,
                  const ibp_kv_rows *q, const ibp_kv_rows *q_out, const int64_t *slots,
                  const int64_t *positions, uint64_t n_tokens, const float *rope,
                  uint64_t n_positions, uint32_t rope_dim, const void *q_norm,
                  const void *k_norm, float eps, unsigned flags, void *stream);

/*
 * ibp_kv_page_bounds -- for every page that holds a new token of the batch
 * (after ibp_kv_append of those tokens), the smallest and the largest key
 * value of each channel over the page's tokens (positions < kv_len).
 *   bounds  cache dtype, [n_pages][n_heads][2][head_dim] (0 = smallest, 1 =
 *           largest), indexed by page id.  Other pages' entries are left as they
 *           were.  A NaN key makes both bounds of its channel NaN.
 * A page that two sequences share and both extend is written by both (race).
 * n_rows is not used.
 * Errors: NULL pointer, sizes, alignment.
 */
int ibp_kv_page_bounds(const ibp_kv_cache *cache, const ibp_kv_batch *batch, void *bounds,
                       void *stream);

/*
 * ibp_kv_attend -- attention of the batch's rows over the cache.  For row r at
 * position p of its sequence and head h, with K and V of head
 * h / (q->n_heads / cache->n_heads), over the positions j it sees:
 *     out = sum_j exp(s_j) V_j / sum_j exp(s_j),   s_j = scale * <q, K_j>
 *     lse = log(sum_j exp(s_j))   (-inf for a row that sees nothing, or only
 *                                  scores of -inf; its out is zeros)
 * Row r sees positions 0 .. kv_len-1 of its sequence, under IBP_KV_CAUSAL
 * those <= p, with window > 0 those > p - window.
 * max_q decides how all sequences are run: where max_q times the query heads of a
 * key head is above 16, single tokens beside a chunk are right but slow (512
 * rows and 63 single tokens over up to 131,072 tokens 2.7 ms).  Two calls, over
 * the sequences up to s and from s on (q_start + s, kv_len + s, page_table + s *
 * table_stride; q, out and lse the same), are faster (0.9 ms).
 *   q, out     n_heads a multiple of the cache's, the same for both; out must
 *              not overlap q (refused where both have the same strides or start).
 *   lse        float[n_rows][q->n_heads] or NULL.
 *   window     0 = none; needs IBP_KV_CAUSAL (IBP_ERR_FLAGS).
 *   workspace  ibp_kv_attend_workspace() bytes, 16 B aligned (NULL if 0).
 * Scores, the softmax and the sums are in 32 bits; the weights exp(s - max)
 * are rounded to the cache's dtype where they multiply V.
 * A NaN or infinite value of V reaches that channel of every row that sees its
 * token, however small the weight, one of zero too: as a NaN, or as the infinity
 * where no NaN and no other infinity meets it.  A score that is NaN or +inf makes its row NaN.
 * Errors: NULL pointer; sizes (workspace too small; a grid past the
 * hardware's limits); alignment; unknown flags; scale not finite or past 2^126.
 */
#define IBP_KV_CAUSAL 1u
int ibp_kv_attend(const ibp_kv_cache *cache, const ibp_kv_batch *batch, const ibp_kv_rows *q,
                  const ibp_kv_rows *out, float scale, uint32_t window, unsigned flags,
                  float *lse, void *workspace, uint64_t workspace_bytes, void *stream);

/* Workspace bytes of ibp_kv_attend for a batch of these sizes (its pointers are
 * not read), on the current device. */
int ibp_kv_attend_workspace(const ibp_kv_cache *cache, const ibp_kv_batch *batch,
                            uint32_t n_q_heads, uint64_t *bytes);

/*
 * ibp_kv_select -- the pages that each row and key head attends: for row r at
 * position p, of its pages 0 .. L (L = p / page_tokens) always the n_first
 * first and the n_last last ones, and of the others the best, up to n_select
 * pages in all.  Page j's score is the largest value that a key within its
 * bounds could have against any query head of the key head's group,
 *     max over heads of sum over channels of max(q * lo_j, q * hi_j),
 * in 64 bits.  A higher score is better; NaN is above all others; of equal ones the
 * lower page is taken.  A page whose table entry is outside [0, n_bounds)
 * scores -inf.
 *   cache     geometry and dtype; its pools are not read, n_pages is not used.
 *   batch     page_table entries index `bounds` (a user whose pages are partly
 *             in host memory gives them ids of their own here).
 *   bounds    as ibp_kv_page_bounds writes them, n_bounds pages.
 *   n_last    >= 1 (the row's own page is always read: its bounds cover later
 *             tokens too); n_first + n_last <= n_select <= IBP_KV_MAX_SELECT.
 *   sel       int32[n_rows][cache->n_heads][n_select], page numbers of the
 *             sequence in ascending order, then -1.
 *   workspace ibp_kv_select_workspace() bytes, 16 B aligned: for each row and key
 *             head about 12 for each of the ceil(max_kv / page_tokens) pages, rounded up
 *             to 256 pages (none where n_select covers them all).  8,192 rows of 8
 *             heads over 4,096 pages take 3.2 GB: a long prompt's rows are best
 *             given some at a time (q and sel from that row on, n_rows and q_start
 *             of them alone, kv_len up to the last of them), one workspace for all.
 */
int ibp_kv_select(const ibp_kv_cache *cache, const ibp_kv_batch *batch, const void *bounds,
                  uint64_t n_bounds, const ibp_kv_rows *q, uint32_t n_first, uint32_t n_last,
                  uint32_t n_select, int32_t *sel, void *workspace, uint64_t workspace_bytes,
                  void *stream);
int ibp_kv_select_workspace(const ibp_kv_cache *cache, const ibp_kv_batch *batch,
                            uint32_t n_select, uint64_t *bytes);

/*
 * ibp_kv_attend_selected -- as ibp_kv_attend under IBP_KV_CAUSAL, each row and
 * key head over the pages of its own list only.
 *   sel  as ibp_kv_select writes it: int32[n_rows][cache->n_heads][n_select].
 *        Entries outside [0, ceil(max_kv / page_tokens)), and one that is not
 *        above the entry before it, are passed over.  (So a list in any other than
 *        ascending order may name a page twice with a smaller entry between; its keys then
 *        count twice.)
 */
int ibp_kv_attend_selected(const ibp_kv_cache *cache, const ibp_kv_batch *batch,
                           const ibp_kv_rows *q, const ibp_kv_rows *out, const int32_t *sel,
                           uint32_t n_select, float scale, float *lse, void *workspace,
                           uint64_t workspace_bytes, void *stream);
int ibp_kv_attend_selected_workspace(const ibp_kv_cache *cache, const ibp_kv_batch *batch,
                                     uint32_t n_q_heads, uint32_t n_select, uint64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* IBP_KV_H */
