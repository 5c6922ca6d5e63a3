/*
 * ibp_kv_pages.h -- the part of the C ABI of libibp.so that gives the requests
 * of a step their pages: from the requests' lengths, on the GPU, the arrays that
 * the paged K/V calls (ibp_kv.h, ibp_kv8.h) take: page tables, q_start,
 * kv_len, and each new token's slot and position.  With it a decode loop (and
 * a HIP graph of one) needs no lengths on the host.
 *
 * Conventions are those of ibp_kv.h.
 */
#ifndef IBP_KV_PAGES_H
#define IBP_KV_PAGES_H

#include "ibp_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IBP_KV_MAX_REQUESTS (1u << 20)

/* The pages of a cache and who holds them.
 *   page_table    int32, a row of table_stride entries per request; entry j of a
 *                 request that holds h tokens is its page of tokens j * page_tokens
 *                 and on, for j < ceil(h / page_tokens).
 *   free_pages    int32[n_pages], a stack of the pages that nobody holds.
 *   n_pages       below 2^31; ids are in [0, n_pages).
 *   max_pages     entries of a row that may be used; of one row at most table_stride.
 *   page_tokens   in [1, IBP_KV_MAX_PAGE_TOKENS]. */
typedef struct {
    int32_t *page_table, *free_pages;
    uint64_t table_stride, n_pages;
    uint32_t max_pages, page_tokens;
} ibp_kv_page_pool;

/* What the requests of a step have and want; n_seqs at most IBP_KV_MAX_REQUESTS.
 *   had         int32[n_seqs]: tokens that request s holds.
 *   keep        int32[n_seqs]: how many of them stay (the first ones; the others were drafts
 *               that are rejected; 0 where the request has ended), or NULL: all.
 *   add         int32[n_seqs]: new tokens of the request in this step.
 *   free_count  int32[1]: pages on the stack.
 *   n_rows      rows of the step's batch, at least all new tokens together; below 2^31. */
typedef struct {
    const int32_t *had, *keep, *add, *free_count;
    uint64_t n_rows;
    uint32_t n_seqs;
} ibp_kv_step;

/* What a step's calls take.
 *   q_start     int32[n_seqs + 1]: the new tokens' rows, request after request; as ibp_kv_batch.
 *   kv_len      int32[n_seqs], as ibp_kv_batch: keep + add, or 0 for a request that is not served.
 *   length      int32[n_seqs]: tokens that the request holds now, the next step's `had`
 *               (keep + add, or had where it is not served).  May be `had` itself.
 *   free_count  int32[1]: pages on the stack now.  May be the step's free_count itself.
 *   unserved    int32[1]: requests that are not served, or NULL.
 *   slots       int64[n_rows]: of each row, page * page_tokens + place, as ibp_kv_append; -1 for a
 *               row behind the last request's, of a request that is not served, or whose page is
 *               outside [0, n_pages).
 *   positions   int64[n_rows]: keep + i of a request's i-th new token; -1 for a row behind the
 *               last request's or of one that is not served.  Or NULL. */
typedef struct {
    int32_t *q_start, *kv_len, *length, *free_count, *unserved;
    int64_t *slots, *positions;
} ibp_kv_assigned;

/*
 * ibp_kv_assign -- one step of the requests.  A request that then needs fewer
 * pages gives those behind its last token back: their ids go on the stack,
 * request after request, lower entries first (an entry outside [0, n_pages) is no
 * page and does not).  Then a request that needs more takes them from the top of the stack,
 * request after request, lower entries first; its page_table entries are written.  Other
 * entries are left as they are, those of pages given back too.
 *   Requests are served in their order.  Those whose rows would end behind
 *   n_rows, that would need more than max_pages pages or hold more than
 *   IBP_KV_MAX_TOKENS tokens are not served.  Where the stack runs short, the first
 *   request whose pages it cannot give is not served, nor is any behind it that needs
 *   pages.  A request that is not served keeps its tokens and pages, `keep` is
 *   not applied, and its rows' slots are -1: such a step places nothing of it and, with
 *   kv_len 0, attends nothing.
 *   Negative lengths count as 0, keep is at most had, a free_count outside [0, n_pages]
 *   is its nearer end, and pages that would pass the stack's n_pages entries
 *   are dropped.
 *   The stack and the lengths are what this call and its caller make them: a page
 *   that is on the stack twice, or there and in a row, is given to two requests.
 *   workspace   ibp_kv_assign_workspace() bytes, 16 B aligned (NULL if 0).
 * Steps of one pool must follow each other: two at a time race.
 * Run again with the same `had`, `keep`, `add` and free_count (outputs elsewhere) it gives the same again.
 * Errors: NULL pointer; sizes; alignment; arrays that overlap (IBP_ERR_SIZE).
 */
int ibp_kv_assign(const ibp_kv_page_pool *pool, const ibp_kv_step *step,
                  const ibp_kv_assigned *out, void *workspace, uint64_t workspace_bytes,
                  void *stream);

/* Workspace bytes of ibp_kv_assign for steps of these sizes (or smaller ones). */
int ibp_kv_assign_workspace(uint32_t n_seqs, uint64_t n_rows, uint64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* IBP_KV_PAGES_H */
