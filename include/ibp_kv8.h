/*
 * ibp_kv8.h -- the part of the C ABI of libibp.so for a paged K/V cache held
 * in 8 bits: half of the memory, and of what attention has to read, of the cache
 * of ibp_kv.h.  A value is an e4m3 number (OCP 8-bit floating point, "e4m3fn":
 * 4 exponent and 3 mantissa bits, largest 448, no infinities) times a power of two
 * that a block of tokens shares in each head:
 *     value = code * 2^(exp - 127).
 * New keys and values are written by ibp_kv8_append, which also norms and
 * rotates them as ibp_kv_append does; ibp_kv8_attend is ibp_kv_attend over such
 * a cache.  A token's row of codes, n_heads x head_dim bytes, is a tensor that
 * ibp_compress_segments takes (with token_stride = n_heads * head_dim).
 *
 * Conventions are those of ibp_kv.h, but that codes count as elements of one byte:
 * code pointers are 16 B aligned, their strides and head_dim multiples of 16.
 * Rows of queries, new keys, new values and outputs are of 16 bits, ibp_kv_rows
 * of the given dtype (IBP_KV_F16 or IBP_KV_BF16).
 */
#ifndef IBP_KV8_H
#define IBP_KV8_H

#include "ibp_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged cache in 8 bits: codes as ibp_kv_cache's values; exponents
 * uint8[n_pages][page_tokens / block_tokens][n_heads], of k and of v.
 *   block_tokens  divides page_tokens: tokens b * block_tokens and on of a page share exponent b.
 *   head_dim      a multiple of 16 in [16, IBP_KV_MAX_HEAD_DIM].
 *   Exponents are in [1, 254] (0 is read as 1, 255 as 254).  A value past the range of the rows' type is
 *   read as up to twice the type's largest number, and as an infinity beyond.
 * No two rows may overlap (IBP_ERR_SIZE). */
typedef struct {
    void *k, *v;
    uint8_t *k_exp, *v_exp;
    uint64_t n_pages;
    uint64_t page_stride, token_stride, head_stride;
    uint32_t page_tokens, block_tokens, n_heads, head_dim;
} ibp_kv8_cache;

/*
 * ibp_kv8_append -- places the new tokens of a batch (row r at its position of its sequence,
 * as ibp_kv_batch says) in the cache; keys, and queries of the same tokens, are normed and
 * rotated on the way as by ibp_kv_append.
 *   In each block that gains tokens, for each head, of K and of V:
 *     e     the least in [1, 254] such that no finite new value is above 448 * 2^(e - 127) in
 *           magnitude (1 if all are zero); but if the block holds tokens of the sequence in front
 *           of the new ones, at least its exponent so far
 *     code  the e4m3 number next to value * 2^(127 - e), of two equally near the one with the even
 *           mantissa; infinities and NaN become NaN
 *     codes of the tokens in front, where the exponent rises: code * 2^(old - e), rounded the same.
 *   Tokens behind the new ones keep their codes and are of no account for e.
 *   A token is not placed whose position is negative or not below max_kv, whose page is
 *   not there, or whose entry of `positions` is outside [0, n_positions); its q_out row is zeros. For e
 *   the last counts as one of zeros: a block that would gain such tokens alone, from its first place on, has
 *   exponent 1 afterwards.
 *   Rows of no sequence, and new tokens past a sequence's first max_q, are left out: their q_out
 *   rows are left as they were.
 *   Two sequences that share a block and both extend it race.
 *   k, v, q, q_out, rope, positions, q_norm, k_norm, eps, flags
 *       as ibp_kv_append's; rows by batch->n_rows; positions int64[n_rows], the rotation's,
 *       required with rope.
 * The arithmetic is in 32 bits and is rounded once, at the end.
 * Errors: as ibp_kv_append's; block_tokens; one memory for k and v or for k_exp and v_exp.
 */
int ibp_kv8_append(const ibp_kv8_cache *cache, const ibp_kv_batch *batch, uint32_t dtype,
                   const ibp_kv_rows *k, const ibp_kv_rows *v, const ibp_kv_rows *q,
                   const ibp_kv_rows *q_out, const int64_t *positions, const float *rope,
                   uint64_t n_positions, uint32_t rope_dim, const void *q_norm,
                   const void *k_norm, float eps, unsigned flags, void *stream);

/*
 * ibp_kv8_attend -- ibp_kv_attend over a cache in 8 bits: the same rows, masks, outputs, log of the
 * sums and refusals (but scale at most 2^125), with K and V the values that the codes and exponents
 * stand for.  They are exact in the rows' type and somewhat past its range (above), but in IBP_KV_F16 below
 * 2^-20, where they are rounded to multiples of 2^-23, and in IBP_KV_BF16 values of V below 2^-94 and of K
 * below 2^-125, which may be taken as zero.  An output is the type's largest number at most, where its row sees
 * no value that is read as an infinity or NaN.
 *   workspace   ibp_kv8_attend_workspace() bytes, 16 B aligned (NULL if 0).
 * The keys of long sequences are shared out over the GPU only where the batch has fewer sequences (those of no
 * rows count too) than it runs workgroups for a key head: where max_q times the query heads of a key head
 * is up to 32, 1024 (512 above 16 or with head_dim above 128, 256 with both) over n_heads, times 4 if
 * 4 divides n_heads; above 32, where each 128 rows and query heads count, 512 (256 with head_dim above 128) over
 * n_heads.  In batches of more, a sequence has one workgroup for each key head (or four): 4 sequences of
 * 16,000 tokens with 40 key heads take 139 us among 101 sequences, 887 us among 128, and 162 in two calls over 64
 * each (as ibp_kv_attend says of chunks beside single tokens, which are faster given apart here too).
 */
int ibp_kv8_attend(const ibp_kv8_cache *cache, const ibp_kv_batch *batch, uint32_t dtype,
                   const ibp_kv_rows *q, const ibp_kv_rows *out, float scale, uint32_t window,
                   unsigned flags, float *lse, void *workspace, uint64_t workspace_bytes,
                   void *stream);

/* Workspace bytes of ibp_kv8_attend for a batch of these sizes (its pointers are not read), on
 * the current device. */
int ibp_kv8_attend_workspace(const ibp_kv8_cache *cache, const ibp_kv_batch *batch,
                             uint32_t n_q_heads, uint64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* IBP_KV8_H */
