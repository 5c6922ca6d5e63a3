// api_kv8.hip -- the extern "C" entry points of include/ibp_kv8.h: argument checks before any HIP
// call, then the launchers of the kernel files.
#include <math.h>

#include "kv8.h"
#include "kv_check.h"

using ibp::set_error;
using namespace ibp::kv::check;

namespace {

// pools: also require the codes and exponents (a workspace query passes false).
int check_cache8(const char* name, const ibp_kv8_cache* c, bool pools, ibp::kv::Cache8* out) {
  if (!c || (pools && (!c->k || !c->v || !c->k_exp || !c->v_exp)))
    return set_error(IBP_ERR_NULL, "%s: cache and its k, v, k_exp and v_exp are required", name);
  if (c->head_dim == 0 || c->head_dim % 16 != 0 || c->head_dim > IBP_KV_MAX_HEAD_DIM)
    return set_error(IBP_ERR_SIZE, "%s: head_dim %u must be a multiple of 16 in [16, %u]", name,
                     c->head_dim, IBP_KV_MAX_HEAD_DIM);
  if (c->n_heads == 0 || c->n_heads > 65535)
    return set_error(IBP_ERR_SIZE, "%s: n_heads %u must be in [1, 65535]", name, c->n_heads);
  if (c->page_tokens == 0 || c->page_tokens > IBP_KV_MAX_PAGE_TOKENS)
    return set_error(IBP_ERR_SIZE, "%s: page_tokens %u must be in [1, %u]", name, c->page_tokens,
                     IBP_KV_MAX_PAGE_TOKENS);
  if (c->block_tokens == 0 || c->page_tokens % c->block_tokens != 0)
    return set_error(IBP_ERR_SIZE, "%s: block_tokens %u must divide page_tokens %u", name,
                     c->block_tokens, c->page_tokens);
  if (c->n_pages > 0x7FFFFFFFull || (pools && c->n_pages == 0))
    return set_error(IBP_ERR_SIZE, "%s: n_pages %llu must be in [1, 2^31)", name,
                     (unsigned long long)c->n_pages);
  if (pools) {
    if (c->page_stride % 16 || c->token_stride % 16 || c->head_stride % 16 || !aligned(c->k, 16) ||
        !aligned(c->v, 16))
      return set_error(IBP_ERR_ALIGN, "%s: k, v must be 16 B aligned, strides multiples of 16", name);
    const uint64_t size[3] = {c->n_pages, c->page_tokens, c->n_heads};
    const uint64_t stride[3] = {c->page_stride, c->token_stride, c->head_stride};
    if (!disjoint(size, stride, 3, c->head_dim))
      return set_error(IBP_ERR_SIZE, "%s: rows of the cache overlap or pass 2^62 elements", name);
    if (c->n_heads > 1 && c->head_stride > 0xFFFFFFFFull)
      return set_error(IBP_ERR_SIZE, "%s: head_stride must be below 2^32", name);
  }
  out->k = (uint8_t*)c->k;
  out->v = (uint8_t*)c->v;
  out->k_exp = c->k_exp;
  out->v_exp = c->v_exp;
  out->page_stride = c->page_stride;
  out->token_stride = c->token_stride;
  out->head_stride = (uint32_t)c->head_stride;
  out->n_pages = (uint32_t)c->n_pages;
  out->n_heads = c->n_heads;
  out->head_dim = c->head_dim;
  out->page_blocks = c->page_tokens / c->block_tokens;
  out->page = ibp::kv::fast_div(c->page_tokens);
  out->block = ibp::kv::fast_div(c->block_tokens);
  return IBP_OK;
}

int check_dtype(const char* name, uint32_t dtype) {
  if (dtype != IBP_KV_F16 && dtype != IBP_KV_BF16)
    return set_error(IBP_ERR_SIZE, "%s: dtype %u must be IBP_KV_F16 or IBP_KV_BF16", name, dtype);
  return IBP_OK;
}

// What check_batch asks of a cache.
ibp::kv::Cache paging(const ibp::kv::Cache8& c) {
  ibp::kv::Cache p = {};
  p.page = c.page;
  p.n_pages = c.n_pages;
  p.n_heads = c.n_heads;
  p.head_dim = c.head_dim;
  return p;
}

}  // namespace

extern "C" {

int ibp_kv8_append(const ibp_kv8_cache* cache, const ibp_kv_batch* batch, uint32_t dtype,
                   const ibp_kv_rows* k, const ibp_kv_rows* v, const ibp_kv_rows* q,
                   const ibp_kv_rows* q_out, const int64_t* positions, const float* rope,
                   uint64_t n_positions, uint32_t rope_dim, const void* q_norm, const void* k_norm,
                   float eps, unsigned flags, void* stream) {
  const char* name = "ibp_kv8_append";
  ibp::kv::Cache8 c;
  ibp::kv::Batch b;
  ibp::kv::Rows kr, vr, qr = {nullptr, 0, 0, 0}, qo = {nullptr, 0, 0, 0};
  int r;
  if (flags & ~IBP_KV_ROPE_INTERLEAVED)
    return set_error(IBP_ERR_FLAGS, "%s: unknown flags 0x%x", name, flags);
  if ((r = check_cache8(name, cache, true, &c)) || (r = check_dtype(name, dtype)) ||
      (r = check_batch(name, batch, paging(c), true, true, &b)) ||
      (r = check_rows(name, "k", k, b.n_rows, c.head_dim, false, &kr)) ||
      (r = check_rows(name, "v", v, b.n_rows, c.head_dim, false, &vr)))
    return r;
  if (kr.n_heads != c.n_heads || vr.n_heads != c.n_heads)
    return set_error(IBP_ERR_SIZE, "%s: k and v must have the cache's %u heads", name, c.n_heads);
  if (!q != !q_out) return set_error(IBP_ERR_NULL, "%s: q and q_out come together", name);
  if (q) {
    if ((r = check_rows(name, "q", q, b.n_rows, c.head_dim, false, &qr)) ||
        (r = check_rows(name, "q_out", q_out, b.n_rows, c.head_dim, true, &qo)) ||
        (r = check_items(name, b.n_rows, qr.n_heads)))
      return r;
    if (qr.n_heads != qo.n_heads)
      return set_error(IBP_ERR_SIZE, "%s: q has %u heads, q_out has %u", name, qr.n_heads, qo.n_heads);
    if (b.n_rows && qr.p == qo.p && !same_strides(qr, qo))
      return set_error(IBP_ERR_SIZE, "%s: q_out in place of q needs q's strides", name);
    if (qr.p != qo.p && same_strides(qr, qo) && rows_overlap(qr, qo, b.n_rows, c.head_dim))
      return set_error(IBP_ERR_SIZE, "%s: q_out overlaps q without being q", name);
  }
  if (c.k == c.v || c.k_exp == c.v_exp)
    return set_error(IBP_ERR_SIZE, "%s: k and v of the cache are the same memory", name);
  if (rope) {
    if (rope_dim == 0 || rope_dim % 16 != 0 || rope_dim > c.head_dim)
      return set_error(IBP_ERR_SIZE, "%s: rope_dim %u must be a multiple of 16 in [16, head_dim]",
                       name, rope_dim);
    if (n_positions > (1ull << 48))
      return set_error(IBP_ERR_SIZE, "%s: n_positions too large", name);
    if (b.n_rows && !positions) return set_error(IBP_ERR_NULL, "%s: rope needs positions", name);
  }
  if (!(eps >= 0.f) || !isfinite(eps))
    return set_error(IBP_ERR_SIZE, "%s: eps must be finite and not negative", name);
  if (!aligned(positions, 8) || !aligned(rope, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16))
    return set_error(IBP_ERR_ALIGN, "%s: misaligned pointer", name);
  if ((r = require_device(name))) return r;
  hipError_t e = ibp::kv::launch_append8(c, dtype, b, kr, vr, qr, qo, positions, rope, n_positions,
                                         rope_dim, (flags & IBP_KV_ROPE_INTERLEAVED) != 0, q_norm,
                                         k_norm, eps, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int ibp_kv8_attend(const ibp_kv8_cache* cache, const ibp_kv_batch* batch, uint32_t dtype,
                   const ibp_kv_rows* q, const ibp_kv_rows* out, float scale, uint32_t window,
                   unsigned flags, float* lse, void* workspace, uint64_t workspace_bytes,
                   void* stream) {
  const char* name = "ibp_kv8_attend";
  ibp::kv::Cache8 c;
  ibp::kv::Batch b;
  ibp::kv::Rows qr, orow;
  int r;
  if (flags & ~IBP_KV_CAUSAL) return set_error(IBP_ERR_FLAGS, "%s: unknown flags 0x%x", name, flags);
  if (window && !(flags & IBP_KV_CAUSAL))
    return set_error(IBP_ERR_FLAGS, "%s: a window needs IBP_KV_CAUSAL", name);
  if ((r = check_cache8(name, cache, true, &c)) || (r = check_dtype(name, dtype)) ||
      (r = check_batch(name, batch, paging(c), true, true, &b)) ||
      (r = check_rows(name, "q", q, b.n_rows, c.head_dim, false, &qr)) ||
      (r = check_rows(name, "out", out, b.n_rows, c.head_dim, true, &orow)) ||
      (r = check_group(name, paging(c), qr.n_heads)) || (r = check_items(name, b.n_rows, qr.n_heads)))
    return r;
  if (orow.n_heads != qr.n_heads)
    return set_error(IBP_ERR_SIZE, "%s: out has %u heads, q has %u", name, orow.n_heads, qr.n_heads);
  if (b.n_rows && (orow.p == qr.p || (same_strides(orow, qr) && rows_overlap(orow, qr, b.n_rows, c.head_dim))))
    return set_error(IBP_ERR_SIZE, "%s: out must not overlap q", name);
  if (!(fabsf(scale) <= 0x1p125f))  // (scores are in the exponent of 2, of keys' halves: times 2.89)
    return set_error(IBP_ERR_SIZE, "%s: scale must be finite, its magnitude at most 2^125", name);
  if (lse && !aligned(lse, 4)) return set_error(IBP_ERR_ALIGN, "%s: misaligned lse", name);
  if ((r = require_device(name))) return r;
  uint64_t need = 0;
  hipError_t e = ibp::kv::attend8_workspace(c, b, qr.n_heads, &need);
  if (e != hipSuccess) return hip_fail(e, name);
  if ((r = check_workspace(name, workspace, workspace_bytes, need))) return r;
  if (b.n_rows == 0 || b.n_seqs == 0 || b.max_q == 0) return ibp::clear_error();
  e = ibp::kv::launch_attend8(c, dtype, b, qr, orow, scale, window > 0x7FFFFFFFu ? 0 : window,
                              (flags & IBP_KV_CAUSAL) != 0, lse, workspace, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int ibp_kv8_attend_workspace(const ibp_kv8_cache* cache, const ibp_kv_batch* batch,
                             uint32_t n_q_heads, uint64_t* bytes) {
  const char* name = "ibp_kv8_attend_workspace";
  if (!bytes) return set_error(IBP_ERR_NULL, "%s: bytes is required", name);
  ibp::kv::Cache8 c;
  ibp::kv::Batch b;
  int r;
  if ((r = check_cache8(name, cache, false, &c)) ||
      (r = check_batch(name, batch, paging(c), false, true, &b)) ||
      (r = check_group(name, paging(c), n_q_heads)) || (r = check_items(name, b.n_rows, n_q_heads)) ||
      (r = require_device(name)))
    return r;
  hipError_t e = ibp::kv::attend8_workspace(c, b, n_q_heads, bytes);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

}  // extern "C"
