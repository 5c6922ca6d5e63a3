// kv_check.h -- argument checks that the entry points of the paged K/V calls share (api_kv*.hip): no
// HIP call but require_device's.  Each returns IBP_OK or sets the message and returns the status.
#pragma once

#include "kv.h"

namespace ibp {
namespace kv {
namespace check {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Workgroups of 256 threads a launch takes (its threads are counted in 32 bits).
constexpr uint64_t kMaxBlocks = 0xFFFFFFull;

inline int hip_fail(hipError_t e, const char* name) {
  if (e == hipErrorInvalidConfiguration)
    return set_error(IBP_ERR_SIZE, "%s: more workgroups than a launch takes", name);
  return set_error(IBP_ERR_HIP, "%s: HIP error %d (%s)", name, (int)e, hipGetErrorString(e));
}

inline int require_device(const char* name) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  return e == hipSuccess ? IBP_OK : hip_fail(e, name);
}

// Whether an array of these sizes and strides (elements, inner runs of
// `inner`) holds no element twice: sorted by stride, each stride covers what
// lies below it.  False also where the extent passes 2^62.
inline bool disjoint(const uint64_t* size, const uint64_t* stride, int n, uint64_t inner) {
  int order[3] = {0, 1, 2};
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if (stride[order[j]] < stride[order[i]]) {
        const int t = order[i];
        order[i] = order[j];
        order[j] = t;
      }
  __uint128_t extent = inner;
  for (int i = 0; i < n; ++i) {
    const uint64_t sz = size[order[i]], st = stride[order[i]];
    if (sz <= 1) continue;
    if (st < extent) return false;
    extent += (__uint128_t)st * (sz - 1);
    if (extent >> 62) return false;
  }
  return true;
}

// Extent of a (tokens, heads, head_dim) array in elements stays below 2^62.
inline bool extent_fits(uint64_t tokens, uint64_t token_stride, uint64_t heads, uint64_t head_stride) {
  const __uint128_t a = (__uint128_t)(tokens ? tokens - 1 : 0) * token_stride;
  const __uint128_t b = (__uint128_t)(heads ? heads - 1 : 0) * head_stride;
  return ((a + b) >> 62) == 0;
}

// Whether rows of a and of b, which have the same strides, share memory: some dt tokens and dh heads
// apart two rows start less than a row apart.
inline bool rows_overlap(const Rows& a, const Rows& b, uint64_t n_tokens, uint32_t head_dim) {
  typedef __int128 wide;
  if (n_tokens == 0) return false;
  const wide d = ((wide)(uintptr_t)b.p - (wide)(uintptr_t)a.p) / 2;
  const wide ts = n_tokens > 1 ? (wide)a.token_stride : 0, hs = a.head_stride, heads = a.n_heads;
  const wide reach = ts * (n_tokens - 1) + hs * (heads - 1) + head_dim;
  if (d >= reach || -d >= reach) return false;
  for (wide dh = 1 - heads; dh < heads; ++dh) {
    const wide rem = d + dh * hs;  // + dt * ts, the nearest to zero: one of two dt
    const wide dt = ts ? -rem / ts : 0;
    for (wide t = dt - 1; t <= dt + 1; ++t)
      if (t > -(wide)n_tokens && t < (wide)n_tokens && rem + t * ts < head_dim && -(rem + t * ts) < head_dim)
        return true;
  }
  return false;
}

inline bool same_strides(const Rows& a, const Rows& b) {
  return a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

// pools: also require k and v (a call that reads neither passes false).
inline int check_cache(const char* name, const ibp_kv_cache* c, bool pools, Cache* out) {
  if (!c || (pools && (!c->k || !c->v)))
    return set_error(IBP_ERR_NULL, "%s: cache and its k and v are required", name);
  if (c->dtype != IBP_KV_F16 && c->dtype != IBP_KV_BF16)
    return set_error(IBP_ERR_SIZE, "%s: dtype %u must be IBP_KV_F16 or IBP_KV_BF16", name, c->dtype);
  if (c->head_dim == 0 || c->head_dim % 8 != 0 || c->head_dim > IBP_KV_MAX_HEAD_DIM)
    return set_error(IBP_ERR_SIZE, "%s: head_dim %u must be a multiple of 8 in [8, %u]", name,
                     c->head_dim, IBP_KV_MAX_HEAD_DIM);
  if (c->n_heads == 0 || c->n_heads > 65535)
    return set_error(IBP_ERR_SIZE, "%s: n_heads %u must be in [1, 65535]", name, c->n_heads);
  if (c->page_tokens == 0 || c->page_tokens > IBP_KV_MAX_PAGE_TOKENS)
    return set_error(IBP_ERR_SIZE, "%s: page_tokens %u must be in [1, %u]", name, c->page_tokens,
                     IBP_KV_MAX_PAGE_TOKENS);
  if (c->n_pages > 0x7FFFFFFFull || (pools && c->n_pages == 0))
    return set_error(IBP_ERR_SIZE, "%s: n_pages %llu must be in [1, 2^31)", name,
                     (unsigned long long)c->n_pages);
  if (pools) {
    if (c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8 || !aligned(c->k, 16) ||
        !aligned(c->v, 16))
      return set_error(IBP_ERR_ALIGN, "%s: k, v must be 16 B aligned, strides multiples of 8", name);
    const uint64_t size[3] = {c->n_pages, c->page_tokens, c->n_heads};
    const uint64_t stride[3] = {c->page_stride, c->token_stride, c->head_stride};
    if (!disjoint(size, stride, 3, c->head_dim))
      return set_error(IBP_ERR_SIZE, "%s: rows of the cache overlap or pass 2^62 elements", name);
    if (c->n_heads > 1 && c->head_stride > 0xFFFFFFFFull)
      return set_error(IBP_ERR_SIZE, "%s: head_stride must be below 2^32", name);
  }
  out->k = (uint16_t*)c->k;
  out->v = (uint16_t*)c->v;
  out->page_stride = c->page_stride;
  out->token_stride = c->token_stride;
  out->head_stride = (uint32_t)c->head_stride;
  out->n_pages = (uint32_t)c->n_pages;
  out->n_heads = c->n_heads;
  out->head_dim = c->head_dim;
  out->page = fast_div(c->page_tokens);
  return IBP_OK;
}

// writes: the rows must not overlap.
inline int check_rows(const char* name, const char* what, const ibp_kv_rows* r, uint64_t n_tokens,
               uint32_t head_dim, bool writes, Rows* out) {
  if (!r || (n_tokens && !r->data)) return set_error(IBP_ERR_NULL, "%s: %s is required", name, what);
  if (r->n_heads == 0 || r->n_heads > 65535)
    return set_error(IBP_ERR_SIZE, "%s: %s: n_heads %u must be in [1, 65535]", name, what,
                     r->n_heads);
  if (r->token_stride % 8 || r->head_stride % 8 || !aligned(r->data, 16))
    return set_error(IBP_ERR_ALIGN, "%s: %s must be 16 B aligned, its strides multiples of 8", name,
                     what);
  if ((r->n_heads > 1 && r->head_stride > 0xFFFFFFFFull) ||
      !extent_fits(n_tokens, r->token_stride, r->n_heads, r->head_stride))
    return set_error(IBP_ERR_SIZE, "%s: %s: strides too large", name, what);
  if (writes) {
    const uint64_t size[2] = {n_tokens, r->n_heads};
    const uint64_t stride[2] = {r->token_stride, r->head_stride};
    if (!disjoint(size, stride, 2, head_dim))
      return set_error(IBP_ERR_SIZE, "%s: rows of %s overlap", name, what);
  }
  out->p = (uint16_t*)r->data;
  out->token_stride = r->token_stride;
  out->head_stride = (uint32_t)r->head_stride;
  out->n_heads = r->n_heads;
  return IBP_OK;
}

// pointers: the arrays are read (a workspace query passes false).  rows: the call has rows, and
// no sequence more than all of them: a larger max_q is none of the launch's size.
inline int check_batch(const char* name, const ibp_kv_batch* b, const Cache& c, bool pointers,
                bool rows, Batch* out) {
  if (!b) return set_error(IBP_ERR_NULL, "%s: batch is required", name);
  if (b->n_rows > 0x7FFFFFFFull || b->n_seqs > 0x7FFFFFFFu || b->max_q > 0x7FFFFFFFu)
    return set_error(IBP_ERR_SIZE, "%s: n_rows, n_seqs and max_q must be below 2^31", name);
  if (b->max_kv > IBP_KV_MAX_TOKENS)
    return set_error(IBP_ERR_SIZE, "%s: max_kv %u must be at most %u", name, b->max_kv,
                     IBP_KV_MAX_TOKENS);
  const uint32_t max_pages = b->max_kv ? c.page.div(b->max_kv - 1) + 1 : 0;
  if (b->n_seqs > 1 && b->table_stride < max_pages)
    return set_error(IBP_ERR_SIZE, "%s: table_stride %llu is below the %u pages of max_kv", name,
                     (unsigned long long)b->table_stride, max_pages);
  if (b->table_stride > (1ull << 40))
    return set_error(IBP_ERR_SIZE, "%s: table_stride too large", name);
  if (pointers && b->n_seqs) {
    if (!b->q_start || !b->kv_len || (max_pages && !b->page_table))
      return set_error(IBP_ERR_NULL, "%s: q_start, kv_len and page_table are required", name);
    if (!aligned(b->q_start, 4) || !aligned(b->kv_len, 4) || !aligned(b->page_table, 4))
      return set_error(IBP_ERR_ALIGN, "%s: misaligned index array", name);
  }
  out->q_start = b->q_start;
  out->kv_len = b->kv_len;
  out->table = b->page_table;
  out->table_stride = b->table_stride;
  out->n_rows = (uint32_t)b->n_rows;
  out->n_seqs = b->n_seqs;
  out->max_q = rows && b->max_q > b->n_rows ? (uint32_t)b->n_rows : b->max_q;
  out->max_kv = b->max_kv;
  out->max_pages = max_pages;
  return IBP_OK;
}

inline int check_group(const char* name, const Cache& c, uint32_t n_q_heads) {
  if (n_q_heads == 0 || n_q_heads > 65535 || n_q_heads % c.n_heads != 0)
    return set_error(IBP_ERR_SIZE, "%s: %u query heads are no multiple of the cache's %u", name,
                     n_q_heads, c.n_heads);
  return IBP_OK;
}

inline int check_items(const char* name, uint64_t rows, uint64_t heads) {
  if (rows * heads > kMaxBlocks)
    return set_error(IBP_ERR_SIZE, "%s: rows x heads must be below 2^24", name);
  return IBP_OK;
}

inline int check_workspace(const char* name, const void* ws, uint64_t have, uint64_t need) {
  if (need == 0) return IBP_OK;
  if (!ws) return set_error(IBP_ERR_NULL, "%s: a workspace of %llu bytes is required", name,
                            (unsigned long long)need);
  if (have < need)
    return set_error(IBP_ERR_SIZE, "%s: workspace of %llu bytes, %llu needed", name,
                     (unsigned long long)have, (unsigned long long)need);
  if (!aligned(ws, 16)) return set_error(IBP_ERR_ALIGN, "%s: misaligned workspace", name);
  return IBP_OK;
}

inline int check_select(const char* name, uint32_t n_select) {
  if (n_select == 0 || n_select > IBP_KV_MAX_SELECT)
    return set_error(IBP_ERR_SIZE, "%s: n_select %u must be in [1, %u]", name, n_select,
                     IBP_KV_MAX_SELECT);
  return IBP_OK;
}

}  // namespace check
}  // namespace kv
}  // namespace ibp
