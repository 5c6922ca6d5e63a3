// api_kv.hip -- the extern "C" entry points of include/ibp_kv.h: argument
// checks before any HIP call, then the launchers of the kernel files.
#include <math.h>

#include "kv_check.h"

using ibp::set_error;
using namespace ibp::kv::check;

namespace {

// Both attention calls; n_select == 0: over the whole cache.
int attend(const char* name, const ibp_kv_cache* cache, const ibp_kv_batch* batch,
           const ibp_kv_rows* q, const ibp_kv_rows* out, const int32_t* sel, uint32_t n_select,
           float scale, uint32_t window, bool causal, float* lse, void* workspace,
           uint64_t workspace_bytes, void* stream) {
  ibp::kv::Cache c;
  ibp::kv::Batch b;
  ibp::kv::Rows qr, orow;
  int r;
  if ((r = check_cache(name, cache, true, &c)) || (r = check_batch(name, batch, c, true, true, &b)) ||
      (r = check_rows(name, "q", q, b.n_rows, c.head_dim, false, &qr)) ||
      (r = check_rows(name, "out", out, b.n_rows, c.head_dim, true, &orow)) ||
      (r = check_group(name, c, qr.n_heads)) || (r = check_items(name, b.n_rows, qr.n_heads)))
    return r;
  if (orow.n_heads != qr.n_heads)
    return set_error(IBP_ERR_SIZE, "%s: out has %u heads, q has %u", name, orow.n_heads, qr.n_heads);
  if (b.n_rows && (orow.p == qr.p || (same_strides(orow, qr) && rows_overlap(orow, qr, b.n_rows, c.head_dim))))
    return set_error(IBP_ERR_SIZE, "%s: out must not overlap q", name);
  if (!(fabsf(scale) <= 0x1p126f))  // (scores are in the exponent of 2: times 1.44)
    return set_error(IBP_ERR_SIZE, "%s: scale must be finite, its magnitude at most 2^126", name);
  if (n_select && b.n_rows) {
    if (!sel) return set_error(IBP_ERR_NULL, "%s: sel is required", name);
    if (!aligned(sel, 4)) return set_error(IBP_ERR_ALIGN, "%s: misaligned sel", name);
  }
  if (lse && !aligned(lse, 4)) return set_error(IBP_ERR_ALIGN, "%s: misaligned lse", name);
  if ((r = require_device(name))) return r;
  uint64_t need = 0;
  hipError_t e = ibp::kv::attend_workspace(c, b, qr.n_heads, n_select, &need);
  if (e != hipSuccess) return hip_fail(e, name);
  if ((r = check_workspace(name, workspace, workspace_bytes, need))) return r;
  if (b.n_rows == 0 || b.n_seqs == 0 || b.max_q == 0) return ibp::clear_error();
  e = ibp::kv::launch_attend(c, cache->dtype, b, qr, orow, n_select ? sel : nullptr, n_select, scale,
                             window > 0x7FFFFFFFu ? 0 : window, causal, lse, workspace,
                             (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int attend_workspace(const char* name, const ibp_kv_cache* cache, const ibp_kv_batch* batch,
                     uint32_t n_q_heads, uint32_t n_select, uint64_t* bytes) {
  if (!bytes) return set_error(IBP_ERR_NULL, "%s: bytes is required", name);
  ibp::kv::Cache c;
  ibp::kv::Batch b;
  int r;
  if ((r = check_cache(name, cache, false, &c)) || (r = check_batch(name, batch, c, false, true, &b)) ||
      (r = check_group(name, c, n_q_heads)) || (r = check_items(name, b.n_rows, n_q_heads)) ||
      (r = require_device(name)))
    return r;
  hipError_t e = ibp::kv::attend_workspace(c, b, n_q_heads, n_select, bytes);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

}  // namespace

extern "C" {

int ibp_kv_append(const ibp_kv_cache* cache, const ibp_kv_rows* k, const ibp_kv_rows* v,
                  const ibp_kv_rows* q, const ibp_kv_rows* q_out, const int64_t* slots,
                  const int64_t* positions, uint64_t n_tokens, const float* rope,
                  uint64_t n_positions, uint32_t rope_dim, const void* q_norm, const void* k_norm,
                  float eps, unsigned flags, void* stream) {
  const char* name = "ibp_kv_append";
  ibp::kv::Cache c;
  ibp::kv::Rows kr, vr, qr = {nullptr, 0, 0, 0}, qo = {nullptr, 0, 0, 0};
  int r;
  if (flags & ~IBP_KV_ROPE_INTERLEAVED)
    return set_error(IBP_ERR_FLAGS, "%s: unknown flags 0x%x", name, flags);
  if (n_tokens > 0x7FFFFFFFull)
    return set_error(IBP_ERR_SIZE, "%s: n_tokens must be below 2^31", name);
  if ((r = check_cache(name, cache, true, &c)) ||
      (r = check_rows(name, "k", k, n_tokens, c.head_dim, false, &kr)) ||
      (r = check_rows(name, "v", v, n_tokens, c.head_dim, false, &vr)))
    return r;
  if (kr.n_heads != c.n_heads || vr.n_heads != c.n_heads)
    return set_error(IBP_ERR_SIZE, "%s: k and v must have the cache's %u heads", name, c.n_heads);
  if (!q != !q_out) return set_error(IBP_ERR_NULL, "%s: q and q_out come together", name);
  if (q) {
    if ((r = check_rows(name, "q", q, n_tokens, c.head_dim, false, &qr)) ||
        (r = check_rows(name, "q_out", q_out, n_tokens, c.head_dim, true, &qo)))
      return r;
    if (qr.n_heads != qo.n_heads)
      return set_error(IBP_ERR_SIZE, "%s: q has %u heads, q_out has %u", name, qr.n_heads,
                       qo.n_heads);
    if (n_tokens && qr.p == qo.p && !same_strides(qr, qo))
      return set_error(IBP_ERR_SIZE, "%s: q_out in place of q needs q's strides", name);
    if (qr.p != qo.p && same_strides(qr, qo) && rows_overlap(qr, qo, n_tokens, c.head_dim))
      return set_error(IBP_ERR_SIZE, "%s: q_out overlaps q without being q", name);
  }
  if (c.k == c.v)
    return set_error(IBP_ERR_SIZE, "%s: k and v of the cache are the same memory", name);
  if (rope) {
    if (rope_dim == 0 || rope_dim % 16 != 0 || rope_dim > c.head_dim)
      return set_error(IBP_ERR_SIZE, "%s: rope_dim %u must be a multiple of 16 in [16, head_dim]",
                       name, rope_dim);
    if (n_positions > (1ull << 48))
      return set_error(IBP_ERR_SIZE, "%s: n_positions too large", name);
    if (n_tokens && !positions)
      return set_error(IBP_ERR_NULL, "%s: rope needs positions", name);
  }
  if (n_tokens && !slots) return set_error(IBP_ERR_NULL, "%s: slots is required", name);
  if (!(eps >= 0.f) || !isfinite(eps))
    return set_error(IBP_ERR_SIZE, "%s: eps must be finite and not negative", name);
  if (!aligned(slots, 8) || !aligned(positions, 8) || !aligned(rope, 16) || !aligned(q_norm, 16) ||
      !aligned(k_norm, 16))
    return set_error(IBP_ERR_ALIGN, "%s: misaligned pointer", name);
  if ((r = require_device(name))) return r;
  hipError_t e = ibp::kv::launch_append(
      c, cache->dtype, kr, vr, qr, qo, slots, positions, (uint32_t)n_tokens, rope, n_positions,
      rope_dim, (flags & IBP_KV_ROPE_INTERLEAVED) != 0, q_norm, k_norm, eps, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int ibp_kv_page_bounds(const ibp_kv_cache* cache, const ibp_kv_batch* batch, void* bounds,
                       void* stream) {
  const char* name = "ibp_kv_page_bounds";
  ibp::kv::Cache c;
  ibp::kv::Batch b;
  int r;
  if ((r = check_cache(name, cache, true, &c)) ||
      (r = check_batch(name, batch, c, true, false, &b)))
    return r;
  if (!bounds) return set_error(IBP_ERR_NULL, "%s: bounds is required", name);
  if (!aligned(bounds, 16)) return set_error(IBP_ERR_ALIGN, "%s: misaligned bounds", name);
  if ((r = require_device(name))) return r;
  b.n_rows = 0x7FFFFFFFu;
  hipError_t e = ibp::kv::launch_page_bounds(c, cache->dtype, b, bounds, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int ibp_kv_attend(const ibp_kv_cache* cache, const ibp_kv_batch* batch, const ibp_kv_rows* q,
                  const ibp_kv_rows* out, float scale, uint32_t window, unsigned flags, float* lse,
                  void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* name = "ibp_kv_attend";
  if (flags & ~IBP_KV_CAUSAL) return set_error(IBP_ERR_FLAGS, "%s: unknown flags 0x%x", name, flags);
  if (window && !(flags & IBP_KV_CAUSAL))
    return set_error(IBP_ERR_FLAGS, "%s: a window needs IBP_KV_CAUSAL", name);
  return attend(name, cache, batch, q, out, nullptr, 0, scale, window, (flags & IBP_KV_CAUSAL) != 0,
                lse, workspace, workspace_bytes, stream);
}

int ibp_kv_attend_workspace(const ibp_kv_cache* cache, const ibp_kv_batch* batch,
                            uint32_t n_q_heads, uint64_t* bytes) {
  return attend_workspace("ibp_kv_attend_workspace", cache, batch, n_q_heads, 0, bytes);
}

int ibp_kv_select(const ibp_kv_cache* cache, const ibp_kv_batch* batch, const void* bounds,
                  uint64_t n_bounds, const ibp_kv_rows* q, uint32_t n_first, uint32_t n_last,
                  uint32_t n_select, int32_t* sel, void* workspace, uint64_t workspace_bytes,
                  void* stream) {
  const char* name = "ibp_kv_select";
  ibp::kv::Cache c;
  ibp::kv::Batch b;
  ibp::kv::Rows qr;
  int r;
  if ((r = check_cache(name, cache, false, &c)) || (r = check_batch(name, batch, c, true, true, &b)) ||
      (r = check_rows(name, "q", q, b.n_rows, c.head_dim, false, &qr)) ||
      (r = check_group(name, c, qr.n_heads)) || (r = check_items(name, b.n_rows, qr.n_heads)) ||
      (r = check_select(name, n_select)))
    return r;
  if (n_last == 0 || n_first > n_select || n_last > n_select - n_first)
    return set_error(IBP_ERR_SIZE, "%s: n_last >= 1 and n_first + n_last <= n_select are needed",
                     name);
  if (n_bounds > 0x7FFFFFFFull)
    return set_error(IBP_ERR_SIZE, "%s: n_bounds must be below 2^31", name);
  if ((n_bounds && !bounds) || (b.n_rows && !sel))
    return set_error(IBP_ERR_NULL, "%s: bounds and sel are required", name);
  if (!aligned(bounds, 16) || !aligned(sel, 4))
    return set_error(IBP_ERR_ALIGN, "%s: misaligned pointer", name);
  const uint64_t need = ibp::kv::select_workspace(c, b, n_select);
  if ((r = check_workspace(name, workspace, workspace_bytes, need))) return r;
  if ((r = require_device(name))) return r;
  hipError_t e = ibp::kv::launch_select(c, cache->dtype, b, bounds, (uint32_t)n_bounds, qr, n_first,
                                        n_last, n_select, sel, workspace, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int ibp_kv_select_workspace(const ibp_kv_cache* cache, const ibp_kv_batch* batch,
                            uint32_t n_select, uint64_t* bytes) {
  const char* name = "ibp_kv_select_workspace";
  if (!bytes) return set_error(IBP_ERR_NULL, "%s: bytes is required", name);
  ibp::kv::Cache c;
  ibp::kv::Batch b;
  int r;
  if ((r = check_cache(name, cache, false, &c)) || (r = check_batch(name, batch, c, false, true, &b)) ||
      (r = check_items(name, b.n_rows, c.n_heads)) || (r = check_select(name, n_select)))
    return r;
  *bytes = ibp::kv::select_workspace(c, b, n_select);
  return ibp::clear_error();
}

int ibp_kv_attend_selected(const ibp_kv_cache* cache, const ibp_kv_batch* batch,
                           const ibp_kv_rows* q, const ibp_kv_rows* out, const int32_t* sel,
                           uint32_t n_select, float scale, float* lse, void* workspace,
                           uint64_t workspace_bytes, void* stream) {
  const char* name = "ibp_kv_attend_selected";
  int r = check_select(name, n_select);
  if (r) return r;
  return attend(name, cache, batch, q, out, sel, n_select, scale, 0, true, lse, workspace,
                workspace_bytes, stream);
}

int ibp_kv_attend_selected_workspace(const ibp_kv_cache* cache, const ibp_kv_batch* batch,
                                     uint32_t n_q_heads, uint32_t n_select, uint64_t* bytes) {
  const char* name = "ibp_kv_attend_selected_workspace";
  int r = check_select(name, n_select);
  if (r) return r;
  return attend_workspace(name, cache, batch, n_q_heads, n_select, bytes);
}

}  // extern "C"
