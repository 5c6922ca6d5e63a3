// api_kv_pages.hip -- the extern "C" entry points of include/ibp_kv_pages.h: argument checks before
// any HIP call, then the launcher of kv_pages.hip.
#include "kv_check.h"
#include "kv_pages.h"

using ibp::set_error;
using namespace ibp::kv::check;

namespace {

int check_sizes(const char* name, uint32_t n_seqs, uint64_t n_rows) {
  if (n_seqs > IBP_KV_MAX_REQUESTS || n_rows > 0x7FFFFFFFull)
    return set_error(IBP_ERR_SIZE, "%s: n_seqs must be at most %u, n_rows below 2^31", name,
                     IBP_KV_MAX_REQUESTS);
  return IBP_OK;
}

struct Range {
  const void* p;
  uint64_t bytes;
  bool written;
};

}  // namespace

extern "C" {

int ibp_kv_assign(const ibp_kv_page_pool* pool, const ibp_kv_step* step, const ibp_kv_assigned* out,
                  void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* name = "ibp_kv_assign";
  if (!pool || !step || !out)
    return set_error(IBP_ERR_NULL, "%s: pool, step and out are required", name);
  int r;
  if ((r = check_sizes(name, step->n_seqs, step->n_rows))) return r;
  if (pool->page_tokens == 0 || pool->page_tokens > IBP_KV_MAX_PAGE_TOKENS)
    return set_error(IBP_ERR_SIZE, "%s: page_tokens %u must be in [1, %u]", name, pool->page_tokens,
                     IBP_KV_MAX_PAGE_TOKENS);
  if (pool->n_pages == 0 || pool->n_pages > 0x7FFFFFFFull)
    return set_error(IBP_ERR_SIZE, "%s: n_pages %llu must be in [1, 2^31)", name,
                     (unsigned long long)pool->n_pages);
  if (pool->max_pages > 0x7FFFFFFFu || pool->table_stride > (1ull << 31))
    return set_error(IBP_ERR_SIZE, "%s: max_pages and table_stride must be below 2^31", name);
  if (step->n_seqs > 1 && pool->table_stride < pool->max_pages)
    return set_error(IBP_ERR_SIZE, "%s: table_stride %llu is below max_pages %u", name,
                     (unsigned long long)pool->table_stride, pool->max_pages);
  const uint64_t n = step->n_seqs;
  if (!pool->free_pages || !step->free_count || !out->q_start || !out->free_count ||
      (n && pool->max_pages && !pool->page_table) ||
      (n && (!step->had || !step->add || !out->kv_len || !out->length)) || (step->n_rows && !out->slots))
    return set_error(IBP_ERR_NULL, "%s: a required array is NULL", name);
  if (!aligned(pool->page_table, 4) || !aligned(pool->free_pages, 4) || !aligned(step->had, 4) ||
      !aligned(step->keep, 4) || !aligned(step->add, 4) || !aligned(step->free_count, 4) ||
      !aligned(out->q_start, 4) || !aligned(out->kv_len, 4) || !aligned(out->length, 4) ||
      !aligned(out->free_count, 4) || !aligned(out->unserved, 4) || !aligned(out->slots, 8) ||
      !aligned(out->positions, 8))
    return set_error(IBP_ERR_ALIGN, "%s: misaligned array", name);
  const uint64_t table = n ? ((n - 1) * pool->table_stride + pool->max_pages) * 4 : 0;
  const Range ranges[] = {{pool->page_table, table, true},
                          {pool->free_pages, pool->n_pages * 4, true},
                          {step->had, n * 4, false},
                          {step->keep, n * 4, false},
                          {step->add, n * 4, false},
                          {step->free_count, 4, false},
                          {out->q_start, n * 4 + 4, true},
                          {out->kv_len, n * 4, true},
                          {out->length, n * 4, true},
                          {out->free_count, 4, true},
                          {out->unserved, 4, true},
                          {out->slots, step->n_rows * 8, true},
                          {out->positions, step->n_rows * 8, true}};
  constexpr int kRanges = sizeof ranges / sizeof *ranges;
  for (int i = 0; i < kRanges; ++i)
    for (int j = i + 1; j < kRanges; ++j) {
      const Range &a = ranges[i], &b = ranges[j];
      if ((!a.written && !b.written) || !a.p || !b.p || a.bytes == 0 || b.bytes == 0) continue;
      if (a.p == b.p && ((a.p == step->had && i == 2 && j == 8) || (i == 5 && j == 9))) continue;
      const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
      if (x < y ? y - x < a.bytes : x - y < b.bytes)
        return set_error(IBP_ERR_SIZE, "%s: two of the arrays overlap", name);
    }
  if ((r = check_workspace(name, workspace, workspace_bytes,
                           ibp::kv::assign_workspace(step->n_seqs, step->n_rows))) ||
      (r = require_device(name)))
    return r;
  const ibp::kv::PagePool p = {pool->page_table, pool->free_pages, pool->table_stride,
                               (uint32_t)pool->n_pages, pool->max_pages, ibp::kv::fast_div(pool->page_tokens)};
  const ibp::kv::Step st = {step->had, step->keep, step->add, step->free_count, (uint32_t)step->n_rows,
                            step->n_seqs};
  hipError_t e = ibp::kv::launch_assign(p, st, *out, workspace, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, name);
  return ibp::clear_error();
}

int ibp_kv_assign_workspace(uint32_t n_seqs, uint64_t n_rows, uint64_t* bytes) {
  const char* name = "ibp_kv_assign_workspace";
  if (!bytes) return set_error(IBP_ERR_NULL, "%s: bytes is required", name);
  int r = check_sizes(name, n_seqs, n_rows);
  if (r) return r;
  *bytes = ibp::kv::assign_workspace(n_seqs, n_rows);
  return ibp::clear_error();
}

}  // extern "C"
