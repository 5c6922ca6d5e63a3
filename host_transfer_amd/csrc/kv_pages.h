// kv_pages.h -- what the pages' assignment (kv_pages.hip) and its C ABI (api_kv_pages.hip) share.
#pragma once

#include "ibp_kv_pages.h"
#include "kv.h"

namespace ibp {
namespace kv {

struct PagePool {
  int32_t *table, *free_pages;
  uint64_t table_stride;
  uint32_t n_pages, max_pages;
  FastDiv page;
};

struct Step {
  const int32_t *had, *keep, *add, *free_count;
  uint32_t n_rows, n_seqs;
};

uint64_t assign_workspace(uint32_t n_seqs, uint64_t n_rows);
hipError_t launch_assign(const PagePool& pool, const Step& step, const ibp_kv_assigned& out,
                         void* workspace, hipStream_t s);

}  // namespace kv
}  // namespace ibp
