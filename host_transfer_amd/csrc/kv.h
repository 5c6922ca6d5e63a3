// kv.h -- what the paged K/V kernels and their C ABI (api_kv.hip) share:
// device views of the caller's structs, launchers, small device helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ibp_internal.h"
#include "ibp_kv.h"

namespace ibp {

// Sets this thread's ibp_last_error() text and returns `code` (api.hip).
int set_error(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int clear_error();

namespace kv {

// n / d for n < 2^31 by a multiplication: with l = ceil(log2 d) and m =
// ceil(2^(31+l) / d), n*m >> (31+l) is exact, since m*d exceeds 2^(31+l) by
// less than d <= 2^l (Granlund and Montgomery, "Division by invariant integers
// using multiplication", PLDI 1994, theorem 4.2).  m < 2^32 for d < 2^31.
struct FastDiv {
  uint32_t d, m, l;
  __host__ __device__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)(n << 1) * m) >> 32) >> l;
  }
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return FastDiv{d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), l};
}

// The cache, its strides in elements.
struct Cache {
  uint16_t *k, *v;
  uint64_t page_stride, token_stride;
  uint32_t head_stride, n_pages, n_heads, head_dim;
  FastDiv page;
};

struct Rows {
  uint16_t* p;
  uint64_t token_stride;
  uint32_t head_stride, n_heads;
};

struct Batch {
  const int32_t *q_start, *kv_len, *table;
  uint64_t table_stride;
  uint32_t n_rows, n_seqs, max_q, max_kv, max_pages;
};

// One sequence of a batch, clamped to the buffers: rows [row0, row0 + q_len),
// row row0 + i at position first + i; n_keys tokens can be read.
struct Seq {
  int32_t row0, q_len, first, n_keys;
};
__device__ __forceinline__ Seq load_seq(const Batch& b, uint32_t s) {
  Seq r;
  const int32_t n_rows = (int32_t)b.n_rows;
  const int32_t a = b.q_start[s], e = b.q_start[s + 1];
  const int32_t kv = max(b.kv_len[s], 0);
  r.row0 = min(max(a, 0), n_rows);
  const int32_t end = min(max(e, r.row0), n_rows);
  r.first = kv - (e - r.row0);
  r.q_len = min(end - r.row0, (int32_t)b.max_q);
  r.n_keys = min(kv, (int32_t)b.max_kv);
  return r;
}

// The sequence that row r belongs to: the last s with q_start[s] <= r, if r
// is below q_start[s + 1] and among the first max_q; -1 if there is none.
__device__ __forceinline__ int32_t seq_of_row(const Batch& b, int32_t r) {
  int32_t lo = 0, hi = (int32_t)b.n_seqs;  // q_start[lo] <= r < q_start[hi], as far as known
  if (hi == 0 || b.q_start[0] > r) return -1;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (b.q_start[mid] <= r) lo = mid;
    else hi = mid;
  }
  if (r >= b.q_start[lo + 1] || r - max(b.q_start[lo], 0) >= (int32_t)b.max_q) return -1;
  return lo;
}

__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }

template <typename T>
struct Vec8 {
  typedef T type __attribute__((ext_vector_type(8)));
};

hipError_t launch_append(const Cache& c, uint32_t dtype, const Rows& k, const Rows& v,
                         const Rows& q, const Rows& q_out, const int64_t* slots,
                         const int64_t* positions, uint32_t n_tokens, const float* rope,
                         uint64_t n_positions, uint32_t rope_dim, bool interleaved,
                         const void* q_norm, const void* k_norm, float eps, hipStream_t s);

hipError_t launch_page_bounds(const Cache& c, uint32_t dtype, const Batch& b, void* bounds,
                              hipStream_t s);

uint64_t select_workspace(const Cache& c, const Batch& b, uint32_t n_select);
hipError_t launch_select(const Cache& c, uint32_t dtype, const Batch& b, const void* bounds,
                         uint32_t n_bounds, const Rows& q, uint32_t n_first, uint32_t n_last,
                         uint32_t n_select, int32_t* sel, void* workspace, hipStream_t s);

// sel == nullptr: over each sequence's whole cache; else over the selected pages.
hipError_t attend_workspace(const Cache& c, const Batch& b, uint32_t n_q_heads, uint32_t n_select,
                            uint64_t* bytes);
hipError_t launch_attend(const Cache& c, uint32_t dtype, const Batch& b, const Rows& q,
                         const Rows& out, const int32_t* sel, uint32_t n_select, float scale,
                         uint32_t window, bool causal, float* lse, void* workspace,
                         hipStream_t s);

}  // namespace kv
}  // namespace ibp
