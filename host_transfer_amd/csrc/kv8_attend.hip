// kv8_attend.hip -- attention over a paged cache in 8 bits: how a call is run.
#include "kv8_attend.h"

namespace ibp {
namespace kv {

namespace {

// Planned as over a cache in 16 bits (kv_attend.hip).
Cache geometry(const Cache8& c) {
  Cache g = {};
  g.n_pages = c.n_pages;
  g.n_heads = c.n_heads;
  g.head_dim = c.head_dim;
  g.page = c.page;
  return g;
}

}  // namespace

hipError_t attend8_workspace(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint64_t* bytes) {
  AttendPlan p;
  const Cache g = geometry(c);
  hipError_t e = make_plan(g, b, n_q_heads, 0, 0, &p);
  if (e == hipSuccess) *bytes = partial_bytes(g, b, n_q_heads, p);
  return e;
}

hipError_t launch_attend8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q, const Rows& out,
                          float scale, uint32_t window, bool causal, float* lse, void* workspace,
                          hipStream_t s) {
  AttendPlan p;
  hipError_t e = make_plan(geometry(c), b, q.n_heads, 0, window, &p);
  if (e != hipSuccess) return e;
  Partial part;
  part.splits = p.splits;
  part.head_dim = c.head_dim;
  part.o = (float*)workspace;
  part.ms = (float2*)(part.o + (uint64_t)b.n_rows * q.n_heads * p.splits * c.head_dim);
  e = p.few ? launch_decode8(p, c, dtype, b, q, out, scale, window, causal, lse, part, s)
            : launch_chunk8(p, c, dtype, b, q, out, scale, window, causal, lse, part, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join(dtype, b, out, part, lse, s);
}

}  // namespace kv
}  // namespace ibp
