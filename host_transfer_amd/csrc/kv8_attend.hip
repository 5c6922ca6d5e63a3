// kv8_attend.hip -- attention over a paged cache in 8 bits: how a call is run.
#include "kv8_attend.h"

namespace ibp {
namespace kv {

namespace {

// What the plan over a cache in 16 bits (kv_attend.hip) asks of one.
Cache geometry(const Cache8& c) {
  Cache g = {};
  g.n_pages = c.n_pages;
  g.n_heads = c.n_heads;
  g.head_dim = c.head_dim;
  g.page = c.page;
  return g;
}

// As over a cache in 16 bits, but for:
//   columns  up to 32 rows that share their keys (drafted tokens with their group of heads) are few: in
//            two columns of 16 (24 sequences of 20 such rows over up to 8,192 tokens 89 us as chunks).
//   splits   as many workgroups as the GPU runs at a time, rather than a few more: 20 sequences
//            of 40 heads over 2,048 tokens 87 us with 5 splits (1,000 workgroups for 1,024 places), 96 with
//            6, 91 with 11; 131,072-token contexts 151 us with 128, 162 with 256.  Where that leaves
//            more than a quarter of the places empty, as many as two or three such rounds hold,
//            if these are fuller.
hipError_t plan8(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint32_t window, AttendPlan* p,
                 uint32_t* columns) {
  hipError_t e = make_plan(geometry(c), b, n_q_heads, 0, window, p);
  const uint64_t rows = (uint64_t)b.max_q * (n_q_heads / c.n_heads);
  *columns = rows <= 16 ? 1 : 2;
  if (e != hipSuccess || rows > 32) return e;
  DeviceInfo di;
  if ((e = device_info(&di)) != hipSuccess) return e;
  p->few = true;
  p->by_length = false;
  p->row_tiles = 1;
  p->heads = c.n_heads % 4 == 0 ? 4 : 1;
  const uint64_t base = (uint64_t)b.n_seqs * (c.n_heads / p->heads);
  const uint64_t places = (uint64_t)di.cus * decode8_groups(c.head_dim, *columns);
  uint64_t keys = b.max_kv;
  if (window && keys > (uint64_t)window + b.max_q) keys = (uint64_t)window + b.max_q;
  uint64_t most = keys / (256 / p->heads);  // keys that are worth a split
  if (most > kMaxSplits) most = kMaxSplits;
  if (most < 1) most = 1;
  uint64_t splits = 1, full = 0;  // of a round's places, in 1024ths
  for (uint64_t round = base ? (base + places - 1) / places : 1, i = 0; i < 3 && full < 768; ++i, ++round) {
    uint64_t n = base ? round * places / base : 1;
    if (n > most) n = most;
    const uint64_t f = n * base * 1024 / (round * places);
    if (f > full + (i ? 64 : 0)) {
      splits = n;
      full = f;
    }
  }
  p->splits = (uint32_t)splits;
  p->blocks = base * splits;
  const uint64_t units = (uint64_t)b.n_rows * n_q_heads;
  return p->blocks > 0xFFFFFFull || (p->splits > 64 && units > 0x3FFFFFull)
             ? hipErrorInvalidConfiguration : hipSuccess;
}

}  // namespace

// (Sized without a window, which asks for no more splits.)
hipError_t attend8_workspace(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint64_t* bytes) {
  AttendPlan p;
  uint32_t columns;
  hipError_t e = plan8(c, b, n_q_heads, 0, &p, &columns);
  if (e == hipSuccess) *bytes = partial_bytes(geometry(c), b, n_q_heads, p);
  return e;
}

hipError_t launch_attend8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q, const Rows& out,
                          float scale, uint32_t window, bool causal, float* lse, void* workspace,
                          hipStream_t s) {
  AttendPlan p;
  uint32_t columns;
  hipError_t e = plan8(c, b, q.n_heads, window, &p, &columns);
  if (e != hipSuccess) return e;
  Partial part;
  part.splits = p.splits;
  part.head_dim = c.head_dim;
  part.o = (float*)workspace;
  part.ms = (float2*)(part.o + (uint64_t)b.n_rows * q.n_heads * p.splits * c.head_dim);
  e = p.few ? launch_decode8(p, columns, c, dtype, b, q, out, scale, window, causal, lse, part, s)
            : launch_chunk8(p, c, dtype, b, q, out, scale, window, causal, lse, part, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join(dtype, b, out, part, lse, s);
}

}  // namespace kv
}  // namespace ibp
