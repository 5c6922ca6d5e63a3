// kv_attend.hip -- attention over a paged cache, whole or over selected pages.
#include "ibp_device.h"
#include "kv_mfma.h"

namespace ibp {
namespace kv {

namespace {

// How a call is run.
//   few    Up to 16 rows share a sequence's keys (one new token, or a few, with its group of
//          heads), or each row has its own list of pages.
//   heads  Four key heads to a workgroup where their number allows: its waves then read
//          neighbouring parts of the same token rows (OPT-13B decode 172 -> 162 us), instead of
//          different keys of one head.
//   splits The keys of a row tile over several workgroups until the GPU has eight a CU (few:
//          more than it runs at a time, so that the last ones to finish are short; 4 a CU took
//          175 / 340 us, 8 172 / 314, 12 166 / 320 for OPT-13B decode / 131072-token contexts)
//          or two (many rows: as many as it runs; more only add partial results to write and
//          join, 2048 tokens of 32 heads 62 us with two, 74 with four), but no split below 256
//          keys of a wave's turn (few) or 512.
//   order  Where contexts are as long again as the chunks or longer, up to 64 sequences: the longest
//          sequence's tiles first (k_kv_chunk; chunks of up to 511 over 9,001 to 2,701 tokens 280
//          -> 250 us), else each sequence's last tiles first.
// A window bounds the keys of a tile; the workspace is sized without one, for as many splits or
// more.
hipError_t make_plan(const Cache& c, const Batch& b, uint32_t n_q_heads, uint32_t n_select,
                     uint32_t window, AttendPlan* p) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  const uint32_t group = n_q_heads / c.n_heads;
  const uint64_t rows = (uint64_t)(n_select ? 1 : b.max_q) * group;
  p->few = n_select || rows <= 16;
  const uint64_t tile = p->few ? 16 : kChunkRows;
  p->row_tiles = (uint32_t)((rows + tile - 1) / tile);
  p->heads = p->few && !n_select && c.n_heads % 4 == 0 ? 4 : 1;
  const uint64_t base = (uint64_t)(n_select ? b.n_rows : b.n_seqs) * p->row_tiles * (c.n_heads / p->heads);
  uint64_t keys = n_select ? (uint64_t)n_select * c.page.d : b.max_kv;
  if (window && keys > (uint64_t)window + b.max_q) keys = (uint64_t)window + b.max_q;
  const uint64_t want = (uint64_t)di.cus * (p->few ? 8 : 2);
  uint64_t splits = base ? (want + base - 1) / base : 1;
  const uint64_t least = p->few ? 256 / p->heads : 512;  // keys that are worth a split
  if (splits > keys / least) splits = keys / least;
  if (splits > kMaxSplits) splits = kMaxSplits;
  p->splits = splits < 1 ? 1 : (uint32_t)splits;
  p->blocks = base * p->splits;
  p->by_length = !p->few && longest_first(b);
  // a launch's threads are counted in 32 bits: 256 a workgroup, up to 1024 a row where many
  // splits are joined
  const uint64_t units = (uint64_t)b.n_rows * n_q_heads;
  return p->blocks > 0xFFFFFFull || (p->splits > 64 && units > 0x3FFFFFull)
             ? hipErrorInvalidConfiguration : hipSuccess;
}

// The workspace: [unit][split][head_dim] floats, then [unit][split] (max, sum).
uint64_t partial_bytes(const Cache& c, const Batch& b, uint32_t n_q_heads, const AttendPlan& p) {
  if (p.splits == 1) return 0;
  return (uint64_t)b.n_rows * n_q_heads * p.splits * (c.head_dim + 2) * 4;
}

}  // namespace

hipError_t attend_workspace(const Cache& c, const Batch& b, uint32_t n_q_heads, uint32_t n_select,
                            uint64_t* bytes) {
  AttendPlan p;
  hipError_t e = make_plan(c, b, n_q_heads, n_select, 0, &p);
  if (e == hipSuccess) *bytes = partial_bytes(c, b, n_q_heads, p);
  return e;
}

hipError_t launch_attend(const Cache& c, uint32_t dtype, const Batch& b, const Rows& q,
                         const Rows& out, const int32_t* sel, uint32_t n_select, float scale,
                         uint32_t window, bool causal, float* lse, void* workspace,
                         hipStream_t s) {
  AttendPlan p;
  hipError_t e = make_plan(c, b, q.n_heads, n_select, window, &p);
  if (e != hipSuccess) return e;
  Partial part;
  part.splits = p.splits;
  part.head_dim = c.head_dim;
  part.o = (float*)workspace;
  part.ms = (float2*)(part.o + (uint64_t)b.n_rows * q.n_heads * p.splits * c.head_dim);
  e = p.few ? launch_decode(p, c, dtype, b, q, out, sel, n_select, scale, window, causal, lse, part, s)
            : launch_chunk(p, c, dtype, b, q, out, scale, window, causal, lse, part, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join(dtype, b, out, part, lse, s);
}

}  // namespace kv
}  // namespace ibp
