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

bool few_rows(const Cache8& c, const Batch& b, uint32_t n_q_heads) {
  return (uint64_t)b.max_q * (n_q_heads / c.n_heads) <= 32;
}

// Few rows.  The keys of up to kMaxShared sequences are shared out by their lengths, over as many
// workgroups as the GPU runs at a time (a few more make a second, nearly empty round: 20 sequences of 40
// heads over 2,048 tokens 87 us with 1,000 workgroups for 1,024 places, 96 with 1,200), or two for each
// sequence if these are more; not where sequences alone fill the GPU.
hipError_t plan8(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint32_t window, Plan8* p) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  *p = Plan8{};
  p->rows = b.max_q * (n_q_heads / c.n_heads);
  p->head_group = c.n_heads % 4 == 0 ? 4 : 1;
  p->places = b.n_seqs;
  const uint64_t head_blocks = c.n_heads / p->head_group;
  const uint64_t at_once = di.cus * decode8_groups(c.head_dim, p->rows > 16 ? 2 : 1) / head_blocks;
  uint64_t keys = b.max_kv;
  if (window && keys > (uint64_t)window + b.max_q) keys = (uint64_t)window + b.max_q;
  const uint64_t tiles = (keys + 31) / 32;
  if (b.n_seqs && b.n_seqs <= kMaxShared && b.n_seqs < at_once && tiles > 4 &&
      b.n_seqs * tiles < (1u << 31)) {  // (all sequences' tiles are summed in 32 bits)
    uint64_t shares = at_once > 2 * (uint64_t)b.n_seqs ? at_once : 2 * (uint64_t)b.n_seqs;
    if (shares > b.n_seqs * tiles) shares = b.n_seqs * tiles;
    if (shares > kMaxSplits) shares = kMaxSplits;
    p->shares = p->places = (uint32_t)shares;
    // (a launch's threads are counted in 32 bits)
    p->wide_join = shares > 32 * (uint64_t)b.n_seqs && tiles > 32 && (uint64_t)b.n_rows * n_q_heads <= 0x3FFFFFull;
  } else if (tiles <= 4 && (uint64_t)b.n_seqs * c.n_heads <= (uint64_t)di.cus * 4) {
    p->head_group = 1;  // a tile to each wave, none waits for another's
  }
  return (uint64_t)p->places * (c.n_heads / p->head_group) > 0xFFFFFFull ? hipErrorInvalidConfiguration : hipSuccess;
}

// Many rows, as over a cache in 16 bits but for the splits: as many as fill the workgroups that the GPU runs at a
// time in whole rounds (7 sequences of one row tile and 2 heads over up to 91,718 tokens: 126 us with 37 splits, whose
// 518 workgroups are six too many, 90 with 36).
hipError_t plan_chunk8(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint32_t window, AttendPlan* p) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e == hipSuccess) e = make_plan(geometry(c), b, n_q_heads, 0, window, p);
  if (e != hipSuccess || p->splits <= 1) return e;
  const uint64_t base = p->blocks / p->splits, places = (uint64_t)di.cus * (c.head_dim <= 128 ? 2 : 1);
  uint64_t splits = 1, full = 0;  // of a round's places, in 1024ths
  for (uint64_t round = (base + places - 1) / places, i = 0; i < 3 && full < 800; ++i, ++round) {
    uint64_t n = round * places / base;
    if (n > p->splits) n = p->splits;
    const uint64_t f = n * base * 1024 / (round * places);
    if (f > full + (i ? 64 : 0)) {
      splits = n;
      full = f;
    }
  }
  p->splits = (uint32_t)splits;
  p->blocks = base * splits;
  return e;
}

constexpr uint64_t kHeadBytes = (uint64_t)kMaxShared * sizeof(int2);

uint64_t plan8_bytes(const Cache8& c, const Plan8& p) {
  return p.shares ? kHeadBytes + (uint64_t)p.places * c.n_heads * p.rows * (c.head_dim + 2) * 4 : 0;
}

}  // namespace

hipError_t attend8_workspace(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint64_t* bytes) {
  if (few_rows(c, b, n_q_heads)) {
    Plan8 p;
    hipError_t e = plan8(c, b, n_q_heads, 0, &p);  // (a window asks for no more of it)
    if (e == hipSuccess) *bytes = plan8_bytes(c, p);
    return e;
  }
  AttendPlan p;  // (as many splits as it could be, a window asks for no more)
  hipError_t e = make_plan(geometry(c), b, n_q_heads, 0, 0, &p);
  if (e == hipSuccess) *bytes = partial_bytes(geometry(c), b, n_q_heads, p);
  return e;
}

hipError_t launch_attend8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q, const Rows& out,
                          float scale, uint32_t window, bool causal, float* lse, void* workspace,
                          hipStream_t s) {
  if (few_rows(c, b, q.n_heads)) {
    Plan8 p;
    hipError_t e = plan8(c, b, q.n_heads, window, &p);
    if (e != hipSuccess) return e;
    p.heads = (int2*)workspace;
    p.o = (float*)((char*)workspace + kHeadBytes);
    p.ms = (float2*)(p.o + (uint64_t)p.places * c.n_heads * p.rows * c.head_dim);
    return launch_decode8(p, c, dtype, b, q, out, scale, window, causal, lse, s);
  }
  AttendPlan p;
  hipError_t e = plan_chunk8(c, b, q.n_heads, window, &p);
  if (e != hipSuccess) return e;
  Partial part;
  part.splits = p.splits;
  part.head_dim = c.head_dim;
  part.o = (float*)workspace;
  part.ms = (float2*)(part.o + (uint64_t)b.n_rows * q.n_heads * p.splits * c.head_dim);
  e = launch_chunk8(p, c, dtype, b, q, out, scale, window, causal, lse, part, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join(dtype, b, out, part, lse, s);
}

}  // namespace kv
}  // namespace ibp
