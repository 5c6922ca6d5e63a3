// kv8_attend.hip -- attention over a paged cache in 8 bits: how a call is run.
#include "kv8_attend.h"

namespace ibp {
namespace kv {

namespace {

bool few_rows(const Cache8& c, const Batch& b, uint32_t n_q_heads) {
  return (uint64_t)b.max_q * (n_q_heads / c.n_heads) <= 32;
}

// A workgroup of 1024 to each row's join, not a wave: few rows of many splits.
bool wide_join(const DeviceInfo& di, const Cache8& c, const Batch& b, const Plan8& p) {
  return p.row_tiles == 1 && p.shares > 32 * (uint64_t)b.n_seqs &&
         (uint64_t)b.n_seqs * c.n_heads * p.rows <= (uint64_t)di.cus * 2;
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
  p->row_tiles = 1;
  p->head_group = c.n_heads % 4 == 0 ? 4 : 1;
  p->places = b.n_seqs;
  const uint64_t head_blocks = c.n_heads / p->head_group;
  const uint64_t at_once = di.cus * decode8_groups(c.head_dim, p->rows > 16 ? 2 : 1) / head_blocks;
  uint64_t keys = b.max_kv;
  if (window && keys > (uint64_t)window + b.max_q) keys = (uint64_t)window + b.max_q;
  const uint64_t tiles = (keys + 31) / 32;
  // (all sequences' tiles are summed in 32 bits; without the window, as a call with one has no larger workspace)
  if (b.n_seqs && b.n_seqs <= kMaxShared && b.n_seqs < at_once && tiles > 4 &&
      b.n_seqs * (((uint64_t)b.max_kv + 31) / 32) < (1u << 31)) {
    uint64_t shares = at_once > 2 * (uint64_t)b.n_seqs ? at_once : 2 * (uint64_t)b.n_seqs;
    if (shares > b.n_seqs * tiles) shares = b.n_seqs * tiles;
    if (shares > kMaxSplits) shares = kMaxSplits;
    p->shares = p->places = (uint32_t)shares;
    p->wide_join = wide_join(di, c, b, *p) && tiles > 32;
  } else if (tiles <= 4 && (uint64_t)b.n_seqs * c.n_heads <= (uint64_t)di.cus * 4) {
    p->head_group = 1;  // a tile to each wave, none waits for another's
  }
  return (uint64_t)p->places * (c.n_heads / p->head_group) > 0xFFFFFFull ? hipErrorInvalidConfiguration : hipSuccess;
}

// Many rows, as over a cache in 16 bits (kv_attend.hip) but for the splits: where the row tiles leave places among
// the workgroups that the GPU runs at a time, the keys of all tiles are shared out over these by their lengths,
// which differ between sequences.  Equal numbers of splits for all tiles took: 24 sequences of 5 to 9 rows for 8 heads each over
// 1,638 to 8,192 tokens 123 us (94 so), 3 chunks of up to 300 over 2,000 to 20,000 265 (198), 2 of up to 256 over
// up to 30,000 215 (189); where the lengths are equal, one chunk of 1,024 over 4,096 tokens, 92 (96: each
// workgroup's look at all lengths).  More rounds of workgroups, where the tiles leave no places: chunks of up to
// 511 over 9,001 tokens 315 us, 264 with a workgroup a tile.  33 to 64 rows as four columns of k_kv8_decode
// instead: 124 and 131 us for the first, 140 for 7 sequences over 91,718 tokens that take 92.
hipError_t plan_chunk8(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint32_t window, AttendPlan* p,
                       Plan8* plan) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  *plan = Plan8{};
  *p = AttendPlan{};
  const uint32_t group = n_q_heads / c.n_heads;
  p->row_tiles = (uint32_t)(((uint64_t)b.max_q * group + kChunkRows - 1) / kChunkRows);
  p->by_length = longest_first(b);
  const uint64_t items = (uint64_t)b.n_seqs * p->row_tiles;
  const uint64_t at_once = di.cus * (c.head_dim <= 128 ? 2 : 1) / c.n_heads;
  const uint64_t by_rows = b.n_seqs + (uint64_t)b.n_rows * group / kChunkRows;
  const uint64_t active = items < by_rows ? items : by_rows;  // (more have no rows)
  uint64_t keys = b.max_kv;
  if (window && keys > (uint64_t)window + b.max_q) keys = (uint64_t)window + b.max_q;
  const uint64_t steps = (keys + 63) / 64 + 1;
  p->blocks = items * c.n_heads;
  if (items && items <= kMaxShared && active < at_once && steps >= 2 * kLeastSteps &&
      items * (((uint64_t)b.max_kv + 63) / 64 + 1) < (1u << 31)) {  // (as above)
    uint64_t shares = active * (steps / kLeastSteps);
    if (shares > at_once) shares = at_once;
    if (shares > kMaxSplits) shares = kMaxSplits;
    plan->shares = plan->places = (uint32_t)shares;
    plan->row_tiles = p->row_tiles;
    plan->rows = p->row_tiles > 1 ? kChunkRows : b.max_q * group;
    plan->wide_join = wide_join(di, c, b, *plan);
    p->blocks = shares * c.n_heads;
  }
  return p->blocks > 0xFFFFFFull ? hipErrorInvalidConfiguration : hipSuccess;
}

constexpr uint64_t kHeadBytes = (uint64_t)(kMaxShared + kMaxSplits) * sizeof(int2);

uint64_t plan8_bytes(const Cache8& c, const Plan8& p) {
  return p.shares ? kHeadBytes + (uint64_t)p.places * c.n_heads * p.rows * (c.head_dim + 2) * 4 : 0;
}
void place_in(void* workspace, const Cache8& c, Plan8* p) {
  if (!p->shares) return;
  p->heads = (int2*)workspace;
  p->firsts = p->heads + kMaxShared;
  p->o = (float*)((char*)workspace + kHeadBytes);
  p->ms = (float2*)(p->o + (uint64_t)p->places * c.n_heads * p->rows * c.head_dim);
}

}  // namespace

hipError_t attend8_workspace(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint64_t* bytes) {
  if (few_rows(c, b, n_q_heads)) {
    Plan8 p;
    hipError_t e = plan8(c, b, n_q_heads, 0, &p);  // (a window asks for no more of it)
    if (e == hipSuccess) *bytes = plan8_bytes(c, p);
    return e;
  }
  AttendPlan p;
  Plan8 plan;
  hipError_t e = plan_chunk8(c, b, n_q_heads, 0, &p, &plan);
  if (e == hipSuccess) *bytes = plan8_bytes(c, plan);
  return e;
}

hipError_t launch_attend8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q, const Rows& out,
                          float scale, uint32_t window, bool causal, float* lse, void* workspace,
                          hipStream_t s) {
  if (few_rows(c, b, q.n_heads)) {
    Plan8 p;
    hipError_t e = plan8(c, b, q.n_heads, window, &p);
    if (e != hipSuccess) return e;
    place_in(workspace, c, &p);
    return launch_decode8(p, c, dtype, b, q, out, scale, window, causal, lse, s);
  }
  AttendPlan p;
  Plan8 plan;
  hipError_t e = plan_chunk8(c, b, q.n_heads, window, &p, &plan);
  if (e != hipSuccess) return e;
  place_in(workspace, c, &plan);
  e = launch_chunk8(p, plan, c, dtype, b, q, out, scale, window, causal, lse, s);
  return e != hipSuccess || plan.shares == 0 ? e : launch_join8(plan, c, dtype, b, out, lse, s);
}

}  // namespace kv
}  // namespace ibp
