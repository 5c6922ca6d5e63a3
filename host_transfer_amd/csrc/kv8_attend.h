// kv8_attend.h -- how attention over a cache in 8 bits is run, and its launchers.
#pragma once

#include "kv8.h"

namespace ibp {
namespace kv {

// Workgroups of k_kv8_decode that a CU runs at a time, by its registers (columns of 16 rows).
constexpr uint32_t decode8_groups(uint32_t head_dim, uint32_t columns) {
  return head_dim <= 128 ? (columns == 1 ? 4 : 2) : (columns == 1 ? 2 : 1);
}
constexpr uint32_t kMaxShared = 1024;  // sequences whose keys are split over workgroups

// Few rows: up to 32 that share a key head.  A head group (one key head or four) has `places` workgroups:
// one for each sequence (shares 0), or `shares` that the sequences' keys are split over by their
// lengths, which the kernel reads.  A split sequence's results are in the workspace:
// heads[sequence] = (its first place, its splits), o float[place][key head][row][head_dim], ms
// float2[place][key head][row] of (base, sum).
struct Plan8 {
  uint32_t shares, places, rows, head_group;
  bool wide_join;
  int2* heads;
  float* o;
  float2* ms;
};

hipError_t launch_decode8(const Plan8& p, const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q,
                          const Rows& out, float scale, uint32_t window, bool causal, float* lse,
                          hipStream_t s);
hipError_t launch_chunk8(const AttendPlan& p, const Cache8& c, uint32_t dtype, const Batch& b,
                         const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                         float* lse, Partial part, hipStream_t s);

}  // namespace kv
}  // namespace ibp
