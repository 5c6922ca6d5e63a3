// kv8_attend.h -- how attention over a cache in 8 bits is run, and its launchers.
#pragma once

#include "kv8.h"

namespace ibp {
namespace kv {

// Workgroups of k_kv8_decode that a CU runs at a time, by its registers (columns of 16 rows).  Measured with heads
// of 128; those of up to 64 are run as these, though their registers leave room for five and three.
constexpr uint32_t decode8_groups(uint32_t head_dim, uint32_t columns) {
  return head_dim <= 128 ? (columns == 1 ? 4 : 2) : (columns == 1 ? 2 : 1);
}
hipError_t launch_decode8(const Plan8& p, const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q,
                          const Rows& out, float scale, uint32_t window, bool causal, float* lse,
                          hipStream_t s);
hipError_t launch_chunk8(const AttendPlan& p, const Plan8& plan, const Cache8& c, uint32_t dtype, const Batch& b,
                         const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                         float* lse, hipStream_t s);
// Split rows' results together, where keys were shared out.
hipError_t launch_join8(const Plan8& p, const Cache8& c, uint32_t dtype, const Batch& b, const Rows& out, float* lse,
                        hipStream_t s);

}  // namespace kv
}  // namespace ibp
