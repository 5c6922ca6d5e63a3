// kv8_attend.h -- launchers of attention over a cache in 8 bits.
#pragma once

#include "kv8.h"

namespace ibp {
namespace kv {

hipError_t launch_decode8(const AttendPlan& p, const Cache8& c, uint32_t dtype, const Batch& b,
                          const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                          float* lse, Partial part, hipStream_t s);
hipError_t launch_chunk8(const AttendPlan& p, const Cache8& c, uint32_t dtype, const Batch& b,
                         const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                         float* lse, Partial part, hipStream_t s);

}  // namespace kv
}  // namespace ibp
