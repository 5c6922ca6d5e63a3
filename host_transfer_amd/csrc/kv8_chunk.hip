// kv8_chunk.hip -- attention of a chunk of new tokens over a cache in 8 bits.
#include "kv8_attend.h"
#include "kv_chunk.h"

namespace ibp {
namespace kv {

namespace {

template <typename T, int DP, bool kExact>
hipError_t run_chunk8(const AttendPlan& p, const Shared8& c, const Batch& b, const Rows& q,
                      const Rows& out, float scale, uint32_t window, bool causal, float* lse,
                      hipStream_t s) {
  hipLaunchKernelGGL((k_kv_chunk<T, DP, kExact, Shared8>), dim3((uint32_t)p.blocks), dim3(kThreads), 0, s, c,
                     b, q, out, scale, window, causal, p.row_tiles, p.by_length, Partial{nullptr, nullptr, 1, 0}, lse);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk8(const AttendPlan& p, const Plan8& plan, const Cache8& c, uint32_t dtype, const Batch& b,
                         const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                         float* lse, hipStream_t s) {
  Shared8 cache;
  (Cache8&)cache = c;
  cache.plan = plan;
#define IBP_KV8_CHUNK(T, DP, E) \
  run_chunk8<T, DP, E>(p, cache, b, q, out, scale, window, causal, lse, s)
#define IBP_KV8_CHUNK_T(T)                                                                     \
  (c.head_dim == 64    ? IBP_KV8_CHUNK(T, 64, true)                                            \
   : c.head_dim < 64   ? IBP_KV8_CHUNK(T, 64, false)                                           \
   : c.head_dim <= 96  ? IBP_KV8_CHUNK(T, 96, false)                                           \
   : c.head_dim < 128  ? IBP_KV8_CHUNK(T, 128, false)                                          \
   : c.head_dim == 128 ? IBP_KV8_CHUNK(T, 128, true)                                           \
   : c.head_dim <= 192 ? IBP_KV8_CHUNK(T, 192, false)                                          \
   : c.head_dim < 256  ? IBP_KV8_CHUNK(T, 256, false)                                          \
                       : IBP_KV8_CHUNK(T, 256, true))
  return dtype == IBP_KV_F16 ? IBP_KV8_CHUNK_T(_Float16) : IBP_KV8_CHUNK_T(__bf16);
#undef IBP_KV8_CHUNK_T
#undef IBP_KV8_CHUNK
}

}  // namespace kv
}  // namespace ibp
