// kv8.h -- what the kernels over the 8-bit paged cache and their C ABI (api_kv8.hip) share.
#pragma once

#include "ibp_kv8.h"
#include "kv_mfma.h"

namespace ibp {
namespace kv {

// The cache; codes and strides in bytes.
struct Cache8 {
  uint8_t *k, *v, *k_exp, *v_exp;
  uint64_t page_stride, token_stride;
  uint32_t head_stride, n_pages, n_heads, head_dim, page_blocks;
  FastDiv page, block;
};

hipError_t launch_append8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& k, const Rows& v,
                          const Rows& q, const Rows& q_out, const int64_t* positions, const float* rope,
                          uint64_t n_positions, uint32_t rope_dim, bool interleaved,
                          const void* q_norm, const void* k_norm, float eps, hipStream_t s);

hipError_t attend8_workspace(const Cache8& c, const Batch& b, uint32_t n_q_heads, uint64_t* bytes);
hipError_t launch_attend8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q, const Rows& out,
                          float scale, uint32_t window, bool causal, float* lse, void* workspace,
                          hipStream_t s);

// The exponent of a block: the least e in [1, 254] with most <= 448 * 2^(e - 127), most >= 0 finite.
// 448 = 1.75 * 2^8; the bits of `most` are its exponent and, below, its mantissa.
__device__ __forceinline__ uint32_t exponent_of(float most) {
  const uint32_t u = __float_as_uint(most);
  const int32_t e = (int32_t)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}
__device__ __forceinline__ uint32_t valid_exponent(uint32_t e) { return min(max(e, 1u), 254u); }
// 2^(e - 127), e in [1, 254]
__device__ __forceinline__ float power_of(uint32_t e) { return __uint_as_float(e << 23); }

}  // namespace kv
}  // namespace ibp
