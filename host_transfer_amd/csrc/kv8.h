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

constexpr uint32_t kMaxShared = 1024;  // items whose keys are shared out over workgroups
constexpr uint32_t kLeastSteps = 8;    // of k_kv_chunk (64 keys each), that are worth a workgroup

// How keys are shared out.  An item is a sequence (few rows: up to 32 that share a key head) or a tile of
// kChunkRows of its rows: item (row_tiles - 1 - tile) * n_seqs + sequence.  A head group (one key head or four)
// has `places` workgroups: one for each item (shares 0), or those that the items' keys are split over by
// their lengths, which the kernel reads, at least one for each item and at most `shares` where that is enough.
// A split item's results are in the workspace: heads[item] = (its first place, its splits), firsts[place] = (the
// item that is split from there on, its splits; 0 elsewhere; many rows only), o
// float[place][key head][row of the item][head_dim], ms float2[place][key head][row] of (base, sum).
struct Plan8 {
  uint32_t shares, places, rows, row_tiles, head_group;
  bool wide_join;
  int2 *heads, *firsts;
  float* o;
  float2* ms;
};
// A cache with its plan, as the chunk kernel takes it.
struct Shared8 : Cache8 {
  Plan8 plan;
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

// The weights' range over a cache in 8 bits (Base in kv_mfma.h).  In bf16 they are 2^-31 where those of the
// 16-bit cache are 2^-8: a sum over 2^30 keys of the type's largest values (2^24 in k_kv_chunk, where weights may
// grow by 2^kRoom) stays below 2^128, and what a weight near the largest makes of a value, read as its
// half, is no number below fp32's least normal one down to values of 2^-94.  They are so for scores of any
// size, as weights of 1 would let two of the largest values pass 2^128: the 31 are no part of the base, which is the
// largest score (to the last place of base + 31, so that this sum is exact).  With bases up to 2^20 a weight
// is 2^(score - (base + 31)), beyond 2^((score - base) - 31).
template <typename T>
struct In8 {};
template <>
struct Base<In8<_Float16>> : Base<_Float16> {};
template <>
struct Base<In8<__bf16>> {
  static constexpr float kLift = 0.f, kRoom = 7.f, kBeside = 31.f;
};
template <>
__device__ __forceinline__ float next_base<In8<__bf16>>(float base, float most) {
  return fmaxf(base, (most + Base<In8<__bf16>>::kBeside) - Base<In8<__bf16>>::kBeside);
}

// Codes as halves of their 16-bit values, with their block's power of two: the largest that rows of a
// type's numbers are rounded up to, 2^16 and 2^128, are past that type.  Scores and outputs are then taken kScale times.
// (The conversion takes the power's exponent field alone: 0 is 2^-127.)
template <typename T>
struct Read8;
template <>
struct Read8<__bf16> {
  static constexpr float kScale = 2.f;
  static __device__ __forceinline__ float power(uint32_t e) { return __uint_as_float((valid_exponent(e) - 1) << 23); }
  static __device__ __forceinline__ V8<__bf16> eight(uint32_t a, uint32_t b, float power) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    const v2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, power, false);
    const v2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, power, true);
    const v2 z = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, power, false);
    const v2 w = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, power, true);
    return V8<__bf16>{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
  }
};
template <>
struct Read8<_Float16> {
  static constexpr float kScale = 2.f;
  static __device__ __forceinline__ float power(uint32_t e) { return power_of(min(max(e, 2u), 254u) - 1); }
  static __device__ __forceinline__ V8<_Float16> eight(uint32_t a, uint32_t b, float power) {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    const v2 x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, power, false);
    const v2 y = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, power, true);
    const v2 z = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, power, false);
    const v2 w = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, power, true);
    return V8<_Float16>{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
  }
};

}  // namespace kv
}  // namespace ibp
