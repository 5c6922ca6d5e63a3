// kv_mfma.h -- matrix-core pieces shared by the attention kernels.
//
// Operand layouts (gfx950, wave64).  16x16x32: lane l holds of A row l%16, of B
// column l%16, k = 8*(l/16) .. +7; of the result column l%16, rows 4*(l/16) + r
// in register r.  32x32x16: A row / B column l%32, k = 8*(l/32) .. +7; of the
// result column l%32, row 8*(r/4) + 4*(l/32) + r%4 in register r.
//
// Both attention kernels compute S^T = K Q^T and O^T = V^T P^T.  A lane then
// holds scores of one query only (its column), so the softmax needs no
// broadcast, and the scores it holds are, once exponentiated, its part of the
// second product's B operand as they stand: the order of the keys inside a
// product's k does not matter as long as both operands use the same, so k is
// numbered the way the first product leaves its rows.
#pragma once

#include "kv.h"

namespace ibp {
namespace kv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T>
using V8 = typename Vec8<T>::type;

__device__ __forceinline__ f32x4 mfma16(V8<_Float16> a, V8<_Float16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(V8<__bf16> a, V8<__bf16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(V8<_Float16> a, V8<_Float16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(V8<__bf16> a, V8<__bf16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Waits until results of matrix instructions can be read by others.  The
// compiler does so itself where the reader follows in the same basic block; where a
// branch lay between (the scores' masks) its output had no wait on the
// taken path, and the scores read were old ones now and then.  20 wait states
// cover the longest form used here (19 for 16 passes).
__device__ __forceinline__ void settle(f32x4& a, f32x4& b) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3" : "+v"(a), "+v"(b));
}
__device__ __forceinline__ void settle(f32x4& a) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3" : "+v"(a));
}
__device__ __forceinline__ void settle(f32x16& a) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3" : "+v"(a));
}
__device__ __forceinline__ void settle(f32x16& a, f32x16& b) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 3" : "+v"(a), "+v"(b));
}
template <typename V, int N>
__device__ __forceinline__ void settle(V (&a)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) settle(a[i], a[i + 1]);
  if (N % 2) settle(a[N - 1]);
}

// Transposed LDS read: the 16 lanes of a group point at four rows of 16 values
// (lane i of the group at row i/4, columns 4*(i%4) .. +3); lane i gets column i of the
// four rows.
template <typename T>
__device__ __forceinline__ s16x4 read_tr(const T* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
}
template <typename T>
__device__ __forceinline__ V8<T> join(s16x4 lo, s16x4 hi) {
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(V8<T>, v);
}

// max / sum over lanes l, l^32 (and l^16): both halves end with the result.
__device__ __forceinline__ float max_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_quarter(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_quarter(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// The base that a row's exponents are taken against follows the row's largest score so far at a
// distance: it is raised, to kLift below that score, when the score passes it by kRoom, so that
// few steps of k_kv_chunk rescale what was summed before them (k_kv_decode, whose vector ALU has
// time, raises it with every new maximum).  The largest weight lies between 2^kLift
// and 2^kRoom, where its rounding is as exact as near 1.  bf16 has the range of fp32: weights up to 1, so
// that sums of large values pass 2^128 no sooner than the values' own.  fp16 has none below
// 2^-24 and its full precision only from 2^-14 up: with its weights near the type's upper end
// 2^-26 of the largest one still has all of it, and what is lost of n smaller ones is below n * 2^-37
// of the largest (with weights up to 1 it was n * 2^-25: 30,000 weights of 2^-25, 7.5e-4 of
// the sum together, came out 2 % short).  Scores past 2^20 are the base themselves: their
// distance to another base would be rounded by more than the room can bear.
template <typename T>
struct Base;
template <>
struct Base<_Float16> {
  static constexpr float kLift = 12.f, kRoom = 15.f;
};
template <>
struct Base<__bf16> {
  static constexpr float kLift = -8.f, kRoom = 0.f;
};
template <typename T>
__device__ __forceinline__ float next_base(float base, float most) {
  return fmaxf(base, fabsf(most) < 0x1p20f ? most - Base<T>::kLift : most);
}

// 16 B from global memory through a global-address-space pointer.
template <typename T>
__device__ __forceinline__ V8<T> load_row8(const T* p) {
  typedef __attribute__((address_space(1))) const V8<T> global_v8;
  return *(global_v8*)(uintptr_t)p;
}

// What a masked or missing key reads: zeros, so that nothing that lies in unused memory
// (a NaN times a weight of zero is a NaN) reaches the product with the values.
static __device__ const uint4 zero_row[IBP_KV_MAX_HEAD_DIM / 8] = {};

// Infinities and NaNs among values.  Whoever sees one has it in that channel, whatever its weight (which
// may be rounded to zero, in one split of the keys and not in another): a NaN, or an infinity if it
// meets no NaN and no other infinity.  Among keys that only some of a product's rows see, such a
// value times the weight of zero of a row that does not see it would be a NaN, so it stays
// out of the product (finite_part).  Elsewhere it goes in, and leaves no output finite that it
// meets, since any weight times it is no number: probe() finds that at the end.  In both cases a second
// product of the values' codes with the rows' visibility (1 or 0) counts, exactly for up to
// 127 keys, what each output sees: +inf counts 1, -inf 128, NaN 16384 (add_odd).
template <typename T>
__device__ __forceinline__ V8<T> finite_part(V8<T> v) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (!isfinite((float)v[e])) v[e] = (T)0.f;
  return v;
}
template <typename T>
__device__ __forceinline__ V8<T> odd_code(V8<T> v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (float)v[e];
    v[e] = (T)(isfinite(x) ? 0.f : x > 0.f ? 1.f : x < 0.f ? 128.f : 16384.f);
  }
  return v;
}
// A NaN of the products may stand for an infinity (times 0): what it is is counted here.  One that
// was counted is 0x7FFFFFFF, whose low bits no product of 16-bit values leaves set.
__device__ __forceinline__ float add_odd(float o, float count) {
  const uint32_t n = (uint32_t)count;
  if (n == 0 || __float_as_uint(o) == 0x7FFFFFFFu) return o;
  if (isnan(o)) o = 0.f;
  if (n & 127u) o += INFINITY;
  if ((n >> 7) & 127u) o -= INFINITY;
  return n >> 14 || isnan(o) ? __uint_as_float(0x7FFFFFFFu) : o;
}
// Not zero if one of the outputs is no number.
template <typename V, int N>
__device__ __forceinline__ float probe(const V (&o)[N]) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int r = 0; r < (int)(sizeof(V) / sizeof(float)); ++r) x[r % 4] = fmaf(o[t][r], 0.f, x[r % 4]);
  return (x[0] + x[1]) + (x[2] + x[3]);
}
// A partial result times its factor.
__device__ __forceinline__ float scaled(float o, float factor) { return isfinite(o) ? o * factor : o; }
// An output from its sum of values and the inverse of its sum of weights (0: there is no weight, the
// output is 0).  A mean of T's numbers is none past T's largest one; what the weights' rounding adds could
// make an infinity of it.
template <typename T>
__device__ __forceinline__ T mean(float o, float inv) {
  constexpr float kMost = __is_same(T, _Float16) ? 65504.f : 0x1.FEp127f;
  float x = inv == 0.f ? 0.f : o * inv;
  if (isfinite(o)) x = x > kMost ? kMost : x < -kMost ? -kMost : x;  // (a NaN stays)
  return (T)x;
}
template <typename T>
__device__ __forceinline__ bool any_odd(V8<T> v) {
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) odd = odd || !isfinite((float)v[e]);
  return odd;
}

// Where a row's partial results of the splits of its keys lie in the
// workspace: float[unit][split][head_dim], then float2[unit][split] of (base,
// sum); unit = row * heads + head.  Scores in the exponent of 2.
struct Partial {
  float* o;
  float2* ms;
  uint32_t splits, head_dim;
  __device__ float* row(uint64_t unit, uint32_t split) const {
    return o + (unit * splits + split) * head_dim;
  }
};

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

constexpr uint32_t kMaxSplits = 1024;

// How a call is run: kernel, tiles of rows, splits of the keys.
struct AttendPlan {
  bool few;            // few rows share their keys: kv_decode.hip, else kv_chunk.hip
  uint32_t row_tiles;  // of a sequence and key head (of a row and key head in lists)
  uint32_t heads;      // key heads of a workgroup of kv_decode.hip
  uint32_t splits;
  bool by_length;      // kv_chunk.hip: the longest sequences' tiles first
  uint64_t blocks;
};

hipError_t launch_decode(const AttendPlan& p, const Cache& c, uint32_t dtype, const Batch& b,
                         const Rows& q, const Rows& out, const int32_t* sel, uint32_t n_select,
                         float scale, uint32_t window, bool causal, float* lse, Partial part,
                         hipStream_t s);
constexpr uint32_t kChunkRows = 128;  // rows of a workgroup of kv_chunk.hip
hipError_t launch_chunk(const AttendPlan& p, const Cache& c, uint32_t dtype, const Batch& b,
                        const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                        float* lse, Partial part, hipStream_t s);
hipError_t launch_join(uint32_t dtype, const Batch& b, const Rows& out, Partial part, float* lse,
                       hipStream_t s);

}  // namespace kv
}  // namespace ibp
