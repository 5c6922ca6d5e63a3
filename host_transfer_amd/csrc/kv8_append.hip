// kv8_append.hip -- new keys and values into a paged cache of e4m3 codes, with each head's norm and
// rotation on the way (queries too).
#include "ibp_device.h"
#include "kv8.h"

namespace ibp {
namespace kv {

namespace {

constexpr uint32_t kWaves = 4;  // of a workgroup; each works by itself

// The call's norm and rotation, and the part of a head that a lane holds: two pieces of eight
// channels such that the rotation stays inside the lane (pieces c and c + rope_dim / 16 where halves
// turn, two neighbouring ones elsewhere).
struct Turning {
  const float* rope;
  const int64_t* positions;
  uint64_t n_positions;
  uint32_t rope_dim, head_dim;
  bool interleaved;
  float eps;
};
struct Pieces {
  uint32_t c0, c1;
  bool has0, has1, halves, turns;
};
__device__ __forceinline__ Pieces pieces_of(const Turning& t, uint32_t c) {
  const uint32_t pieces = t.head_dim / 8, turned = t.rope ? t.rope_dim / 8 : 0;
  Pieces p;
  p.halves = !t.interleaved && c < turned / 2;
  p.c0 = t.interleaved ? 2 * c : p.halves ? c : turned + 2 * (c - turned / 2);
  p.c1 = p.halves ? c + turned / 2 : p.c0 + 1;
  p.has0 = p.c0 < pieces;
  p.has1 = p.c1 < pieces;
  p.turns = t.interleaved ? p.c0 < turned : p.halves;  // turned is even: c1 turns with c0
  return p;
}
// A token's cosines and sines for this lane's pieces.
__device__ __forceinline__ void load_turn(const Turning& t, const Pieces& p, uint64_t pos, float (&co)[8],
                                          float (&si)[8]) {
  // halves: of channels 8 c0 .. +7; interleaved: of pairs 4 c0 .. +7 (both pieces)
  const float* row = t.rope + pos * t.rope_dim + (t.interleaved ? p.c0 * 4 : p.c0 * 8);
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const float4 a = *(const float4*)(row + e), b = *(const float4*)(row + t.rope_dim / 2 + e);
    co[e] = a.x, co[e + 1] = a.y, co[e + 2] = a.z, co[e + 3] = a.w;
    si[e] = b.x, si[e + 1] = b.y, si[e + 2] = b.z, si[e + 3] = b.w;
  }
}
// Norm (over the L lanes of the head) and rotation of the pieces x and y.
template <typename T, int L>
__device__ __forceinline__ void turn(const Turning& t, const Pieces& p, bool norm, const V8<T> (&w)[2],
                                     bool rotates, const float (&co)[8], const float (&si)[8], float (&x)[8],
                                     float (&y)[8]) {
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
    for (int d = 1; d < L; d <<= 1) ss += __shfl_xor(ss, d, L);
    const float inv = 1.0f / sqrtf(ss / (float)t.head_dim + t.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = x[e] * inv * to_f32(w[0][e]);
      y[e] = y[e] * inv * to_f32(w[1][e]);
    }
  }
  if (!rotates || !p.turns) return;
  if (t.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float x0 = x[e], y0 = y[e];
      x[e] = x0 * co[e / 2] - x[e + 1] * si[e / 2];
      x[e + 1] = x[e + 1] * co[e / 2] + x0 * si[e / 2];
      y[e] = y0 * co[4 + e / 2] - y[e + 1] * si[4 + e / 2];
      y[e + 1] = y[e + 1] * co[4 + e / 2] + y0 * si[4 + e / 2];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x0 = x[e];
      x[e] = x0 * co[e] - y[e] * si[e];
      y[e] = y[e] * co[e] + x0 * si[e];
    }
  }
}

// Eight values times inv, a power of two, as codes: to the nearest, ties to even, by the conversion
// itself; x + 0 * x is x, and NaN for an infinity.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf(x[e], 0.f, x[e]) * inv;
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}
__device__ __forceinline__ void decode4(uint32_t c, float* x) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
}

// The largest finite magnitude (fmaxf passes over the NaN that a value that is none becomes).
__device__ __forceinline__ float largest(const float (&x)[8], float most) {
#pragma unroll
  for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(fmaf(x[e], 0.f, x[e])));
  return most;
}

// Waves 0 .. kv_units-1: a wave per (sequence, block that gains tokens, K|V and head, heads
// innermost), L lanes per token row, so that 64 / L tokens are read at a time.  It sees all of
// the block's new tokens, so the exponent needs no other wave; up to kKeep turns of rows stay in
// registers between its maximum and their codes, further ones are formed again from
// memory (L2).  The blocks are counted by sequence, up to seq_blocks each, or (seq_blocks 0), where
// that would be more units than there are rows (a long prompt beside many single tokens), by
// rows, of which the first of each block works.  kHeads: few new tokens a block, many sequences: the lanes of
// a wave hold HW heads' rows of one token, each head's exponent its own lanes' (227 single tokens of
// 40 heads of 64 17.5 us without, 8.3 with).  Where the exponent rises, the tokens in front of the new ones
// are rounded to it.
// The waves behind: queries, a wave (several, `parts`, for few rows) per row, as k_kv_append.
// Bound by reading the 16-bit rows and writing them or half of them: 16,800 rows of 32 + 8 + 8 heads of 128
// (387 MB) 88 us, 4.4 TB/s (155 with four kept turns, whose registers leave two waves a SIMD; 92 with
// a launch each for keys and queries, 94 with the queries first, 89 with both in turn).  One token's call 5.4
// us, its chain of lookups; the rows are requested ahead of it.
template <typename T, int L, bool kHeads>
__global__ __launch_bounds__(256, 4) void k_kv8_append(Cache8 cache, Batch b, Rows k, Rows v, Rows q, Rows q_out,
                                                    Turning t, const T* __restrict__ q_norm,
                                                    const T* __restrict__ k_norm, uint32_t seq_blocks,
                                                    uint64_t kv_units, uint32_t parts) {
  constexpr uint32_t HW = kWave / L;  // rows of a wave at a time
  constexpr uint32_t kStep = kHeads ? 1 : HW;  // tokens of a turn
  constexpr uint32_t kKeep = 2;
  typedef V8<T> v8;
  const uint32_t lane = threadIdx.x % kWave, c = lane % L, sub = lane / L;
  const Pieces p = pieces_of(t, c);
  uint64_t u = ((uint64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + uniform(threadIdx.x / kWave);
  if (u < kv_units) {
    const uint32_t side = kHeads ? (cache.n_heads + HW - 1) / HW : cache.n_heads;  // units of K, of V
    const uint32_t hh = (uint32_t)(u % (2 * side));
    u /= 2 * side;
    const bool is_v = hh >= side;
    const uint32_t h = (is_v ? hh - side : hh) * (kHeads ? HW : 1) + (kHeads ? sub : 0);
    const uint32_t turn_at = kHeads ? 0 : sub;  // this lane's token of a turn
    const int32_t s = seq_blocks ? (int32_t)(u / seq_blocks) : seq_of_row(b, (int32_t)u);
    if (s < 0) return;
    const Seq sq = load_seq(b, (uint32_t)s);
    const int32_t from = max(sq.first, 0), to = min(sq.first + sq.q_len, sq.n_keys);
    const uint32_t B = cache.block.d;
    int64_t base64, begin64;
    if (seq_blocks) {
      base64 = ((int64_t)cache.block.div((uint32_t)from) + (int64_t)(u % seq_blocks)) * B;
      begin64 = base64 > from ? base64 : from;
    } else {  // the row that is the block's first new one
      begin64 = sq.first + ((int64_t)u - sq.row0);
      if (begin64 < from) return;
      base64 = (int64_t)cache.block.div((uint32_t)begin64) * B;
      if (begin64 != base64 && begin64 != from) return;
    }
    if (begin64 >= to) return;
    const int32_t base = (int32_t)base64, begin = (int32_t)begin64, end = (int32_t)(base64 + B < to ? base64 + B : to);
    const uint32_t page = cache.page.div((uint32_t)base), in = (uint32_t)base - page * cache.page.d;
    const int32_t id = b.table[(uint64_t)(uint32_t)s * b.table_stride + page];
    const bool there = id >= 0 && (uint32_t)id < cache.n_pages;  // (looked at once the rows are on their way)
    const bool norm = !is_v && k_norm, rotates = !is_v && t.rope;
    v8 w[2] = {};
    if (norm) {
      if (p.has0) w[0] = load_row8(k_norm + p.c0 * 8);
      if (p.has1) w[1] = load_row8(k_norm + p.c1 * 8);
    }
    const Rows& src = is_v ? v : k;
    // token `at`, normed and rotated; false if it is not placed (its values are then zeros)
    auto row = [&](int32_t at, float (&x)[8], float (&y)[8]) -> bool {
      bool on = at < end && (!kHeads || h < cache.n_heads);
      const uint32_t r = (uint32_t)(sq.row0 + (at - sq.first));
      int64_t pos = 0;
      if (t.rope) {
        if (on) pos = t.positions[r];
        on = on && pos >= 0 && (uint64_t)pos < t.n_positions;
      }
      const T* from_ = (const T*)src.p + r * src.token_stride + (uint64_t)h * src.head_stride;
      v8 a = {}, d = {};
      if (on && p.has0) a = load_row8(from_ + p.c0 * 8);
      if (on && p.has1) d = load_row8(from_ + p.c1 * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = to_f32(a[e]), y[e] = to_f32(d[e]);
      if (norm || rotates) {
        float co[8], si[8];
        if (rotates && on && p.turns) load_turn(t, p, (uint64_t)pos, co, si);
        turn<T, L>(t, p, norm, w, rotates && on, co, si, x, y);
#pragma unroll
        for (int e = 0; e < 8; ++e)  // (0 / sqrt(0) of what is not there)
          if (!on) x[e] = y[e] = 0.f;
      }
      return on;
    };
    float x[kKeep][8], y[kKeep][8], most = 0.f;
    bool on[kKeep];
#pragma unroll
    for (uint32_t i = 0; i < kKeep; ++i) {
      on[i] = row(begin + (int32_t)(i * kStep + turn_at), x[i], y[i]);
      most = largest(y[i], largest(x[i], most));
    }
    if (!there || (kHeads && h >= cache.n_heads)) return;  // (whole heads leave: no lane that another asks)
    uint8_t* codes = (is_v ? cache.v : cache.k) + (uint64_t)(uint32_t)id * cache.page_stride +
                     (uint64_t)in * cache.token_stride + (uint64_t)h * cache.head_stride;
    uint8_t* exp = (is_v ? cache.v_exp : cache.k_exp) +
                   ((uint64_t)(uint32_t)id * cache.page_blocks + cache.block.div(in)) * cache.n_heads + h;
    const uint32_t was = begin > base ? valid_exponent(*exp) : 1;
    auto put = [&](int32_t at, const float (&x)[8], const float (&y)[8], float inv) {
      uint8_t* dst = codes + (uint64_t)(uint32_t)(at - base) * cache.token_stride;
      if (p.has0) *(uint2*)(dst + p.c0 * 8) = encode8(x, inv);
      if (p.has1) *(uint2*)(dst + p.c1 * 8) = encode8(y, inv);
    };
    for (int32_t at = begin + (int32_t)(kKeep * kStep); at < end; at += kStep) {
      float xx[8], yy[8];
      row(at + (int32_t)turn_at, xx, yy);
      most = largest(yy, largest(xx, most));
    }
#pragma unroll
    for (int d = 1; d < (kHeads ? L : kWave); d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
    const uint32_t e = max(exponent_of(most), was);
    const float inv = __uint_as_float(e < 254 ? (254 - e) << 23 : 0x400000u);
    if (begin > base && e > was) {
      const float shift = e - was < 127 ? __uint_as_float((127 + was - e) << 23) : 0.f;
#pragma unroll 4
      for (int32_t at = base + (int32_t)turn_at; at < begin; at += kStep) {
        uint8_t* dst = codes + (uint64_t)(uint32_t)(at - base) * cache.token_stride;
        float xx[8];
        if (p.has0) {
          const uint2 old = *(const uint2*)(dst + p.c0 * 8);
          decode4(old.x, xx);
          decode4(old.y, xx + 4);
          *(uint2*)(dst + p.c0 * 8) = encode8(xx, shift);
        }
        if (p.has1) {
          const uint2 old = *(const uint2*)(dst + p.c1 * 8);
          decode4(old.x, xx);
          decode4(old.y, xx + 4);
          *(uint2*)(dst + p.c1 * 8) = encode8(xx, shift);
        }
      }
    }
    if ((kHeads ? c : lane) == 0) *exp = (uint8_t)e;
#pragma unroll
    for (uint32_t i = 0; i < kKeep; ++i)
      if (on[i]) put(begin + (int32_t)(i * kStep + turn_at), x[i], y[i], inv);
    for (int32_t at = begin + (int32_t)(kKeep * kStep); at < end; at += kStep) {
      float xx[8], yy[8];
      if (row(at + (int32_t)turn_at, xx, yy)) put(at + (int32_t)turn_at, xx, yy, inv);
    }
    return;
  }
  u -= kv_units;
  const uint64_t r64 = u / parts;
  if (q.n_heads == 0 || r64 >= b.n_rows) return;
  const uint32_t r = (uint32_t)r64, part = (uint32_t)(u - r64 * parts);
  const uint32_t per_part = (q.n_heads + parts - 1) / parts;
  const uint32_t h_begin = part * per_part, h_end = min(h_begin + per_part, q.n_heads);
  // the next heads' pieces are on their way while these are turned, the first ones during the
  // chain of loads that says whether the row is placed
  const T* src = (const T*)q.p + r * q.token_stride;
  auto heads = [&](uint32_t h, v8& a, v8& d) {
    a = d = v8{};
    if (h < h_end && p.has0) a = load_row8(src + (uint64_t)h * q.head_stride + p.c0 * 8);
    if (h < h_end && p.has1) d = load_row8(src + (uint64_t)h * q.head_stride + p.c1 * 8);
  };
  v8 a, d;
  heads(h_begin + sub, a, d);
  const int64_t pos = t.rope ? t.positions[r] : 0;
  const int32_t s = seq_of_row(b, (int32_t)r);
  if (s < 0) return;
  const Seq sq = load_seq(b, (uint32_t)s);
  const int32_t at = sq.first + ((int32_t)r - sq.row0);
  bool placed = at >= 0 && at < sq.n_keys && (!t.rope || (pos >= 0 && (uint64_t)pos < t.n_positions));
  if (placed) {
    const int32_t id = b.table[(uint64_t)s * b.table_stride + cache.page.div((uint32_t)at)];
    placed = id >= 0 && (uint32_t)id < cache.n_pages;
  }
  float co[8], si[8];
  if (placed && t.rope && p.turns) load_turn(t, p, (uint64_t)pos, co, si);
  v8 w[2] = {};
  if (q_norm) {
    if (p.has0) w[0] = load_row8(q_norm + p.c0 * 8);
    if (p.has1) w[1] = load_row8(q_norm + p.c1 * 8);
  }
  for (uint32_t h = h_begin + sub; h - sub < h_end; h += HW) {
    v8 next_a, next_d;
    heads(h + HW, next_a, next_d);
    if (q_norm || t.rope) {
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = to_f32(a[e]), y[e] = to_f32(d[e]);
      turn<T, L>(t, p, q_norm != nullptr, w, placed && t.rope, co, si, x, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = (T)x[e], d[e] = (T)y[e];
    }
    if (!placed) a = d = v8{};
    T* dst = (T*)q_out.p + r * q_out.token_stride + (uint64_t)h * q_out.head_stride;
    if (h < h_end && p.has0) *(v8*)(dst + p.c0 * 8) = a;
    if (h < h_end && p.has1) *(v8*)(dst + p.c1 * 8) = d;
    a = next_a;
    d = next_d;
  }
}

template <typename T, int L>
hipError_t run_append8(const Cache8& c, const Batch& b, const Rows& k, const Rows& v, const Rows& q,
                       const Rows& q_out, const Turning& t, const void* q_norm, const void* k_norm,
                       hipStream_t s) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  // new tokens of a sequence touch this many blocks at most
  uint32_t seq_blocks = (uint32_t)(((uint64_t)b.max_q + c.block.d - 2) / c.block.d) + 1;
  uint64_t kv_units = (uint64_t)b.n_seqs * seq_blocks;
  if (kv_units > b.n_rows) {
    kv_units = b.n_rows;
    seq_blocks = 0;
  }
  // Few new tokens a block leave most lanes of a wave per head idle: then a head to each of their groups, once
  // there are more waves than the GPU holds (below, a block whose exponent rises is rounded anew faster
  // with its tokens side by side).
  constexpr uint32_t HW = kWave / L;
  const bool by_heads = 2 * b.max_q <= HW && 2 * b.max_q <= c.n_heads &&
                        kv_units * 2 * c.n_heads > (uint64_t)di.cus * 16;
  kv_units *= 2 * (by_heads ? (c.n_heads + HW - 1) / HW : c.n_heads);
  // few rows: a row's queries over several waves, until every CU has eight
  const uint32_t turns = (q.n_heads * L + kWave - 1) / kWave;
  uint32_t parts = (uint32_t)(((uint64_t)di.cus * 8 + b.n_rows - 1) / b.n_rows);
  if (parts > turns) parts = turns;
  if (parts == 0) parts = 1;
  const uint64_t units = kv_units + (q.n_heads ? (uint64_t)b.n_rows * parts : 0);
  const uint64_t blocks = (units + kWaves - 1) / kWaves;
  // (one dimension's threads are counted in 32 bits; waves past the last unit find no row)
  const uint64_t layers = (blocks + 0xFFFFFEull) / 0xFFFFFFull;
  if (layers > 65535) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)((blocks + layers - 1) / layers), (uint32_t)layers);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, c, b, k, v, q, q_out, t, (const T*)q_norm, (const T*)k_norm,
                       seq_blocks, kv_units, parts);
    return hipGetLastError();
  };
  return by_heads ? launch(k_kv8_append<T, L, true>) : launch(k_kv8_append<T, L, false>);
}

}  // namespace

hipError_t launch_append8(const Cache8& c, uint32_t dtype, const Batch& b, const Rows& k, const Rows& v,
                          const Rows& q, const Rows& q_out, const int64_t* positions, const float* rope,
                          uint64_t n_positions, uint32_t rope_dim, bool interleaved,
                          const void* q_norm, const void* k_norm, float eps, hipStream_t s) {
  if (b.n_rows == 0 || b.n_seqs == 0 || b.max_q == 0) return hipSuccess;
  const Turning t = {rope, positions, n_positions, rope_dim, c.head_dim, interleaved, eps};
  // lanes of a head: pairs of turned pieces, then pairs of the rest
  const uint32_t turned = rope ? rope_dim / 8 : 0;
  const uint32_t lanes = turned / 2 + (c.head_dim / 8 - turned + 1) / 2;
#define IBP_KV8_APPEND_L(T, L) run_append8<T, L>(c, b, k, v, q, q_out, t, q_norm, k_norm, s)
#define IBP_KV8_APPEND(T) \
  (lanes <= 4 ? IBP_KV8_APPEND_L(T, 4) : lanes <= 8 ? IBP_KV8_APPEND_L(T, 8) : IBP_KV8_APPEND_L(T, 16))
  return dtype == IBP_KV_F16 ? IBP_KV8_APPEND(_Float16) : IBP_KV8_APPEND(__bf16);
#undef IBP_KV8_APPEND
#undef IBP_KV8_APPEND_L
}

}  // namespace kv
}  // namespace ibp
