// kv_append.hip -- new keys and values into a paged cache (with each head's
// norm and rotation on the way, queries too), and the pages' key bounds.
#include "ibp_device.h"
#include "kv_mfma.h"

namespace ibp {
namespace kv {

namespace {

template <typename T>
__device__ __forceinline__ void load8(const T* p, float x[8]) {
  const typename Vec8<T>::type v = *(const typename Vec8<T>::type*)p;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f32(v[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float x[8]) {
  typename Vec8<T>::type v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (T)x[i];
  *(typename Vec8<T>::type*)p = v;
}

// A wave (or several, for few tokens) per token; L lanes (a power of two) per head, the heads
// in the order queries, keys, values.  A lane holds two pieces of eight channels of its head
// such that the rotation stays inside it: pieces c and c + rope_dim / 16 where halves turn (c <
// rope_dim / 16), two neighbouring ones elsewhere.  So the token's cosines and
// sines, its slot and the norms' weights are read once and stay in registers for all of its
// heads; what is left is one pass over the rows.  The norm's sum of squares goes over the L
// lanes by butterflies.  Bound by reading and writing the rows: 16,000 tokens of 32 + 8 + 8
// heads of 128 (402 MB) 79 us, 5.1 TB/s; with a group of lanes per (token, head), each reading
// its part of the rotation, 292 us.
template <typename T, int L>
__global__ __launch_bounds__(256) void k_kv_append(Cache cache, Rows k, Rows v, Rows q, Rows q_out,
                                                   const int64_t* __restrict__ slots,
                                                   const int64_t* __restrict__ positions,
                                                   uint32_t n_tokens, uint32_t parts,
                                                   const float* __restrict__ rope,
                                                   uint64_t n_positions, uint32_t rope_dim,
                                                   bool interleaved, const T* __restrict__ q_norm,
                                                   const T* __restrict__ k_norm, float eps) {
  constexpr uint32_t HW = kWave / L;  // heads of a wave at a time
  typedef V8<T> v8;
  const uint32_t lane = threadIdx.x % kWave;
  const uint32_t c = lane % L, sub = lane / L;
  const uint32_t pieces = cache.head_dim / 8, turned = rope ? rope_dim / 8 : 0;
  const bool halves = !interleaved && c < turned / 2;
  const uint32_t c0 = interleaved ? 2 * c : halves ? c : turned + 2 * (c - turned / 2);
  const uint32_t c1 = halves ? c + turned / 2 : c0 + 1;
  const bool has0 = c0 < pieces, has1 = c1 < pieces;
  const bool turns = interleaved ? c0 < turned : halves;  // turned is even: c1 turns with c0
  v8 wq[2] = {}, wk[2] = {};
  if (q_norm) {
    if (has0) wq[0] = load_row8(q_norm + c0 * 8);
    if (has1) wq[1] = load_row8(q_norm + c1 * 8);
  }
  if (k_norm) {
    if (has0) wk[0] = load_row8(k_norm + c0 * 8);
    if (has1) wk[1] = load_row8(k_norm + c1 * 8);
  }
  const uint32_t heads = q.n_heads + 2 * cache.n_heads;
  const uint32_t per_part = (heads + parts - 1) / parts;
  const uint64_t capacity = (uint64_t)cache.n_pages * cache.page.d;
  for (uint64_t u = (uint64_t)blockIdx.x * 4 + uniform(threadIdx.x / kWave);
       u < (uint64_t)n_tokens * parts; u += (uint64_t)gridDim.x * 4) {
    const uint32_t t = parts == 1 ? (uint32_t)u : (uint32_t)(u / parts);
    const uint32_t part = parts == 1 ? 0 : (uint32_t)(u - (uint64_t)t * parts);
    const int64_t slot = slots[t];
    const int64_t pos = rope ? positions[t] : 0;
    const bool placed = slot >= 0 && (uint64_t)slot < capacity &&
                        (!rope || (pos >= 0 && (uint64_t)pos < n_positions));
    uint64_t at = 0;
    float co[8], si[8];
    if (placed) {
      const uint64_t page = (uint64_t)slot / cache.page.d;
      at = page * cache.page_stride + ((uint64_t)slot - page * cache.page.d) * cache.token_stride;
      if (turns) {
        // halves: of channels 8 c0 .. +7; interleaved: of pairs 4 c0 .. +7 (both pieces)
        const float* row = rope + (uint64_t)pos * rope_dim + (interleaved ? c0 * 4 : c0 * 8);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 a = *(const float4*)(row + e), b = *(const float4*)(row + rope_dim / 2 + e);
          co[e] = a.x, co[e + 1] = a.y, co[e + 2] = a.z, co[e + 3] = a.w;
          si[e] = b.x, si[e + 1] = b.y, si[e + 2] = b.z, si[e + 3] = b.w;
        }
      }
    }
    const uint32_t h_end = min((part + 1) * per_part, heads);
    for (uint32_t h0 = part * per_part; h0 < h_end; h0 += HW) {
      const uint32_t hh = h0 + sub;
      const bool on = hh < h_end;
      const bool is_q = hh < q.n_heads;
      const bool is_v = hh >= q.n_heads + cache.n_heads;
      const bool reads = on && placed, writes = on && (placed || is_q);
      const uint32_t h = is_q ? hh : hh - q.n_heads - (is_v ? cache.n_heads : 0);
      const T* src = is_q   ? (const T*)q.p + t * q.token_stride + (uint64_t)h * q.head_stride
                     : is_v ? (const T*)v.p + t * v.token_stride + (uint64_t)h * v.head_stride
                            : (const T*)k.p + t * k.token_stride + (uint64_t)h * k.head_stride;
      T* dst = is_q ? (T*)q_out.p + t * q_out.token_stride + (uint64_t)h * q_out.head_stride
                    : (T*)(is_v ? cache.v : cache.k) + at + (uint64_t)h * cache.head_stride;
      v8 a = {}, b = {};
      if (reads && has0) a = load_row8(src + c0 * 8);
      if (reads && has1) b = load_row8(src + c1 * 8);
      const T* norm = is_q ? q_norm : is_v ? nullptr : k_norm;
      if (!is_v && (norm || turned)) {  // the same for the L lanes of a head
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = to_f32(a[e]), y[e] = to_f32(b[e]);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
          for (int d = 1; d < L; d <<= 1) ss += __shfl_xor(ss, d, L);
          const float inv = 1.0f / sqrtf(ss / (float)cache.head_dim + eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = x[e] * inv * to_f32(is_q ? wq[0][e] : wk[0][e]);
            y[e] = y[e] * inv * to_f32(is_q ? wq[1][e] : wk[1][e]);
          }
        }
        if (turns && placed) {
          if (interleaved) {
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
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = (T)x[e], b[e] = (T)y[e];
        if (!placed) a = b = v8{};  // (0 / sqrt(0) of a token that is not placed is not written)
      }
      if (writes && has0) *(v8*)(dst + c0 * 8) = a;
      if (writes && has1) *(v8*)(dst + c1 * 8) = b;
    }
  }
}

template <typename T, int L>
hipError_t run_append(const Cache& c, const Rows& k, const Rows& v, const Rows& q,
                      const Rows& q_out, const int64_t* slots, const int64_t* positions,
                      uint32_t n_tokens, const float* rope, uint64_t n_positions,
                      uint32_t rope_dim, bool interleaved, const void* q_norm, const void* k_norm,
                      float eps, hipStream_t s) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  // few tokens: a token's heads over several waves, until every CU has eight
  const uint32_t heads = q.n_heads + 2 * c.n_heads, turns = (heads * L + kWave - 1) / kWave;
  uint32_t parts = (uint32_t)(((uint64_t)di.cus * 8 + n_tokens - 1) / n_tokens);
  if (parts > turns) parts = turns;
  const uint64_t want = ((uint64_t)n_tokens * parts + 3) / 4;
  const uint64_t cap = (uint64_t)di.cus * 8;
  hipLaunchKernelGGL((k_kv_append<T, L>), dim3((uint32_t)(want < cap ? want : cap)), dim3(256), 0,
                     s, c, k, v, q, q_out, slots, positions, n_tokens, parts, rope, n_positions,
                     rope_dim, interleaved, (const T*)q_norm, (const T*)k_norm, eps);
  return hipGetLastError();
}

template <typename T>
__device__ __forceinline__ T nan_min(T a, T b) {
  return (b < a || b != b) ? b : a;
}
template <typename T>
__device__ __forceinline__ T nan_max(T a, T b) {
  return (b > a || b != b) ? b : a;
}

// A thread per (page, head, eight channels): it walks the page's tokens, eight loads in flight
// (one at a time 34 us where this takes 27).  Bound by reading the keys: 1,639 pages of 32 tokens,
// 8 heads of 128 (114 MB) 27 us, 4.2 TB/s; two or four threads a piece 25 to 27 us.
template <typename T>
__global__ __launch_bounds__(256) void k_kv_page_bounds(Cache cache, Batch b, T* __restrict__ bounds,
                                                        uint32_t chunks) {
  const uint32_t s = blockIdx.y;
  const Seq q = load_seq(b, s);
  if (q.q_len <= 0) return;
  const int32_t from = max(q.first, 0);
  const int32_t to = min(q.first + q.q_len, q.n_keys);  // new positions [from, to)
  if (from >= to) return;
  const uint32_t p0 = cache.page.div((uint32_t)from), p1 = cache.page.div((uint32_t)to - 1);
  const uint32_t per_page = cache.n_heads * chunks;
  const uint64_t n = (uint64_t)(p1 - p0 + 1) * per_page;
  for (uint64_t u = (uint64_t)blockIdx.x * 256 + threadIdx.x; u < n;
       u += (uint64_t)gridDim.x * 256) {
    const uint32_t page = p0 + (uint32_t)(u / per_page);
    const uint32_t rest = (uint32_t)(u % per_page);
    const uint32_t h = rest / chunks, c = rest % chunks;
    const int32_t id = b.table[(uint64_t)s * b.table_stride + page];
    if (id < 0 || (uint32_t)id >= cache.n_pages) continue;
    const uint32_t n_tok = min(cache.page.d, (uint32_t)q.n_keys - page * cache.page.d);
    const T* src = (const T*)cache.k + (uint64_t)(uint32_t)id * cache.page_stride +
                   (uint64_t)h * cache.head_stride + c * 8;
    float lo[8], hi[8];
    load8(src, lo);
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = lo[i];
    // eight tokens in flight; past the last one the first is read again
    for (uint32_t t = 1; t < n_tok; t += 8) {
      float x[8][8];
#pragma unroll
      for (uint32_t a = 0; a < 8; ++a) load8(src + (t + a < n_tok ? t + a : 0) * cache.token_stride, x[a]);
#pragma unroll
      for (uint32_t a = 0; a < 8; ++a)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = nan_min(lo[i], x[a][i]);
          hi[i] = nan_max(hi[i], x[a][i]);
        }
    }
    T* dst = bounds + ((uint64_t)(uint32_t)id * cache.n_heads + h) * 2 * cache.head_dim + c * 8;
    store8(dst, lo);
    store8(dst + cache.head_dim, hi);
  }
}

template <typename T>
hipError_t run_page_bounds(const Cache& c, const Batch& b, void* bounds, hipStream_t s) {
  const uint32_t chunks = c.head_dim / 8;
  const uint32_t pages = min(c.page.div(b.max_q ? b.max_q - 1 : 0) + 2, b.max_pages);
  const uint64_t n = (uint64_t)pages * c.n_heads * chunks;
  uint64_t blocks = (n + 255) / 256;
  if (blocks > 65535) blocks = 65535;
  for (uint32_t s0 = 0; s0 < b.n_seqs; s0 += 65535) {
    Batch part = b;
    part.q_start += s0;
    part.kv_len += s0;
    part.table += (uint64_t)s0 * b.table_stride;
    part.n_seqs = b.n_seqs - s0 < 65535 ? b.n_seqs - s0 : 65535;
    hipLaunchKernelGGL(k_kv_page_bounds<T>, dim3((uint32_t)blocks, part.n_seqs), dim3(256), 0, s,
                       c, part, (T*)bounds, chunks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_append(const Cache& c, uint32_t dtype, const Rows& k, const Rows& v,
                         const Rows& q, const Rows& q_out, const int64_t* slots,
                         const int64_t* positions, uint32_t n_tokens, const float* rope,
                         uint64_t n_positions, uint32_t rope_dim, bool interleaved,
                         const void* q_norm, const void* k_norm, float eps, hipStream_t s) {
  if (n_tokens == 0) return hipSuccess;
  // lanes of a head: pairs of turned pieces, then pairs of the rest
  const uint32_t turned = rope ? rope_dim / 8 : 0;
  const uint32_t lanes = turned / 2 + (c.head_dim / 8 - turned + 1) / 2;
#define IBP_KV_APPEND_L(T, L)                                                                  \
  run_append<T, L>(c, k, v, q, q_out, slots, positions, n_tokens, rope, n_positions, rope_dim, \
                   interleaved, q_norm, k_norm, eps, s)
#define IBP_KV_APPEND(T)                                                                    \
  (lanes <= 4 ? IBP_KV_APPEND_L(T, 4) : lanes <= 8 ? IBP_KV_APPEND_L(T, 8) : IBP_KV_APPEND_L(T, 16))
  return dtype == IBP_KV_F16 ? IBP_KV_APPEND(_Float16) : IBP_KV_APPEND(__bf16);
#undef IBP_KV_APPEND
#undef IBP_KV_APPEND_L
}

hipError_t launch_page_bounds(const Cache& c, uint32_t dtype, const Batch& b, void* bounds,
                              hipStream_t s) {
  if (b.n_seqs == 0 || b.max_q == 0 || b.max_pages == 0) return hipSuccess;
  return dtype == IBP_KV_F16 ? run_page_bounds<_Float16>(c, b, bounds, s)
                             : run_page_bounds<__bf16>(c, b, bounds, s);
}

}  // namespace kv
}  // namespace ibp
