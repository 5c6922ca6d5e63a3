// kv_append.hip -- new keys and values into a paged cache (with each head's
// norm and rotation on the way, queries too), and the pages' key bounds.
#include "ibp_device.h"
#include "kv.h"

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

// G lanes (a power of two, >= head_dim / 8) hold one head, eight channels
// each; lanes past head_dim hold zeros.  Norm: the sum of squares over the G
// lanes by butterflies.  Rotation of halves: the partner channel sits
// rope_dim / 16 lanes away (rope_dim % 16 == 0), so one shuffle per channel
// brings it; interleaved pairs lie in one lane.
template <int G>
__device__ __forceinline__ void norm_rotate(float x[8], uint32_t c, uint32_t head_dim,
                                            const float* w, float eps, const float* rope,
                                            uint32_t rope_dim, bool interleaved) {
  if (w) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
    for (int d = 1; d < G; d <<= 1) ss += __shfl_xor(ss, d, G);
    const float inv = 1.0f / sqrtf(ss / (float)head_dim + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
  }
  if (!rope) return;
  const uint32_t half = rope_dim / 2;
  if (interleaved) {
    if (c * 8 >= rope_dim) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float co = rope[c * 4 + i], si = rope[half + c * 4 + i];
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * co - b * si;
      x[2 * i + 1] = b * co + a * si;
    }
    return;
  }
  const uint32_t hl = half / 8;
  const bool first = c < hl, turns = c < 2 * hl;
  const uint32_t other = turns ? (first ? c + hl : c - hl) : c;
  const uint32_t t = turns ? (first ? c : c - hl) * 8 : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __shfl(x[i], other, G);
    const float co = rope[t + i], si = rope[half + t + i];
    if (turns) x[i] = first ? x[i] * co - y * si : x[i] * co + y * si;
  }
}

// A group of G lanes per (token, head), the heads of a token in the order
// queries, keys, values.
template <typename T, int G>
__global__ __launch_bounds__(256) void k_kv_append(Cache cache, Rows k, Rows v, Rows q, Rows q_out,
                                                   const int64_t* __restrict__ slots,
                                                   const int64_t* __restrict__ positions,
                                                   uint64_t n_units, FastDiv heads,
                                                   const float* __restrict__ rope,
                                                   uint64_t n_positions, uint32_t rope_dim,
                                                   bool interleaved, const T* __restrict__ q_norm,
                                                   const T* __restrict__ k_norm, float eps) {
  const uint32_t c = threadIdx.x % G;
  const uint32_t hd = cache.head_dim;
  const bool live = c * 8 < hd;
  for (uint64_t u = (uint64_t)blockIdx.x * (256 / G) + threadIdx.x / G; u < n_units;
       u += (uint64_t)gridDim.x * (256 / G)) {
    const uint32_t t = heads.div((uint32_t)u);
    uint32_t h = (uint32_t)u - t * heads.d;
    const int64_t slot = slots[t];
    const int64_t pos = rope ? positions[t] : 0;
    const bool placed = slot >= 0 && (uint64_t)slot < (uint64_t)cache.n_pages * cache.page.d &&
                        (!rope || (pos >= 0 && (uint64_t)pos < n_positions));
    const bool is_q = h < q.n_heads;
    const bool is_v = h >= q.n_heads + cache.n_heads;
    if (!placed && !is_q) continue;  // the same for all G lanes of the group
    const T* src;
    T* dst;
    if (is_q) {
      src = (const T*)q.p + t * q.token_stride + (uint64_t)h * q.head_stride;
      dst = (T*)q_out.p + t * q_out.token_stride + (uint64_t)h * q_out.head_stride;
    } else {
      h -= q.n_heads + (is_v ? cache.n_heads : 0);
      const uint32_t page = (uint32_t)((uint64_t)slot / cache.page.d);
      const uint32_t in = (uint32_t)((uint64_t)slot - (uint64_t)page * cache.page.d);
      const uint64_t at = page * cache.page_stride + in * cache.token_stride +
                          (uint64_t)h * cache.head_stride;
      const Rows& r = is_v ? v : k;
      src = (const T*)r.p + t * r.token_stride + (uint64_t)h * r.head_stride;
      dst = (T*)(is_v ? cache.v : cache.k) + at;
    }
    if (is_v) {  // copied bit for bit
      if (live) ((uint4*)dst)[c] = ((const uint4*)src)[c];
      continue;
    }
    float x[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (placed) {
      if (live) load8(src + c * 8, x);
      const T* norm = is_q ? q_norm : k_norm;
      if (norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0.f;
        if (live) load8(norm + c * 8, w);
      }
      if (norm || rope)
        norm_rotate<G>(x, c, hd, norm ? w : nullptr, eps,
                       rope ? rope + (uint64_t)pos * rope_dim : nullptr, rope_dim, interleaved);
    }
    if (live) store8(dst + c * 8, x);
  }
}

template <typename T, int G>
hipError_t run_append(const Cache& c, const Rows& k, const Rows& v, const Rows& q,
                      const Rows& q_out, const int64_t* slots, const int64_t* positions,
                      uint32_t n_tokens, const float* rope, uint64_t n_positions,
                      uint32_t rope_dim, bool interleaved, const void* q_norm, const void* k_norm,
                      float eps, hipStream_t s) {
  const uint32_t heads = q.n_heads + 2 * c.n_heads;
  const uint64_t units = (uint64_t)n_tokens * heads;
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  const uint64_t want = (units + 256 / G - 1) / (256 / G);
  const uint64_t cap = (uint64_t)di.cus * 8;
  hipLaunchKernelGGL((k_kv_append<T, G>), dim3((uint32_t)(want < cap ? want : cap)), dim3(256), 0,
                     s, c, k, v, q, q_out, slots, positions, units, fast_div(heads), rope,
                     n_positions, rope_dim, interleaved, (const T*)q_norm, (const T*)k_norm, eps);
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

// A thread per (page, head, eight channels): it walks the page's tokens.
template <typename T>
__global__ __launch_bounds__(256) void k_kv_page_bounds(Cache cache, Batch b, T* __restrict__ bounds,
                                                        uint32_t pages_per_seq, uint32_t chunks) {
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
    float lo[8], hi[8], x[8];
    load8(src, lo);
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = lo[i];
    for (uint32_t t = 1; t < n_tok; ++t) {
      load8(src + t * cache.token_stride, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] = nan_min(lo[i], x[i]);
        hi[i] = nan_max(hi[i], x[i]);
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
                       c, part, (T*)bounds, pages, chunks);
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
#define IBP_KV_APPEND(T)                                                                          \
  (c.head_dim <= 64                                                                               \
       ? run_append<T, 8>(c, k, v, q, q_out, slots, positions, n_tokens, rope, n_positions,       \
                          rope_dim, interleaved, q_norm, k_norm, eps, s)                          \
   : c.head_dim <= 128                                                                            \
       ? run_append<T, 16>(c, k, v, q, q_out, slots, positions, n_tokens, rope, n_positions,      \
                           rope_dim, interleaved, q_norm, k_norm, eps, s)                         \
       : run_append<T, 32>(c, k, v, q, q_out, slots, positions, n_tokens, rope, n_positions,      \
                           rope_dim, interleaved, q_norm, k_norm, eps, s))
  return dtype == IBP_KV_F16 ? IBP_KV_APPEND(_Float16) : IBP_KV_APPEND(__bf16);
#undef IBP_KV_APPEND
}

hipError_t launch_page_bounds(const Cache& c, uint32_t dtype, const Batch& b, void* bounds,
                              hipStream_t s) {
  if (b.n_seqs == 0 || b.max_q == 0 || b.max_pages == 0) return hipSuccess;
  return dtype == IBP_KV_F16 ? run_page_bounds<_Float16>(c, b, bounds, s)
                             : run_page_bounds<__bf16>(c, b, bounds, s);
}

}  // namespace kv
}  // namespace ibp
