// kv_attend.hip -- attention over a paged cache, whole or over selected pages.
#include "ibp_device.h"
#include "kv_mfma.h"

namespace ibp {
namespace kv {

namespace {

// A wave per (row, head).  Tiles of 64 keys: lane = key for the scores, lane =
// channel (every 64th) for the sum over values; running maximum and sum of
// the softmax in 32 bits.
template <typename T, bool kSelected>
__global__ __launch_bounds__(256) void k_kv_attend(Cache cache, Batch b, Rows q, Rows out,
                                                   const int32_t* __restrict__ sel,
                                                   uint32_t n_select, float scale, uint32_t window,
                                                   bool causal, float* __restrict__ lse) {
  const uint32_t lane = threadIdx.x % kWave;
  const uint64_t u = (uint64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (u >= (uint64_t)b.n_rows * q.n_heads) return;
  const uint32_t r = (uint32_t)(u / q.n_heads), h = (uint32_t)(u % q.n_heads);
  const int32_t s = seq_of_row(b, (int32_t)r);
  if (s < 0) return;
  const Seq sq = load_seq(b, s);
  const int32_t i = (int32_t)r - sq.row0;
  if (i < 0 || i >= sq.q_len) return;
  const int32_t pos = sq.first + i;
  const uint32_t kh = h / (q.n_heads / cache.n_heads);
  const int32_t hi = causal ? min(pos + 1, sq.n_keys) : sq.n_keys;  // keys [lo, hi)
  const int32_t lo = window ? max(pos - (int32_t)window + 1, 0) : 0;
  const T* qp = (const T*)q.p + r * q.token_stride + (uint64_t)h * q.head_stride;
  const int32_t* list = kSelected ? sel + ((uint64_t)r * cache.n_heads + kh) * n_select : nullptr;
  const int32_t n_virtual = kSelected ? (int32_t)(n_select * cache.page.d) : hi;
  float m = -INFINITY, z = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int32_t t = kSelected ? 0 : lo / kWave * kWave; t < n_virtual; t += kWave) {
    int32_t j = t + (int32_t)lane;
    bool see = j < n_virtual;
    if (kSelected && see) {
      const uint32_t e = cache.page.div((uint32_t)j);
      const int32_t pg = list[e];
      see = pg >= 0 && (uint32_t)pg < b.max_pages && (e == 0 || pg > list[e - 1]);
      j = see ? pg * (int32_t)cache.page.d + (j - (int32_t)(e * cache.page.d)) : 0;
    }
    see = see && j >= lo && j < hi;
    uint64_t at = 0;
    if (see) {
      const uint32_t page = cache.page.div((uint32_t)j);
      const int32_t id = b.table[(uint64_t)s * b.table_stride + page];
      see = id >= 0 && (uint32_t)id < cache.n_pages;
      at = (uint64_t)(uint32_t)id * cache.page_stride +
           (uint64_t)((uint32_t)j - page * cache.page.d) * cache.token_stride +
           (uint64_t)kh * cache.head_stride;
    }
    float x = -INFINITY;
    if (see) {
      x = 0.f;
      for (uint32_t c = 0; c < cache.head_dim; c += 8) {
        const typename Vec8<T>::type a = *(const typename Vec8<T>::type*)(qp + c);
        const typename Vec8<T>::type k = *(const typename Vec8<T>::type*)((const T*)cache.k + at + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) x += to_f32(a[e]) * to_f32(k[e]);
      }
      x *= scale;
    }
    const uint64_t seen = __ballot(see);
    if (!seen) continue;
    float top = x;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    const float m2 = fmaxf(m, top);
    const float base = m2 == -INFINITY ? 0.f : m2;
    const float keep = __expf(m - base);
    const float p = see ? __expf(x - base) : 0.f;
    float sum = p;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d, kWave);
    z = z * keep + sum;
    m = m2;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= keep;
    for (uint64_t left = seen; left; left &= left - 1) {
      const uint32_t l = (uint32_t)__builtin_ctzll(left);
      const float pl = __shfl(p, l, kWave);
      const T* vp = (const T*)cache.v + lane_u64(at, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t c = lane + e * kWave;
        if (c < cache.head_dim) o[e] += pl * to_f32(vp[c]);
      }
    }
  }
  T* op = (T*)out.p + r * out.token_stride + (uint64_t)h * out.head_stride;
  const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t c = lane + e * kWave;
    if (c < cache.head_dim) op[c] = (T)(o[e] * inv);
  }
  if (lse && lane == 0) lse[u] = z == 0.f ? -INFINITY : m + __logf(z);
}

}  // namespace

namespace {

hipError_t make_plan(const Cache& c, const Batch& b, uint32_t n_q_heads, uint32_t n_select,
                     AttendPlan* p) {
  DeviceInfo di;
  hipError_t e = device_info(&di);
  if (e != hipSuccess) return e;
  const uint32_t group = n_q_heads / c.n_heads;
  const uint64_t rows = (uint64_t)(n_select ? 1 : b.max_q) * group;
  p->few = n_select || rows <= 16;
  p->row_tiles = (uint32_t)((rows + 15) / 16);
  const uint64_t base = (uint64_t)(n_select ? b.n_rows : b.n_seqs) * p->row_tiles * c.n_heads;
  const uint64_t keys = n_select ? (uint64_t)n_select * c.page.d : b.max_kv;
  const uint64_t want = (uint64_t)di.cus * 4;
  uint64_t splits = base ? (want + base - 1) / base : 1;
  if (splits > keys / 256) splits = keys / 256;
  p->splits = splits < 1 ? 1 : (uint32_t)splits;
  p->blocks = base * p->splits;
  if (!p->few) p->splits = 1;
  return p->blocks > 0x7FFFFFFFull ? hipErrorInvalidConfiguration : hipSuccess;
}

// The workspace: [unit][split][head_dim] floats, then [unit][split] (max, sum).
uint64_t partial_bytes(const Cache& c, const Batch& b, uint32_t n_q_heads, const AttendPlan& p) {
  if (p.splits == 1) return 0;
  return (uint64_t)b.n_rows * n_q_heads * p.splits * (c.head_dim + 2) * 4;
}

}  // namespace

hipError_t attend_workspace(const Cache& c, const Batch& b, uint32_t n_q_heads, uint32_t n_select,
                            uint64_t* bytes) {
  AttendPlan p;
  hipError_t e = make_plan(c, b, n_q_heads, n_select, &p);
  if (e == hipSuccess) *bytes = partial_bytes(c, b, n_q_heads, p);
  return e;
}

hipError_t launch_attend(const Cache& c, uint32_t dtype, const Batch& b, const Rows& q,
                         const Rows& out, const int32_t* sel, uint32_t n_select, float scale,
                         uint32_t window, bool causal, float* lse, void* workspace,
                         hipStream_t s) {
  AttendPlan p;
  hipError_t e = make_plan(c, b, q.n_heads, n_select, &p);
  if (e != hipSuccess) return e;
  Partial part;
  part.splits = p.splits;
  part.head_dim = c.head_dim;
  part.o = (float*)workspace;
  part.ms = (float2*)(part.o + (uint64_t)b.n_rows * q.n_heads * p.splits * c.head_dim);
  if (p.few) {
    e = launch_decode(p, c, dtype, b, q, out, sel, n_select, scale, window, causal, lse, part, s);
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_join(dtype, b, out, part, lse, s);
  }
  const uint64_t blocks = ((uint64_t)b.n_rows * q.n_heads + 3) / 4;
#define IBP_KV_ATTEND(T)                                                                           \
  hipLaunchKernelGGL((k_kv_attend<T, false>), dim3((uint32_t)blocks), dim3(256), 0, s, c, b, q, out, \
                     sel, n_select, scale, window, causal, lse)
  if (dtype == IBP_KV_F16) IBP_KV_ATTEND(_Float16);
  else IBP_KV_ATTEND(__bf16);
#undef IBP_KV_ATTEND
  return hipGetLastError();
}

}  // namespace kv
}  // namespace ibp
