// kv_select.hip -- the pages each row and key head attends: a score of every
// page from its key bounds, then the best pages.
#include "ibp_device.h"
#include "kv.h"

namespace ibp {
namespace kv {

namespace {

// Order-preserving image of a score: NaN above everything, then by value; -0
// is +0.  0 is below every image.
__device__ __forceinline__ uint64_t score_key(double x) {
  if (x != x) return ~0ull;
  x += 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// The scored pages of a row at position pos: all of its pages but the first
// n_first and the last n_last, [lo, hi); last = its own page (-1: none).
struct Range {
  int32_t last, lo, hi;
};
__device__ __forceinline__ Range page_range(const Cache& cache, const Batch& b, const Seq& sq,
                                            int32_t pos, uint32_t n_first, uint32_t n_last) {
  Range r;
  pos = min(pos, sq.n_keys - 1);
  r.last = pos < 0 ? -1 : (int32_t)cache.page.div((uint32_t)pos);
  r.lo = min((int32_t)n_first, r.last + 1);
  r.hi = max(r.last + 1 - (int32_t)n_last, r.lo);
  return r;
}

// A wave per (row, key head, page): each lane four channels, summed over the
// lanes by butterflies.  A row that has no more than n_select pages needs no
// scores.
template <typename T>
__global__ __launch_bounds__(256) void k_kv_score(Cache cache, Batch b, const T* __restrict__ bounds,
                                                  uint32_t n_bounds, Rows q, uint32_t n_first,
                                                  uint32_t n_last, uint32_t n_select,
                                                  uint64_t* __restrict__ keys) {
  const uint32_t lane = threadIdx.x % kWave;
  const uint32_t r = blockIdx.x / cache.n_heads, h = blockIdx.x % cache.n_heads;
  const int32_t s = seq_of_row(b, (int32_t)r);
  if (s < 0) return;
  const Seq sq = load_seq(b, s);
  const int32_t i = (int32_t)r - sq.row0;
  if (i < 0 || i >= sq.q_len) return;
  const Range rg = page_range(cache, b, sq, sq.first + i, n_first, n_last);
  if (rg.last + 1 <= (int32_t)n_select) return;
  const uint32_t group = q.n_heads / cache.n_heads, hd = cache.head_dim;
  for (int32_t p = rg.lo + (int32_t)(blockIdx.y * 4 + threadIdx.x / kWave); p < rg.hi;
       p += (int32_t)gridDim.y * 4) {
    const int32_t id = b.table[(uint64_t)s * b.table_stride + p];
    uint64_t key = score_key(-INFINITY);
    if (id >= 0 && (uint32_t)id < n_bounds) {
      const T* lo = bounds + ((uint64_t)(uint32_t)id * cache.n_heads + h) * 2 * hd;
      double best = -INFINITY;
      for (uint32_t g = 0; g < group; ++g) {
        const T* x = (const T*)q.p + r * q.token_stride + (uint64_t)(h * group + g) * q.head_stride;
        double sum = 0.0;
        for (uint32_t c = lane; c < hd; c += kWave) {
          const double v = to_f32(x[c]);
          const double a = v * to_f32(lo[c]), d = v * to_f32(lo[hd + c]);
          sum += (a > d || a != a) ? a : d;
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d, kWave);
        if (sum > best || sum != sum) best = sum;
        if (best != best) break;
      }
      key = score_key(best);
    }
    if (lane == 0) keys[(uint64_t)blockIdx.x * b.max_pages + p] = key;
  }
}

// A workgroup per (row, key head): the need-th largest key by its bytes from
// the top (a histogram of the candidates that match so far), then the pages
// in order.
__global__ __launch_bounds__(256) void k_kv_pick(Cache cache, Batch b, uint32_t n_first,
                                                 uint32_t n_last, uint32_t n_select,
                                                 const uint64_t* __restrict__ keys,
                                                 int32_t* __restrict__ sel) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_digit, s_need, s_done;
  __shared__ uint32_t s_wave[2][4];
  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const uint32_t r = blockIdx.x / cache.n_heads;
  const int32_t s = seq_of_row(b, (int32_t)r);
  if (s < 0) return;
  const Seq sq = load_seq(b, s);
  const int32_t i = (int32_t)r - sq.row0;
  if (i < 0 || i >= sq.q_len) return;
  const Range rg = page_range(cache, b, sq, sq.first + i, n_first, n_last);
  int32_t* list = sel + (uint64_t)blockIdx.x * n_select;
  if (rg.last + 1 <= (int32_t)n_select) {
    for (uint32_t e = tid; e < n_select; e += 256) list[e] = (int32_t)e <= rg.last ? (int32_t)e : -1;
    return;
  }
  const uint64_t* mine = keys + (uint64_t)blockIdx.x * b.max_pages;
  const uint32_t forced = (uint32_t)(rg.last + 1 - (rg.hi - rg.lo));
  uint32_t need = n_select - forced;  // < hi - lo, since last + 1 > n_select
  uint64_t prefix = 0;
  int shift = 64;
  bool exact = false;  // every candidate that matches the prefix is taken
  while (need && shift > 0 && !exact) {
    shift -= 8;
    hist[tid] = 0;
    __syncthreads();
    for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += 256) {
      const uint64_t k = mine[p];
      if (shift == 56 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = need, d = 255;
      while (hist[d] < left) left -= hist[d--];
      s_digit = d;
      s_need = left;
      s_done = hist[d] == left;
    }
    __syncthreads();
    prefix = (prefix << 8) | s_digit;
    need = s_need;
    exact = s_done != 0;
    __syncthreads();
  }
  // candidates above the prefix, and the first `need` that equal it
  for (uint32_t e = tid; e < n_first; e += 256) list[e] = (int32_t)e;
  for (uint32_t e = tid; e < n_last; e += 256)
    list[n_select - n_last + e] = rg.last + 1 - (int32_t)n_last + (int32_t)e;
  uint32_t out = n_first, equal_before = 0;
  if (n_select == forced) return;
  for (int32_t base = rg.lo; base < rg.hi; base += 256) {
    const int32_t p = base + (int32_t)tid;
    const uint64_t k = p < rg.hi ? mine[p] >> shift : 0;
    const bool above = p < rg.hi && k > prefix, equal = p < rg.hi && k == prefix;
    const uint64_t be = __ballot(equal);
    if (lane == 0) s_wave[0][wave] = (uint32_t)__popcll(be);
    __syncthreads();
    uint32_t rank = equal_before + (uint32_t)__popcll(be & ((1ull << lane) - 1ull));
    for (uint32_t w = 0; w < wave; ++w) rank += s_wave[0][w];
    for (uint32_t w = 0; w < 4; ++w) equal_before += s_wave[0][w];
    const bool take = above || (equal && rank < need);
    const uint64_t bt = __ballot(take);
    if (lane == 0) s_wave[1][wave] = (uint32_t)__popcll(bt);
    __syncthreads();
    uint32_t at = out + (uint32_t)__popcll(bt & ((1ull << lane) - 1ull));
    for (uint32_t w = 0; w < wave; ++w) at += s_wave[1][w];
    for (uint32_t w = 0; w < 4; ++w) out += s_wave[1][w];
    if (take) list[at] = p;
    __syncthreads();
  }
}

template <typename T>
hipError_t run_select(const Cache& c, const Batch& b, const void* bounds, uint32_t n_bounds,
                      const Rows& q, uint32_t n_first, uint32_t n_last, uint32_t n_select,
                      int32_t* sel, uint64_t* keys, hipStream_t s) {
  const uint32_t items = b.n_rows * c.n_heads;
  if (b.max_pages > n_select) {
    const uint32_t y = (b.max_pages + 63) / 64;
    hipLaunchKernelGGL(k_kv_score<T>, dim3(items, y < 64 ? y : 64), dim3(256), 0, s, c, b,
                       (const T*)bounds, n_bounds, q, n_first, n_last, n_select, keys);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_kv_pick, dim3(items), dim3(256), 0, s, c, b, n_first, n_last, n_select, keys,
                     sel);
  return hipGetLastError();
}

}  // namespace

uint64_t select_workspace(const Cache& c, const Batch& b, uint32_t n_select) {
  return b.max_pages > n_select ? (uint64_t)b.n_rows * c.n_heads * b.max_pages * 8 : 0;
}

hipError_t launch_select(const Cache& c, uint32_t dtype, const Batch& b, const void* bounds,
                         uint32_t n_bounds, const Rows& q, uint32_t n_first, uint32_t n_last,
                         uint32_t n_select, int32_t* sel, void* workspace, hipStream_t s) {
  if (b.n_rows == 0 || b.n_seqs == 0) return hipSuccess;
  return dtype == IBP_KV_F16
             ? run_select<_Float16>(c, b, bounds, n_bounds, q, n_first, n_last, n_select, sel,
                                    (uint64_t*)workspace, s)
             : run_select<__bf16>(c, b, bounds, n_bounds, q, n_first, n_last, n_select, sel,
                                  (uint64_t*)workspace, s);
}

}  // namespace kv
}  // namespace ibp
