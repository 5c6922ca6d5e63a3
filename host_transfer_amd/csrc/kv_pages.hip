// kv_pages.hip -- a step's page tables, slots and positions from the requests' lengths.
#include "kv_pages.h"
#include "kv_wave.h"

namespace ibp {
namespace kv {

namespace {

constexpr uint32_t kMostThreads = 1024; // of the workgroup that looks at the requests, one each
constexpr uint32_t kFewThreads = 256;   // of a step of at most as many requests and four times as many rows
constexpr uint32_t kOneRows = 4096;     // rows that this workgroup writes by itself
constexpr uint32_t kSearch = 4096;      // requests whose q_start a workgroup holds in LDS

// What the rows of a request need: page j < held is the request's own, later ones are
// free_pages[last - (j - held)]; its first new token is at position keep, -1 where it is not served.
struct Share {
  int32_t held, last, keep;
};

// Many pages that a request gives back: entries wanted .. wanted + n - 1.
struct Gift {
  uint32_t tid;
  int32_t wanted, n;
};

// Sums that stay at 2^32 - 1 where they would pass it: whatever is compared with them is smaller.
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Exclusive prefix sums over the workgroup's threads; the sums of all in `all`.
template <int N, uint32_t kThreads>
__device__ __forceinline__ void scan(uint32_t (&v)[N], uint32_t (&all)[N], uint32_t (*s)[2]) {
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint32_t before[N];  // of the wave's lanes before this one
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t x = wave_prefix(v[i], [](uint32_t a, uint32_t b) { return add_sat(a, b); });
    before[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x138, 0xf, 0xf, false);  // the lane before
    if (lane == kWave - 1) s[wave][i] = x;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t waves = 0, total = 0;
    for (uint32_t w = 0; w < kThreads / kWave; ++w) {
      const uint32_t y = s[w][i];
      if (w < wave) waves = add_sat(waves, y);
      total = add_sat(total, y);
    }
    v[i] = add_sat(waves, before[i]);
    all[i] = total;
  }
  __syncthreads();
}

__device__ __forceinline__ bool is_page(const PagePool& pool, int32_t id) {
  return id >= 0 && (uint32_t)id < pool.n_pages;
}

// A row's slot and position; the first token of a page that the request takes writes the table's entry.
__device__ __forceinline__ void place(const PagePool& pool, const ibp_kv_assigned& out, uint32_t r,
                                      int32_t s, int32_t i, const Share& share) {
  int64_t slot = -1, pos = -1;
  if (s >= 0 && share.keep >= 0) {
    const uint32_t at = (uint32_t)share.keep + (uint32_t)i, j = pool.page.div(at), in = at - j * pool.page.d;
    int32_t* entry = pool.table + (uint64_t)s * pool.table_stride + j;
    int32_t id;
    if ((int32_t)j < share.held) {
      id = *entry;
    } else {
      id = pool.free_pages[share.last - ((int32_t)j - share.held)];
      if (in == 0) *entry = id;
    }
    pos = at;
    if (is_page(pool, id)) slot = (int64_t)id * pool.page.d + in;
  }
  out.slots[r] = slot;
  if (out.positions) out.positions[r] = pos;
}

// The last s with start[s] <= r (start[0] = 0).
template <typename P>
__device__ __forceinline__ int32_t request_of(P start, uint32_t n, int32_t r) {
  int32_t lo = 0, hi = (int32_t)n;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (start[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One workgroup, a thread per request (some in turn where there are more): new tokens' rows and
// pages to give back and to take by prefix sums, and the ids given back to the stack.  What the
// stack holds in the end decides who is served, so the pages given back are counted for all requests
// first.  Where the step is small (kOne) the same workgroup then writes the rows, from LDS.
//
// Bound by its chain of loads and barriers (lengths, table entries, sums, stack, rows): 20 requests of one
// token 3.7 us, 250 with drafts, five of them ended, 8.2 (12.3 with sums through LDS in 64 bits), 64 with
// 123,000 rows 7.2 and 4 for the rows (2 MB).  One workgroup: sums over several would need a launch each.
template <bool kOne, uint32_t kThreads>
__global__ __launch_bounds__(kThreads) void k_kv_assign(PagePool pool, Step step, ibp_kv_assigned out,
                                                        Share* __restrict__ shares) {
  constexpr uint32_t kWaves = kThreads / kWave;
  __shared__ uint32_t s_sum[kWaves][2];
  __shared__ unsigned int s_unserved;
  __shared__ unsigned int s_taken;
  __shared__ Share s_share[kOne ? kThreads : 1];
  __shared__ int32_t s_start[kOne ? kThreads + 1 : 1];
  __shared__ Gift s_gift[kThreads];
  __shared__ uint32_t s_at[kThreads];
  __shared__ unsigned int s_ended;
  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const uint32_t turns = (step.n_seqs + kThreads - 1) / kThreads;
  if (tid == 0) {
    s_unserved = 0;
    s_taken = 0;
  }
  const uint32_t count0 = (uint32_t)min(max(*step.free_count, 0), (int32_t)pool.n_pages);

  // request t * kThreads + tid, from its lengths and the rows before it
  int32_t had, keep, held, wanted;
  int64_t want;
  uint32_t rows[1], rows_all[1];
  bool fits;
  auto look = [&](uint32_t t, uint32_t rows_before) {
    const uint32_t s = t * kThreads + tid;
    const bool have = s < step.n_seqs;
    had = have ? max(step.had[s], 0) : 0;
    keep = have && step.keep ? min(max(step.keep[s], 0), had) : had;
    const int32_t add = have ? max(step.add[s], 0) : 0;
    want = (int64_t)keep + add;
    rows[0] = (uint32_t)add;
    scan<1, kThreads>(rows, rows_all, s_sum);
    rows[0] = add_sat(rows_before, rows[0]);
    fits = have && want <= (int64_t)IBP_KV_MAX_TOKENS && had <= (int32_t)IBP_KV_MAX_TOKENS &&
           add_sat(rows[0], (uint32_t)add) <= step.n_rows;
    held = fits && had ? (int32_t)pool.page.div((uint32_t)had - 1) + 1 : 0;
    wanted = fits && want ? (int32_t)pool.page.div((uint32_t)want - 1) + 1 : 0;
    held = min(held, (int32_t)pool.max_pages);
    fits = fits && wanted <= (int32_t)pool.max_pages;
  };
  // Pages that the request gives back, its entries from `wanted` on: up to kFew by its own thread, more
  // by the workgroup's waves in turn, kAtOnce entries in flight (`ended` lists those requests; five
  // of 500 pages one after another in their wave, 64 entries at a time, made a step of 250 requests take
  // 20 us where it takes 12).
  constexpr int32_t kFew = 4, kAtOnce = 4 * kWave;
  auto few = [&](uint32_t t, int32_t (&ids)[kFew], int32_t n) {
    const int32_t* row = pool.table + (uint64_t)(t * kThreads + tid) * pool.table_stride + wanted;
#pragma unroll
    for (int32_t j = 0; j < kFew; ++j) ids[j] = row[min(j, n - 1)];
  };
  auto gives = [&](uint32_t t) -> uint32_t {
    const int32_t n = fits ? max(held - wanted, 0) : 0;
    uint32_t some = 0;
    if (tid == 0) s_ended = 0;
    __syncthreads();
    if (n > kFew) {
      s_gift[atomicAdd(&s_ended, 1u)] = Gift{tid, wanted, n};
    } else if (n > 0) {
      int32_t ids[kFew];
      few(t, ids, n);
#pragma unroll
      for (int32_t j = 0; j < kFew; ++j) some += j < n && is_page(pool, ids[j]);
    }
    __syncthreads();
    for (uint32_t e = wave; e < s_ended; e += kWaves) {
      const Gift g = s_gift[e];
      const int32_t* row = pool.table + (uint64_t)(t * kThreads + g.tid) * pool.table_stride + g.wanted;
      uint32_t c = 0;
      for (int32_t j = (int32_t)lane; j < g.n; j += kAtOnce) {
        int32_t ids[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) ids[a] = j + a * kWave < g.n ? row[j + a * kWave] : -1;
#pragma unroll
        for (int a = 0; a < 4; ++a) c += is_page(pool, ids[a]);
      }
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) c += __shfl_xor(c, d);
      if (lane == 0) s_at[g.tid] = c;
    }
    __syncthreads();
    return n > kFew ? s_at[tid] : some;
  };
  // the same entries to the stack, from place `at` on
  auto give = [&](uint32_t t, uint32_t at) {
    at = min(at, 0x7FFFFFFFu);  // past the stack's end already: no sum with an entry's number passes 32 bits
    const int32_t n = fits ? max(held - wanted, 0) : 0;
    if (n > kFew) s_at[tid] = at;
    __syncthreads();
    if (n > 0 && n <= kFew) {
      int32_t ids[kFew];
      few(t, ids, n);
#pragma unroll
      for (int32_t j = 0; j < kFew; ++j)
        if (j < n && is_page(pool, ids[j])) {
          if (at < pool.n_pages) pool.free_pages[at] = ids[j];
          ++at;
        }
    }
    for (uint32_t e = wave; e < s_ended; e += kWaves) {
      const Gift g = s_gift[e];
      const int32_t* row = pool.table + (uint64_t)(t * kThreads + g.tid) * pool.table_stride + g.wanted;
      uint32_t to = s_at[g.tid];
      for (int32_t j = 0; j < g.n; j += kAtOnce) {
        int32_t ids[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int32_t k = j + a * kWave + (int32_t)lane;
          ids[a] = k < g.n ? row[k] : -1;
        }
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const uint64_t there = __ballot(is_page(pool, ids[a]));
          const uint32_t mine = to + (uint32_t)__builtin_popcountll(there & ((1ull << lane) - 1));
          if (is_page(pool, ids[a]) && mine < pool.n_pages) pool.free_pages[mine] = ids[a];
          to += (uint32_t)__builtin_popcountll(there);
        }
      }
    }
  };

  uint32_t rows_before = 0, given = 0, mine = 0;
  for (uint32_t t = 0; t < turns; ++t) {
    look(t, rows_before);
    rows_before = add_sat(rows_before, rows_all[0]);
    mine = gives(t);
    if (turns > 1) {
      uint32_t v[1] = {mine}, all[1];
      scan<1, kThreads>(v, all, s_sum);
      given = add_sat(given, all[0]);
    }
  }
  uint32_t pages_before[2] = {0, 0};  // given back, taken
  const uint32_t rows_total = rows_before;
  rows_before = 0;
  uint32_t avail = min(add_sat(count0, given), pool.n_pages);
  for (uint32_t t = 0; t < turns; ++t) {
    const uint32_t s = t * kThreads + tid;
    if (turns > 1) {
      look(t, rows_before);
      rows_before = add_sat(rows_before, rows_all[0]);
      mine = gives(t);
    }
    const uint32_t need = fits ? (uint32_t)max(wanted - held, 0) : 0;
    uint32_t v[2] = {mine, need}, all[2];
    scan<2, kThreads>(v, all, s_sum);
    if (turns == 1) avail = min(add_sat(count0, all[0]), pool.n_pages);
    const uint32_t upto = add_sat(add_sat(pages_before[1], v[1]), need);
    const bool served = fits && (need == 0 || upto <= avail);
    if (s < step.n_seqs) {
      Share share;
      share.held = held;
      share.last = served ? (int32_t)(avail - 1 - (upto - need)) : 0;
      share.keep = served ? keep : -1;
      if (kOne) {
        s_share[tid] = share;
        s_start[tid] = (int32_t)min(rows[0], step.n_rows);
      } else {
        shares[s] = share;
      }
      out.q_start[s] = (int32_t)min(rows[0], step.n_rows);
      out.kv_len[s] = served ? (int32_t)want : 0;
      out.length[s] = served ? (int32_t)want : had;
      if (!served) atomicAdd(&s_unserved, 1u);
      else if (need) atomicMax(&s_taken, upto);
    }
    give(t, add_sat(add_sat(count0, pages_before[0]), v[0]));
    pages_before[0] = add_sat(pages_before[0], all[0]);
    pages_before[1] = add_sat(pages_before[1], all[1]);
  }
  const int32_t end = (int32_t)min(rows_total, step.n_rows);
  __threadfence_block();
  __syncthreads();
  if (tid == 0) {
    out.q_start[step.n_seqs] = end;
    *out.free_count = (int32_t)(avail - s_taken);
    if (out.unserved) *out.unserved = (int32_t)s_unserved;
  }
  if (kOne) {
    for (uint32_t r = tid; r < step.n_rows; r += kThreads) {
      int32_t s = -1, i = 0;
      Share share = {0, 0, -1};
      if ((int32_t)r < end) {
        s = request_of(s_start, step.n_seqs, (int32_t)r);
        share = s_share[s];
        i = (int32_t)r - s_start[s];
      }
      place(pool, out, r, s, i, share);
    }
  }
}

// The rows of a large step, a thread each.
__global__ __launch_bounds__(256) void k_kv_assign_rows(PagePool pool, Step step, ibp_kv_assigned out,
                                                        const Share* __restrict__ shares) {
  __shared__ int32_t s_start[kSearch];
  const int32_t end = out.q_start[step.n_seqs];
  const bool held = step.n_seqs <= kSearch;
  if (held) {
    for (uint32_t s = threadIdx.x; s < step.n_seqs; s += 256) s_start[s] = out.q_start[s];
    __syncthreads();
  }
  for (uint64_t r = (uint64_t)blockIdx.x * 256 + threadIdx.x; r < step.n_rows; r += (uint64_t)gridDim.x * 256) {
    int32_t s = -1, i = 0;
    Share share = {0, 0, -1};
    if ((int32_t)r < end) {
      s = held ? request_of(s_start, step.n_seqs, (int32_t)r)
               : request_of(out.q_start, step.n_seqs, (int32_t)r);
      share = shares[s];
      i = (int32_t)r - (held ? s_start[s] : out.q_start[s]);
    }
    place(pool, out, (uint32_t)r, s, i, share);
  }
}

bool one_launch(uint32_t n_seqs, uint64_t n_rows) { return n_seqs <= kMostThreads && n_rows <= kOneRows; }

}  // namespace

uint64_t assign_workspace(uint32_t n_seqs, uint64_t n_rows) {
  return one_launch(n_seqs, n_rows) ? 0 : (uint64_t)n_seqs * sizeof(Share);
}

hipError_t launch_assign(const PagePool& pool, const Step& step, const ibp_kv_assigned& out,
                         void* workspace, hipStream_t s) {
  if (one_launch(step.n_seqs, step.n_rows)) {
    if (step.n_seqs <= kFewThreads && step.n_rows <= 4 * kFewThreads)
      hipLaunchKernelGGL((k_kv_assign<true, kFewThreads>), dim3(1), dim3(kFewThreads), 0, s, pool, step, out, nullptr);
    else
      hipLaunchKernelGGL((k_kv_assign<true, kMostThreads>), dim3(1), dim3(kMostThreads), 0, s, pool, step, out, nullptr);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_kv_assign<false, kMostThreads>), dim3(1), dim3(kMostThreads), 0, s, pool, step, out,
                     (Share*)workspace);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || step.n_rows == 0) return e;
  DeviceInfo di;
  if ((e = device_info(&di)) != hipSuccess) return e;
  const uint32_t want = (step.n_rows + 255) / 256, cap = (uint32_t)di.cus * 8;
  hipLaunchKernelGGL(k_kv_assign_rows, dim3(want < cap ? want : cap), dim3(256), 0, s, pool, step, out,
                     (const Share*)workspace);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace ibp
