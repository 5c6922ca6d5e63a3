// kv_select.hip -- the pages each row and key head attends: a score of every
// page from its key bounds, then the best pages.
#include "ibp_device.h"
#include "kv_mfma.h"

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

// A lane exchange inside rows of 16 lanes, as two 32-bit moves in the vector ALU.
template <int kCtrl, int kBanks>
__device__ __forceinline__ double dpp64(double old, double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x), o = (uint64_t)__double_as_longlong(old);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)u, kCtrl,
                                                            0xF, kBanks, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)(o >> 32),
                                                            (int)(uint32_t)(u >> 32), kCtrl, 0xF,
                                                            kBanks, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// x of lane l ^ D
template <int D>
__device__ __forceinline__ double xor_lane(double x) {
  if constexpr (D == 1) return dpp64<0xB1, 0xF>(x, x);        // quad_perm 1,0,3,2
  if constexpr (D == 2) return dpp64<0x4E, 0xF>(x, x);        // quad_perm 2,3,0,1
  if constexpr (D == 4) {                                     // row_shl / row_shr by 4
    const double y = dpp64<0x104, 0x5>(x, x);                 // banks 0, 2: from l + 4
    return dpp64<0x114, 0xA>(y, x);                           // banks 1, 3: from l - 4
  }
  if constexpr (D == 8) return dpp64<0x128, 0xF>(x, x);       // row_ror by 8
  const uint64_t u = (uint64_t)__double_as_longlong(x);       // 16: the other row of a pair
  const auto a = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  const bool up = (__lane_id() & 16) != 0;
  const uint32_t lo = up ? a[0] : a[1], hi = up ? b[0] : b[1];
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double nan_max64(double a, double b) {
  return (b > a || b != b) ? b : a;
}

constexpr int kVecs = 4;          // query vectors (row, head) a wave scores at a time
constexpr int kScorePages = 256;  // pages of a workgroup
constexpr int kAhead = 3;         // steps that are in flight ahead of the one worked on

// Scores of 256 pages (64 a wave) for the vectors of a tile of rows: one row, or as many as
// make four vectors.  LP lanes hold a page's bounds, eight channels each, so that a
// wave reads 64 / LP pages at a time, whole lines, three steps ahead; the vectors stay in
// registers.  With m = hi + lo and r = hi - lo, max(q lo, q hi) is (q m + |q| r) / 2
// wherever all is finite: two fused multiply-adds a channel and vector, at the same rate in 64
// bits as in 32, with one register pair for q and its magnitude.  (Where the sum is not finite
// it is formed again as the definition has it.)  The order of the sum is the same for every
// page, so equal bounds have equal scores.  The four vectors' sums over LP lanes are
// folded together: two exchanges leave each quarter of the lanes with one vector, the rest
// are butterflies, all in the vector ALU.
//
// 64-bit sums decide which pages are read, so that the choice does not depend on the
// order of a 32-bit sum.
template <typename T, int LP>
__global__ __launch_bounds__(256, 2) void k_kv_score(Cache cache, Batch b, const T* __restrict__ bounds,
                                                     uint32_t n_bounds, Rows q, uint32_t n_first,
                                                     uint32_t n_last, uint32_t n_select,
                                                     uint32_t row_tiles, uint32_t rows_per_tile,
                                                     uint32_t page_blocks,
                                                     uint64_t* __restrict__ keys) {
  constexpr int PP = kWave / LP;  // pages at a time
  typedef V8<T> v8;
  const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
  const uint32_t c = lane % LP, sub = lane / LP;
  const uint32_t group = q.n_heads / cache.n_heads, hd = cache.head_dim;
  uint32_t u = blockIdx.x;
  const uint32_t h = u % cache.n_heads;
  u /= cache.n_heads;
  const uint32_t pb = u % page_blocks;
  u /= page_blocks;
  const uint32_t tile = u % row_tiles, s = u / row_tiles;
  const Seq sq = load_seq(b, s);
  const int32_t i0 = (int32_t)(tile * rows_per_tile);
  const int32_t n_i = min(sq.q_len - i0, (int32_t)rows_per_tile);
  if (n_i <= 0) return;
  // the pages that any row of the tile scores (later rows score as many or more)
  const Range rg = page_range(cache, b, sq, sq.first + i0 + n_i - 1, n_first, n_last);
  if (rg.last + 1 <= (int32_t)n_select) return;
  const int32_t p0 = (int32_t)(pb * kScorePages + wave * kWave);  // this wave's 64 pages
  const int32_t lo_p = max(p0, rg.lo), hi_p = min(p0 + kWave, rg.hi);
  if (lo_p >= hi_p) return;
  int32_t id = p0 + (int32_t)lane;  // of page p0 + lane; -1: no bounds
  id = id >= lo_p && id < hi_p ? b.table[(uint64_t)s * b.table_stride + id] : -1;
  if ((uint32_t)id >= n_bounds) id = -1;

  // which row's score a lane ends up with: the vectors of a row lie in all lanes of a page
  // (three or four), in its halves (two) or its quarters
  const uint32_t vi = ((c & (LP / 2)) ? 2u : 0u) + ((c & (LP / 4)) ? 1u : 0u);
  const uint32_t my_i = group >= 3 ? 0 : group == 2 ? vi / 2 : vi;
  const bool writes = c % (group >= 3 ? LP : group == 2 ? LP / 2 : LP / 4) == 0 && my_i < (uint32_t)n_i;
  const uint32_t my_row = (uint32_t)(sq.row0 + i0) + my_i;
  Range own = page_range(cache, b, sq, sq.first + i0 + (int32_t)my_i, n_first, n_last);
  if (!writes || own.last + 1 <= (int32_t)n_select) own.hi = own.lo;
  uint64_t* my_keys = keys + ((uint64_t)my_row * cache.n_heads + h) * b.max_pages;

  const bool live = c * 8 < hd;
  const T* base = bounds + (uint64_t)h * 2 * hd + c * 8;
  const uint64_t page_size = (uint64_t)cache.n_heads * 2 * hd;
  const int steps = (hi_p - p0 + PP - 1) / PP;

  for (uint32_t v0 = 0; v0 < group; v0 += kVecs) {  // one pass unless a row has more than four
    const uint32_t nv = min((uint32_t)kVecs, group * (uint32_t)n_i - v0);
    double x[kVecs][8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const uint32_t m = v0 + v;
      v8 y = {};
      if ((uint32_t)v < nv && live)
        y = load_row8((const T*)q.p + (uint64_t)((uint32_t)(sq.row0 + i0) + m / group) * q.token_stride +
                      (uint64_t)(h * group + m % group) * q.head_stride + c * 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] = (double)to_f32(y[e]);
    }
    v8 lo[kAhead], hi[kAhead];
    auto load = [&](int step, v8& a, v8& d) {
      const int32_t pid = __shfl(id, (step * PP + (int)sub) % kWave);
      const T* at = pid >= 0 && live ? base + (uint64_t)(uint32_t)pid * page_size : (const T*)zero_row;
      a = load_row8(at);
      d = load_row8(pid >= 0 && live ? at + hd : at);
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) load(a, lo[a], hi[a]);
    for (int step0 = 0; step0 < steps; step0 += kAhead) {
#pragma unroll
      for (int ah = 0; ah < kAhead; ++ah) {
        const int step = step0 + ah;
        if (step >= steps) break;
        const v8 la = lo[ah], ha = hi[ah];
        load(step + kAhead, lo[ah], hi[ah]);
        double a[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) a[v] = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double y = (double)to_f32(la[e]), z = (double)to_f32(ha[e]);
          const double m = z + y, r = z - y;
#pragma unroll
          for (int v = 0; v < kVecs; ++v) a[v] = fma(x[v][e], m, fma(fabs(x[v][e]), r, a[v]));
        }
        // lanes with bit LP/2 keep vectors 2, 3; of those, lanes with bit LP/4 the odd one
        auto fold = [&]() {
          const bool up = (lane & (LP / 2)) != 0, odd = (lane & (LP / 4)) != 0;
          const double k0 = (up ? a[2] : a[0]) + xor_lane<LP / 2>(up ? a[0] : a[2]);
          const double k1 = (up ? a[3] : a[1]) + xor_lane<LP / 2>(up ? a[1] : a[3]);
          double r = (odd ? k1 : k0) + xor_lane<LP / 4>(odd ? k0 : k1);
          if constexpr (LP >= 32) r += xor_lane<4>(r);
          if constexpr (LP >= 16) r += xor_lane<2>(r);
          r += xor_lane<1>(r);
          return r * 0.5;
        };
        double r = fold();
        if (__any(!isfinite(r))) {
#pragma unroll
          for (int v = 0; v < kVecs; ++v) {
            a[v] = 0.0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              a[v] += 2.0 * nan_max64(x[v][e] * (double)to_f32(la[e]), x[v][e] * (double)to_f32(ha[e]));
          }
          r = fold();
        }
        if (vi >= nv) r = -INFINITY;
        if (group >= 2) r = nan_max64(r, xor_lane<LP / 4>(r));
        if (group >= 3) r = nan_max64(r, xor_lane<LP / 2>(r));
        const int32_t page = p0 + step * PP + (int32_t)sub;
        const int32_t pid = __shfl(id, step * PP + (int)sub);
        if (page >= own.lo && page < own.hi) {
          uint64_t key = score_key(pid >= 0 ? r : -INFINITY);
          if (v0) {  // this lane wrote it in the pass before
            const uint64_t was = my_keys[page];
            key = key > was ? key : was;
          }
          my_keys[page] = key;
        }
      }
    }
  }
}

// A workgroup per (row, key head): the smallest key taken, found digit by digit
// (histograms of the candidates that agree so far), then the pages in order.  The
// keys are counted from the smallest one, so that the first digit already
// spreads them over its bins.
constexpr uint32_t kDigit = 11, kBins = 1u << kDigit;

template <int NT>
__global__ __launch_bounds__(NT) void k_kv_pick(Cache cache, Batch b, uint32_t n_first,
                                                uint32_t n_last, uint32_t n_select,
                                                const uint64_t* __restrict__ keys,
                                                int32_t* __restrict__ sel) {
  constexpr int NW = NT / kWave;
  constexpr int BPT = kBins / NT;  // bins of a thread
  __shared__ uint32_t hist[kBins];
  __shared__ uint64_t s_lo[NW], s_hi[NW];
  __shared__ uint32_t s_digit, s_need, s_count;
  __shared__ uint32_t s_wave[2][NW];
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
    for (uint32_t e = tid; e < n_select; e += NT) list[e] = (int32_t)e <= rg.last ? (int32_t)e : -1;
    return;
  }
  const uint64_t* mine = keys + (uint64_t)blockIdx.x * b.max_pages;
  for (uint32_t e = tid; e < n_first; e += NT) list[e] = (int32_t)e;
  for (uint32_t e = tid; e < n_last; e += NT)
    list[n_select - n_last + e] = rg.last + 1 - (int32_t)n_last + (int32_t)e;
  uint32_t need = n_select - n_first - n_last;  // < hi - lo, since last + 1 > n_select
  if (need == 0) return;

  uint64_t lo = ~0ull, hi = 0;
  for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += NT) {
    const uint64_t k = mine[p];
    lo = k < lo ? k : lo;
    hi = k > hi ? k : hi;
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint64_t a = (uint64_t)__shfl_xor((long long)lo, d), e = (uint64_t)__shfl_xor((long long)hi, d);
    lo = a < lo ? a : lo;
    hi = e > hi ? e : hi;
  }
  if (lane == 0) {
    s_lo[wave] = lo;
    s_hi[wave] = hi;
  }
  __syncthreads();
  for (int w = 0; w < NW; ++w) {
    lo = s_lo[w] < lo ? s_lo[w] : lo;
    hi = s_hi[w] > hi ? s_hi[w] : hi;
  }
  // keys less lo: `bits` bits; candidates: those whose bits from `shift` up equal `prefix`
  int shift = hi == lo ? 0 : 64 - __clzll((long long)(hi - lo));
  uint64_t prefix = 0;
  bool all = false;  // all candidates are taken
  while (shift > 0 && !all) {
    const int width = shift < (int)kDigit ? shift : (int)kDigit;
    const int next = shift - width;
#pragma unroll
    for (int e = 0; e < BPT; ++e) hist[tid * BPT + e] = 0;
    __syncthreads();
    for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += NT) {
      const uint64_t k = mine[p] - lo;
      if (shift == 64 || (k >> shift) == prefix)
        atomicAdd(&hist[(uint32_t)(k >> next) & ((1u << width) - 1u)], 1u);
    }
    __syncthreads();
    // the bin in which the need-th candidate from the top lies: counts above each thread's bins
    uint32_t own[BPT], sum = 0;
#pragma unroll
    for (int e = 0; e < BPT; ++e) sum += own[e] = hist[kBins - 1 - (tid * BPT + e)];
    const uint32_t incl = wave_inclusive_sum(sum);
    if (lane == kWave - 1) s_wave[0][wave] = incl;
    __syncthreads();
    uint32_t above = incl - sum;
    for (uint32_t w = 0; w < wave; ++w) above += s_wave[0][w];
#pragma unroll
    for (int e = 0; e < BPT; ++e) {
      if (above < need && need <= above + own[e]) {
        s_digit = kBins - 1 - (tid * BPT + e);
        s_need = need - above;
        s_count = own[e];
      }
      above += own[e];
    }
    __syncthreads();
    prefix = (prefix << width) | s_digit;
    need = s_need;
    all = s_count == need;
    shift = next;
  }
  // candidates above the prefix, and the first `need` that equal it
  uint32_t out = n_first, equal_before = 0;
  for (int32_t base = rg.lo; base < rg.hi; base += NT) {
    const int32_t p = base + (int32_t)tid;
    const uint64_t k = p < rg.hi ? mine[p] - lo : 0;
    const uint64_t top = shift == 64 ? 0 : k >> shift;
    const bool above = p < rg.hi && top > prefix, equal = p < rg.hi && top == prefix;
    const uint64_t be = __ballot(equal), ba = __ballot(above);
    if (lane == 0) {
      s_wave[0][wave] = (uint32_t)__popcll(be);
      s_wave[1][wave] = (uint32_t)__popcll(ba);
    }
    __syncthreads();
    // before this thread: `eq` equal ones, of which min(eq, need) are taken, and `ab` above
    uint32_t eq = equal_before + (uint32_t)__popcll(be & ((1ull << lane) - 1ull));
    uint32_t ab = (uint32_t)__popcll(ba & ((1ull << lane) - 1ull));
    uint32_t eq_all = equal_before, ab_all = 0;
    for (uint32_t w = 0; w < NW; ++w) {
      if (w < wave) {
        eq += s_wave[0][w];
        ab += s_wave[1][w];
      }
      eq_all += s_wave[0][w];
      ab_all += s_wave[1][w];
    }
    const uint32_t taken = min(eq, need) - min(equal_before, need);
    if (above || (equal && eq < need)) list[out + ab + taken] = p;
    out += ab_all + min(eq_all, need) - min(equal_before, need);
    equal_before = eq_all;
    __syncthreads();
  }
}

template <typename T>
hipError_t run_select(const Cache& c, const Batch& b, const void* bounds, uint32_t n_bounds,
                      const Rows& q, uint32_t n_first, uint32_t n_last, uint32_t n_select,
                      int32_t* sel, uint64_t* keys, hipStream_t s) {
  const uint32_t items = b.n_rows * c.n_heads;
  if (b.max_pages > n_select) {
    const uint32_t group = q.n_heads / c.n_heads;
    const uint32_t rows = group >= 3 ? 1 : kVecs / group;
    const uint32_t tiles = (b.max_q + rows - 1) / rows;
    const uint32_t page_blocks = (b.max_pages + kScorePages - 1) / kScorePages;
    const uint64_t blocks = (uint64_t)b.n_seqs * tiles * page_blocks * c.n_heads;
    if (blocks > 0x7FFFFFFFull) return hipErrorInvalidConfiguration;
#define IBP_KV_SCORE(LP)                                                                           \
  hipLaunchKernelGGL((k_kv_score<T, LP>), dim3((uint32_t)blocks), dim3(256), 0, s, c, b,           \
                     (const T*)bounds, n_bounds, q, n_first, n_last, n_select, tiles, rows,        \
                     page_blocks, keys)
    if (c.head_dim <= 64) IBP_KV_SCORE(8);
    else if (c.head_dim <= 128) IBP_KV_SCORE(16);
    else IBP_KV_SCORE(32);
#undef IBP_KV_SCORE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (b.max_pages <= 1024)
    hipLaunchKernelGGL(k_kv_pick<256>, dim3(items), dim3(256), 0, s, c, b, n_first, n_last, n_select,
                       keys, sel);
  else
    hipLaunchKernelGGL(k_kv_pick<1024>, dim3(items), dim3(1024), 0, s, c, b, n_first, n_last,
                       n_select, keys, sel);
  return hipGetLastError();
}

}  // namespace

uint64_t select_workspace(const Cache& c, const Batch& b, uint32_t n_select) {
  return b.max_pages > n_select ? (uint64_t)b.n_rows * c.n_heads * b.max_pages * 8 : 0;
}

hipError_t launch_select(const Cache& c, uint32_t dtype, const Batch& b, const void* bounds,
                         uint32_t n_bounds, const Rows& q, uint32_t n_first, uint32_t n_last,
                         uint32_t n_select, int32_t* sel, void* workspace, hipStream_t s) {
  if (b.n_rows == 0 || b.n_seqs == 0 || b.max_q == 0) return hipSuccess;
  return dtype == IBP_KV_F16
             ? run_select<_Float16>(c, b, bounds, n_bounds, q, n_first, n_last, n_select, sel,
                                    (uint64_t*)workspace, s)
             : run_select<__bf16>(c, b, bounds, n_bounds, q, n_first, n_last, n_select, sel,
                                  (uint64_t*)workspace, s);
}

}  // namespace kv
}  // namespace ibp
