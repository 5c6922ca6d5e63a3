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

// Lane exchanges inside rows of 16 lanes, in the vector ALU: x of lane l ^ D.
template <int kCtrl, int kBanks>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, kCtrl, 0xF, kBanks, false);
}
template <int D>
__device__ __forceinline__ uint32_t xor_lane(uint32_t x) {
  if constexpr (D == 1) return dpp<0xB1, 0xF>(x, x);  // quad_perm 1,0,3,2
  if constexpr (D == 2) return dpp<0x4E, 0xF>(x, x);  // quad_perm 2,3,0,1
  if constexpr (D == 4)                               // banks 0, 2: row_shl 4; 1, 3: row_shr 4
    return dpp<0x114, 0xA>(dpp<0x104, 0x5>(x, x), x);
  return dpp<0x128, 0xF>(x, x);                       // row_ror 8
}
template <int D>
__device__ __forceinline__ float max_lane(float x) {
  return fmaxf(x, __uint_as_float(xor_lane<D>(__float_as_uint(x))));
}
__device__ __forceinline__ double nan_max64(double a, double b) {
  return (b > a || b != b) ? b : a;
}

constexpr int kPages = 64;                     // pages of a wave
constexpr uint32_t kScorePages = 4 * kPages;   // of a workgroup

// The workspace of a call: per (row, key head) `pages` 32-bit scores, one bound of the
// terms' sum for every kPages of them, and room for exact scores' images.
struct Scores {
  float* s;
  float* mag;
  uint64_t* exact;
  uint32_t pages;  // a multiple of kScorePages
};

// Scores of 256 pages (64 a wave) in 32 bits, for as many rows of a key head as make 16
// vectors (a row's group padded to a power of two; a larger group in several passes), and the
// largest sum of the terms' magnitudes, from which k_kv_pick bounds the scores' error.
//
// With q split into its positive and negative part the score is a product of [hi, lo] rows
// with [q+, q-] columns for the matrix cores: max(q lo, q hi) = q+ hi + q- lo where all is
// finite, the rows read and passed through LDS as k_kv_decode does.  The magnitudes are the same
// product of absolute values.  So the bounds are read once, at the rate of memory, for
// 16 vectors: 8 rows of 32 heads over up to 4,096 pages (100 MB of bounds) 22 us, 280 rows that share two
// sequences' pages 26 us; with 16 pages' pieces side by side in a load 25 and 32 us; 64-bit sums of
// all pages in the vector ALU took 40 and 146 us.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_kv_score(Cache cache, Batch b, const T* __restrict__ bounds,
                                                  uint32_t n_bounds, Rows q, uint32_t n_first,
                                                  uint32_t n_last, uint32_t n_select,
                                                  uint32_t row_tiles, uint32_t padded_log2,
                                                  Scores out) {
  constexpr int KS = DP / 32;
  constexpr int CH = DP / 8, RPL = kWave / (2 * CH), NL = 16 / RPL;  // pieces of a bound; loads
  constexpr int LD = 2 * DP + 16;  // LDS row, elements (padded as k_kv_decode's)
  typedef V8<T> v8;
  __shared__ __align__(16) uint32_t s_rows[4][16 * LD / 2];
  const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
  const uint32_t col = lane % 16, quarter = lane / 16;
  const uint32_t group = q.n_heads / cache.n_heads, hd = cache.head_dim;
  uint32_t u = blockIdx.x;
  const uint32_t h = u % cache.n_heads;
  u /= cache.n_heads;
  const uint32_t blocks = out.pages / kScorePages;
  const uint32_t pb = u % blocks;
  u /= blocks;
  const uint32_t tile = u % row_tiles, s = u / row_tiles;
  const Seq sq = load_seq(b, s);
  const uint32_t rows_per_tile = 16u >> padded_log2;
  const int32_t i0 = (int32_t)(tile * rows_per_tile);
  const int32_t n_i = min(sq.q_len - i0, (int32_t)rows_per_tile);
  if (n_i <= 0) return;
  // the pages that any row of the tile scores (later rows score as many or more)
  const Range rg = page_range(cache, b, sq, sq.first + i0 + n_i - 1, n_first, n_last);
  if (rg.last + 1 <= (int32_t)n_select) return;
  const int32_t p0 = (int32_t)(pb * kScorePages + wave * kPages);
  if (p0 >= rg.hi || p0 + kPages <= rg.lo) return;

  const uint32_t i = min(col >> padded_log2, (uint32_t)n_i - 1), g = col & ((1u << padded_log2) - 1);
  const T* qrow = (const T*)q.p + (uint64_t)((uint32_t)(sq.row0 + i0) + i) * q.token_stride;
  const T* base = bounds + (uint64_t)h * 2 * hd;
  const T* zeros = (const T*)zero_row;
  const int32_t* table = b.table + (uint64_t)s * b.table_stride;
  const uint64_t page_size = (uint64_t)cache.n_heads * 2 * hd;
  const bool writes = g == 0 && (col >> padded_log2) < (uint32_t)n_i;
  const uint64_t item = (uint64_t)((uint32_t)(sq.row0 + i0) + i) * cache.n_heads + h;

  v8 qp[KS], qn[KS], qm[KS];  // q+, q-, -q-
  auto load_q = [&](uint32_t v0) {
    const uint32_t e = v0 + g < group ? v0 + g : 0;  // padding: a head twice
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint32_t c = (k * 4 + quarter) * 8;
      const v8 x = load_row8(c < hd ? qrow + (uint64_t)(h * group + e) * q.head_stride + c : zeros);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const bool neg = to_f32(x[r]) < 0.f;  // a NaN stays in q+
        qp[k][r] = neg ? (T)0.f : x[r];
        qn[k][r] = neg ? x[r] : (T)0.f;
        qm[k][r] = neg ? -x[r] : (T)0.f;
      }
    }
  };
  auto absolute = [](v8 x) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(v8, __builtin_bit_cast(u32x4, x) & 0x7FFF7FFFu);
  };
  // ids of the wave's pages first (lane = page), then two sets of 16 pages' bounds in flight
  int32_t id = p0 + (int32_t)lane;
  id = (int32_t)lane < kPages && id >= rg.lo && id < rg.hi ? table[id] : -1;
  const bool bounded = id >= 0 && (uint32_t)id < n_bounds;
  const uint64_t all_there = __ballot(bounded);
  // A page's row is [lo, hi]; neighbouring lanes read its neighbouring pieces (k_kv_decode says why),
  // which pass through LDS, the wave's own part, into the products' order.
  const uint32_t load_row = lane / (2 * CH), part = lane / CH % 2, load_c = lane % CH * 8;
  const bool live = load_c < hd;
  T* put_at = (T*)s_rows[wave] + load_row * LD + part * DP + load_c;
  const T* row_at = (const T*)s_rows[wave] + col * LD + quarter * 8;
  v8 x[2][NL];
  auto load = [&](int a) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int from = a * 16 + (int)load_row + i * RPL;
      const int32_t pid = __shfl(id, from);
      const bool has = (all_there >> from) & 1u;
      x[a % 2][i] = load_row8(has && live ? base + (uint64_t)(uint32_t)pid * page_size + part * hd + load_c
                                          : zeros);
    }
  };
  load(0);
  load_q(0);
  float most = 0.f;
#pragma unroll
  for (int a = 0; a < kPages / 16; ++a) {
    if (a + 1 < kPages / 16) load(a + 1);
#pragma unroll
    for (int i = 0; i < NL; ++i) *(v8*)(put_at + i * RPL * LD) = x[a % 2][i];
    wave_sync();
    const uint32_t there = (uint32_t)(all_there >> (16 * a));
    f32x4 sc, mag;
    for (uint32_t v0 = 0; v0 < group; v0 += 16) {  // one pass up to 16 heads a group
      if (group > 16) load_q(v0);
      f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f}, m = y;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const v8 lo = *(const v8*)(row_at + k * 32), hi = *(const v8*)(row_at + DP + k * 32);
        y = mfma16(hi, qp[k], y);
        m = mfma16(absolute(hi), qp[k], m);
        y = mfma16(lo, qn[k], y);
        m = mfma16(absolute(lo), qm[k], m);
      }
      settle(y, m);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // anything that is no number makes the magnitude infinite, and all scores are formed anew
        const float z = m[r] == m[r] && y[r] == y[r] ? m[r] : INFINITY;
        sc[r] = v0 ? fmaxf(sc[r], y[r]) : y[r];
        mag[r] = v0 ? fmaxf(mag[r], z) : z;
      }
    }
    wave_sync();
    // the largest over a row's vectors, in neighbouring columns
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (padded_log2 > 0) sc[r] = max_lane<1>(sc[r]), mag[r] = max_lane<1>(mag[r]);
      if (padded_log2 > 1) sc[r] = max_lane<2>(sc[r]), mag[r] = max_lane<2>(mag[r]);
      if (padded_log2 > 2) sc[r] = max_lane<4>(sc[r]), mag[r] = max_lane<4>(mag[r]);
      if (padded_log2 > 3) sc[r] = max_lane<8>(sc[r]), mag[r] = max_lane<8>(mag[r]);
      most = fmaxf(most, mag[r]);
      if (!((there >> (4 * quarter + r)) & 1u)) sc[r] = -INFINITY;
    }
    if (writes) *(f32x4*)(out.s + item * out.pages + p0 + a * 16 + 4 * quarter) = sc;
  }
  most = max_half(max_quarter(most));
  if (writes && quarter == 0) out.mag[item * (out.pages / kPages) + p0 / kPages] = most;
}

// A page's score as the definition has it, in 64 bits, by a wave: 2^lp_log2 lanes a head,
// eight channels each, as many heads at a time as that makes.  The order of the sum is the
// same for every page, so equal bounds have equal scores.
template <typename T>
__device__ __forceinline__ double exact_score(const T* __restrict__ lo, const T* q, uint64_t head_stride,
                                              uint32_t group, uint32_t hd, uint32_t lp_log2,
                                              uint32_t lane) {
  const uint32_t c = (lane & ((1u << lp_log2) - 1)) * 8, sub = lane >> lp_log2;
  const bool live = c < hd;
  const V8<T> l = load_row8(live ? lo + c : (const T*)zero_row);
  const V8<T> u = load_row8(live ? lo + hd + c : (const T*)zero_row);
  double best = -INFINITY;
  for (uint32_t g0 = 0; g0 < group; g0 += (uint32_t)kWave >> lp_log2) {
    const bool on = g0 + sub < group;
    const V8<T> x = load_row8(live && on ? q + (g0 + sub) * head_stride + c : (const T*)zero_row);
    double sum = 0.0;
    if (live && on)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double y = (double)to_f32(x[e]);
        sum += nan_max64(y * (double)to_f32(l[e]), y * (double)to_f32(u[e]));
      }
    for (uint32_t d = 1; d < 1u << lp_log2; d <<= 1) sum += __shfl_xor(sum, (int)d, kWave);
    if (on) best = nan_max64(best, sum);
  }
  for (uint32_t d = 1u << lp_log2; d < (uint32_t)kWave; d <<= 1)
    best = nan_max64(best, __shfl_xor(best, (int)d, kWave));
  return best;
}

// Order-preserving image of a 32-bit score (none is a NaN here).
__device__ __forceinline__ uint32_t score_key32(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// A workgroup per (row, key head).  The 32-bit scores are off by at most E = 2^-13 of the
// largest sum of magnitudes (up to 16 products of 32 terms, each of whose additions rounds,
// or cuts, to 2^-23: 2^-14) plus what a flushed result could be.  With T the need-th
// largest of them, the need-th largest exact score lies within E of T, so a page
// more than 2 E above T is taken and one more than 2 E below is not; the few between are
// scored exactly and the best of them taken.  Selections are digit searches: histograms
// of the candidates that agree in the digits so far, counted from the smallest one, so that
// the first digit already spreads them over its bins.
constexpr uint32_t kCachedPages = 12288;  // whose scores LDS holds: 48 KB beside 11.4
constexpr uint32_t kOpen = 256;            // open pages that are ranked one by one
constexpr uint32_t kDigit = 11, kBins = 1u << kDigit;

template <typename T, int NT, bool kCached>
__global__ __launch_bounds__(NT) void k_kv_pick(Cache cache, Batch b, const T* __restrict__ bounds,
                                                uint32_t n_bounds, Rows q, uint32_t n_first,
                                                uint32_t n_last, uint32_t n_select, Scores in,
                                                int32_t* __restrict__ sel) {
  constexpr int NW = NT / kWave;
  constexpr int BPT = kBins / NT;  // bins of a thread
  __shared__ uint32_t hist[kBins];
  __shared__ uint64_t s_lo[NW], s_hi[NW];
  __shared__ uint32_t s_digit, s_need, s_count;
  __shared__ uint32_t s_wave[2][NW];
  __shared__ uint32_t s_open;
  __shared__ uint64_t s_key[kOpen];
  __shared__ int32_t s_page[kOpen];
  extern __shared__ float s_cached[];  // kCached: the scores of pages rg.lo ..
  static_assert(!kCached || kCachedPages * sizeof(float) + sizeof(hist) + sizeof(s_lo) + sizeof(s_hi) +
                                    sizeof(s_wave) + sizeof(s_key) + sizeof(s_page) + 64 <= 65536,
                "the LDS that a workgroup has without asking for more");
  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const uint32_t r = blockIdx.x / cache.n_heads, h = blockIdx.x % cache.n_heads;
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
  float* score = in.s + (uint64_t)blockIdx.x * in.pages;
  const float* mags = in.mag + (uint64_t)blockIdx.x * (in.pages / kPages);
  uint64_t* exact = in.exact + (uint64_t)blockIdx.x * in.pages;
  for (uint32_t e = tid; e < n_first; e += NT) list[e] = (int32_t)e;
  for (uint32_t e = tid; e < n_last; e += NT)
    list[n_select - n_last + e] = rg.last + 1 - (int32_t)n_last + (int32_t)e;
  uint32_t need = n_select - n_first - n_last;  // < hi - lo, since last + 1 > n_select
  if (need == 0) return;

  // the smallest and largest of all threads' lo and hi, to all threads
  auto spread = [&](uint64_t& lo, uint64_t& hi) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const uint64_t x = (uint64_t)__shfl_xor((long long)lo, d), y = (uint64_t)__shfl_xor((long long)hi, d);
      lo = x < lo ? x : lo;
      hi = y > hi ? y : hi;
    }
    __syncthreads();
    if (lane == 0) {
      s_lo[wave] = lo;
      s_hi[wave] = hi;
    }
    __syncthreads();
    for (int w = 0; w < NW; ++w) {
      lo = s_lo[w] < lo ? s_lo[w] : lo;
      hi = s_hi[w] > hi ? s_hi[w] : hi;
    }
  };
  // The n-th largest of key(p) - lo where among(p), all of them below hi - lo + 1, down to a
  // digit where the candidates that agree are all taken, or are no more than `few`:
  // candidates whose bits from `shift` up are above `prefix` are taken, and n of those equal.
  auto search = [&](auto&& among, auto&& key, uint64_t lo, uint64_t hi, uint32_t few, uint32_t& n,
                    int& shift, uint64_t& prefix) {
    shift = hi == lo ? 0 : 64 - __clzll((long long)(hi - lo));
    prefix = 0;
    bool all = false;
    while (shift > 0 && !all) {
      const int width = shift < (int)kDigit ? shift : (int)kDigit;
      const int next = shift - width;
#pragma unroll
      for (int e = 0; e < BPT; ++e) hist[tid * BPT + e] = 0;
      __syncthreads();
      for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += NT) {
        if (!among(p)) continue;
        const uint64_t k = key(p) - lo;
        if (shift == 64 || (k >> shift) == prefix)
          atomicAdd(&hist[(uint32_t)(k >> next) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      // the bin in which the n-th candidate from the top lies: counts above each thread's bins
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
        if (above < n && n <= above + own[e]) {
          s_digit = kBins - 1 - (tid * BPT + e);
          s_need = n - above;
          s_count = own[e];
        }
        above += own[e];
      }
      __syncthreads();
      prefix = (prefix << width) | s_digit;
      n = s_need;
      all = s_count == n || s_count <= few;
      shift = next;
      __syncthreads();
    }
  };

  uint64_t lo32 = ~0ull, hi32 = 0;  // of the 32-bit scores' images
  for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += NT) {
    const float x = score[p];
    if (kCached) s_cached[p - rg.lo] = x;
    const uint64_t k = score_key32(x);
    lo32 = k < lo32 ? k : lo32;
    hi32 = k > hi32 ? k : hi32;
  }
  auto score_of = [&](int32_t p) { return kCached ? s_cached[p - rg.lo] : score[p]; };
  spread(lo32, hi32);

  // E, and the border of the 32-bit scores, or rather two values that it lies between: the ends
  // of a bin that holds few of them
  float mag = 0.f;
  for (int32_t e = rg.lo / kPages + (int32_t)tid; e <= (rg.hi - 1) / kPages; e += NT)
    mag = fmaxf(mag, mags[e]);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) mag = fmaxf(mag, __shfl_xor(mag, d, kWave));
  if (lane == 0) s_wave[0][wave] = __float_as_uint(mag);
  __syncthreads();
  for (int w = 0; w < NW; ++w) mag = fmaxf(mag, __uint_as_float(s_wave[0][w]));
  const bool numbers = mag < 1e38f;  // (a sum near the largest number may have passed it)
  float sure = INFINITY, maybe = -INFINITY;  // above `sure`: taken; from `maybe` up: perhaps
  if (numbers) {
    uint64_t prefix;
    uint32_t n = need;
    int shift;
    search([](int32_t) { return true; }, [&](int32_t p) { return (uint64_t)score_key32(score_of(p)); },
           lo32, hi32, 8, n, shift, prefix);
    auto value = [](uint64_t k) {
      return __uint_as_float((uint32_t)k >> 31 ? (uint32_t)k & 0x7FFFFFFFu : ~(uint32_t)k);
    };
    const uint64_t first = lo32 + (prefix << shift), last = lo32 + ((prefix + 1) << shift) - 1;
    const float e2 = 2.f * (mag * 0x1p-13f + 0x1p-100f);
    sure = value(last < hi32 ? last : hi32) + e2;
    maybe = value(first) - e2;
  }
  auto taken = [&](int32_t p) { return numbers && score_of(p) > sure; };
  auto open = [&](int32_t p) { return !numbers || (score_of(p) >= maybe && score_of(p) <= sure); };
  if (tid == 0) s_open = 0;
  __syncthreads();
  uint32_t n_taken = 0;
  for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += NT) {
    n_taken += taken(p);
    if (open(p)) {
      const uint32_t e = atomicAdd(&s_open, 1u);
      if (e < kOpen) s_page[e] = p;
    }
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) n_taken += __shfl_xor(n_taken, d, kWave);
  if (lane == 0) s_wave[0][wave] = n_taken;
  __syncthreads();
  n_taken = 0;
  for (int w = 0; w < NW; ++w) n_taken += s_wave[0][w];
  const uint32_t n_open = s_open;
  need -= n_taken;  // of the open ones; at least one, the border itself
  const uint32_t group = q.n_heads / cache.n_heads, hd = cache.head_dim;
  const uint32_t lp_log2 = hd <= 64 ? 3 : hd <= 128 ? 4 : 5;
  const T* qrow = (const T*)q.p + r * q.token_stride + (uint64_t)h * group * q.head_stride;
  const int32_t* table = b.table + (uint64_t)s * b.table_stride;
  auto exact_key = [&](int32_t p) {
    const int32_t id = table[p];
    double x = -INFINITY;
    if (id >= 0 && (uint32_t)id < n_bounds)
      x = exact_score(bounds + ((uint64_t)(uint32_t)id * cache.n_heads + h) * 2 * hd, qrow,
                      q.head_stride, group, hd, lp_log2, lane);
    return score_key(x);
  };
  int shift = 64;   // (64: all open ones are taken)
  uint64_t prefix = 0, lo = 0, hi = 0;
  bool listed = false;  // whether the open ones' 32-bit scores now say if they are taken
  if (n_open > need && n_open <= kOpen) {
    // few: each one's rank among them
    for (uint32_t e = wave; e < n_open; e += NW) {
      const uint64_t k = exact_key(s_page[e]);
      if (lane == 0) s_key[e] = k;
    }
    __syncthreads();
    if (tid < n_open) {
      const uint64_t k = s_key[tid];
      const int32_t p = s_page[tid];
      uint32_t rank = 0;
      for (uint32_t e = 0; e < n_open; ++e) rank += s_key[e] > k || (s_key[e] == k && s_page[e] < p);
      const float x = rank < need ? INFINITY : -INFINITY;
      if (kCached) s_cached[p - rg.lo] = x;
      else score[p] = x;
    }
    listed = true;
  } else if (n_open > need) {
    for (int32_t base = rg.lo + (int32_t)wave * kWave; base < rg.hi; base += NT) {
      const int32_t p = base + (int32_t)lane;
      for (uint64_t left = __ballot(p < rg.hi && open(p)); left; left &= left - 1) {
        const int32_t at = base + __builtin_ctzll(left);
        const uint64_t k = exact_key(at);
        if (lane == 0) exact[at] = k;
      }
    }
    __syncthreads();
    lo = ~0ull;
    for (int32_t p = rg.lo + (int32_t)tid; p < rg.hi; p += NT) {
      if (!open(p)) continue;
      const uint64_t k = exact[p];
      lo = k < lo ? k : lo;
      hi = k > hi ? k : hi;
    }
    spread(lo, hi);
    search(open, [&](int32_t p) { return exact[p]; }, lo, hi, 0, need, shift, prefix);
  }
  __syncthreads();
  // the taken, the open ones above the prefix, and the first `need` that equal it
  uint32_t out = n_first, equal_before = 0;
  for (int32_t base = rg.lo; base < rg.hi; base += NT) {
    const int32_t p = base + (int32_t)tid;
    bool above = p < rg.hi && (taken(p) || (listed && score_of(p) == INFINITY));
    bool equal = p < rg.hi && !listed && open(p);
    if (equal && shift < 64) {
      const uint64_t top = (exact[p] - lo) >> shift;
      above = top > prefix;
      equal = top == prefix;
    }
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
    const uint32_t before = min(eq, need) - min(equal_before, need);
    if (above || (equal && eq < need)) list[out + ab + before] = p;
    out += ab_all + min(eq_all, need) - min(equal_before, need);
    equal_before = eq_all;
    __syncthreads();
  }
}

uint32_t padded_pages(const Batch& b) {
  return (b.max_pages + kScorePages - 1) / kScorePages * kScorePages;
}

template <typename T>
hipError_t run_select(const Cache& c, const Batch& b, const void* bounds, uint32_t n_bounds,
                      const Rows& q, uint32_t n_first, uint32_t n_last, uint32_t n_select,
                      int32_t* sel, void* workspace, hipStream_t s) {
  const uint32_t items = b.n_rows * c.n_heads;
  if (items > 0xFFFFFFFFull / (b.max_pages <= 1024 ? 256 : 1024)) return hipErrorInvalidConfiguration;
  Scores sc = {nullptr, nullptr, nullptr, padded_pages(b)};
  if (b.max_pages > n_select) {
    sc.exact = (uint64_t*)workspace;
    sc.s = (float*)(sc.exact + (uint64_t)items * sc.pages);
    sc.mag = sc.s + (uint64_t)items * sc.pages;
    const uint32_t group = q.n_heads / c.n_heads;
    uint32_t padded_log2 = 0;
    while ((1u << padded_log2) < group && padded_log2 < 4) ++padded_log2;
    const uint32_t rows = 16u >> padded_log2;
    const uint32_t tiles = (b.max_q + rows - 1) / rows;
    uint64_t blocks = (uint64_t)b.n_seqs * tiles;  // (its factors: below 2^24, 2^23 and 2^16)
    if (blocks <= 0xFFFFFFull) blocks *= (uint64_t)(sc.pages / kScorePages) * c.n_heads;
    if (blocks > 0xFFFFFFull) return hipErrorInvalidConfiguration;
#define IBP_KV_SCORE(DP)                                                                            \
  hipLaunchKernelGGL((k_kv_score<T, DP>), dim3((uint32_t)blocks), dim3(256), 0, s, c, b,            \
                     (const T*)bounds, n_bounds, q, n_first, n_last, n_select, tiles, padded_log2, sc)
    if (c.head_dim <= 64) IBP_KV_SCORE(64);
    else if (c.head_dim <= 128) IBP_KV_SCORE(128);
    else IBP_KV_SCORE(256);
#undef IBP_KV_SCORE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#define IBP_KV_PICK(NT, CACHED)                                                                    \
  hipLaunchKernelGGL((k_kv_pick<T, NT, CACHED>), dim3(items), dim3(NT), CACHED ? b.max_pages * 4 : 0, \
                     s, c, b, (const T*)bounds, n_bounds, q, n_first, n_last, n_select, sc, sel)
  if (b.max_pages <= 1024) IBP_KV_PICK(256, true);
  else if (b.max_pages <= kCachedPages) IBP_KV_PICK(1024, true);
  else IBP_KV_PICK(1024, false);
#undef IBP_KV_PICK
  return hipGetLastError();
}

}  // namespace

uint64_t select_workspace(const Cache& c, const Batch& b, uint32_t n_select) {
  if (b.max_pages <= n_select) return 0;
  const uint64_t pages = padded_pages(b);
  return (uint64_t)b.n_rows * c.n_heads * (pages * 12 + pages / kPages * 4);
}

hipError_t launch_select(const Cache& c, uint32_t dtype, const Batch& b, const void* bounds,
                         uint32_t n_bounds, const Rows& q, uint32_t n_first, uint32_t n_last,
                         uint32_t n_select, int32_t* sel, void* workspace, hipStream_t s) {
  if (b.n_rows == 0 || b.n_seqs == 0 || b.max_q == 0) return hipSuccess;
  return dtype == IBP_KV_F16
             ? run_select<_Float16>(c, b, bounds, n_bounds, q, n_first, n_last, n_select, sel,
                                    workspace, s)
             : run_select<__bf16>(c, b, bounds, n_bounds, q, n_first, n_last, n_select, sel,
                                  workspace, s);
}

}  // namespace kv
}  // namespace ibp
