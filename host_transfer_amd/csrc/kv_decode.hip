// kv_decode.hip -- attention of few rows that share their keys: one new token
// (or a few) of a sequence with the query heads of one key head, over the
// whole cache or over the row's selected pages.
#include <algorithm>

#include "ibp_device.h"
#include "kv_mfma.h"

namespace ibp {
namespace kv {

namespace {

constexpr int kTile = 32;                // keys of a wave's step
constexpr int kWaves = 4;

// A workgroup per (up to 16 rows that share a key head, split of their keys).
// Its four waves take 32 keys at a time, in turn, each with a running
// maximum and sum of its own; nothing is shared until the end, so no wave waits
// for another.
//
// Bound by the reading of K and V: 4 * D bytes a key against 4 * D * 16
// operations of the matrix cores, 1/10 of their rate at the rate of HBM, so
// that empty columns (a group smaller than 16 rows) cost nothing.  Neighbouring lanes read
// neighbouring pieces of a row, K as well as V: a load of 64 pieces then touches 8 lines.  (With K in
// the first product's own order, 16 rows side by side, each load looked up 64, and the L1's
// lookups bound what comes from L2: lists of 280 rows 196 against 155 us in all; from HBM
// 300 against 291.)  Both pass through LDS, its wave's own part, K first, then V in its place:
// the first product reads rows, the second one transposed.  LDS rows are padded by
// 32 B: the eight rows that half a wave reads then lie in eight different 32 B
// windows of the banks for every head_dim that is a multiple of 32.
//
// Measured (with the join): 20 sequences of up to 2,048 tokens, 40 heads (814 MB) 158 us, 5.2 TB/s;
// 4 sequences of up to 131,072 tokens, 32 query heads on 8 key heads (1.61 GB) 292 us, 5.5 TB/s, as
// a large copy runs; 8 rows' lists of 2,048 tokens (67 MB) 22 us.  Lists come from L2 more than from HBM
// and want three waves a SIMD (280 rows' lists 133 us in all with three, 155 with two, 172
// with four, which spill); whole contexts two (131,072 tokens 291 us, 300 with three).  Loads of the next
// tile issued while this one is computed made both slower (160 and 295 us).
template <typename T, int DP, bool kSelected, int kHeads>
__global__ __launch_bounds__(256, kSelected && DP <= 128 ? 3 : 1) void k_kv_decode(
    Cache cache, Batch b, Rows q, Rows out, const int32_t* __restrict__ sel, uint32_t n_select,
    float scale_log2, uint32_t window, bool causal, uint32_t row_tiles, Partial part,
    float* __restrict__ lse) {
  constexpr int KS = DP / 32;   // products of the scores
  constexpr int DT = DP / 16;   // tiles of the output
  constexpr int LD = DP + 16;   // LDS row, elements
  constexpr int CH = DP / 8;    // 16 B pieces of a row
  constexpr int RPL = kWave / CH, NL = kTile / RPL;  // rows of a load, loads of a tile
  constexpr int WORDS = kTile * LD / 2;  // of a wave; 16 rows of DP floats fit
  static_assert(16 * DP <= WORDS, "the end's exchange fits the V tiles");
  constexpr int kTurns = kWaves / kHeads;           // waves that share a key head
  constexpr int kBlockKeys = kTile * kTurns;
  __shared__ __align__(16) uint32_t s_v[kWaves][WORDS];
  __shared__ float s_m[kWaves][16], s_z[kWaves][16];

  const uint32_t lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
  const uint32_t col = lane % 16, quarter = lane / 16;
  const uint32_t group = q.n_heads / cache.n_heads;
  const uint32_t hd = cache.head_dim;

  // block -> (sequence or row, row tile, split, key head), heads innermost: the
  // heads of a token lie side by side in memory
  uint32_t u = blockIdx.x;
  const uint32_t head_blocks = cache.n_heads / kHeads;
  const uint32_t kh = u % head_blocks * kHeads + wave % kHeads;
  u /= head_blocks;
  const uint32_t split = u % part.splits;
  u /= part.splits;
  const uint32_t tile = u % row_tiles;
  u /= row_tiles;

  int32_t s = (int32_t)u, i0 = 0;
  if (kSelected) {
    s = seq_of_row(b, (int32_t)u);
    if (s < 0) return;
  }
  const Seq sq = load_seq(b, (uint32_t)s);
  if (kSelected) {
    i0 = (int32_t)u - sq.row0;
    if (i0 < 0 || i0 >= sq.q_len) return;
  }
  // rows of this tile: m = i * group + g, [m0, m1)
  const uint32_t n_m = (kSelected ? 1u : (uint32_t)max(sq.q_len, 0)) * group;
  const uint32_t m0 = tile * 16;
  if (m0 >= n_m) return;
  const uint32_t m1 = min(m0 + 16, n_m);
  const bool have = m0 + col < m1;
  const uint32_t m = have ? m0 + col : m1 - 1;
  const int32_t i = i0 + (int32_t)(m / group);
  const uint32_t head = kh * group + m % group;
  const uint32_t row = (uint32_t)(sq.row0 + i);

  // keys that this lane's row sees, [lo, hi), and those that any row of the tile sees
  const int32_t pos = max(sq.first + i, -1);
  const int32_t pos_a = max(sq.first + i0 + (int32_t)(m0 / group), -1);
  const int32_t pos_e = max(sq.first + i0 + (int32_t)((m1 - 1) / group), -1);
  const int32_t w = (int32_t)window;
  const int32_t lo = w ? max(pos - w + 1, 0) : 0;
  const int32_t hi = causal ? min(pos + 1, sq.n_keys) : sq.n_keys;
  const int32_t lo_a = w ? max(pos_a - w + 1, 0) : 0;   // least lo
  const int32_t lo_e = w ? max(pos_e - w + 1, 0) : 0;   // greatest
  const int32_t hi_a = causal ? min(pos_a + 1, sq.n_keys) : sq.n_keys;  // least hi
  const int32_t hi_e = causal ? min(pos_e + 1, sq.n_keys) : sq.n_keys;  // greatest

  // the split's keys, whole tiles of the workgroup (virtual keys where pages are listed)
  const int32_t from = kSelected ? 0 : lo_a / kBlockKeys * kBlockKeys;
  const int32_t to = kSelected ? (int32_t)(n_select * cache.page.d) : hi_e;
  const int32_t tiles = max(to - from + kBlockKeys - 1, 0) / kBlockKeys;
  const int32_t per = (tiles + (int32_t)part.splits - 1) / (int32_t)part.splits;
  const int32_t begin = from + min((int32_t)split * per, tiles) * kBlockKeys;
  const int32_t end = min(from + min(((int32_t)split + 1) * per, tiles) * kBlockKeys, to);

  const T* qp = (const T*)q.p + row * q.token_stride + (uint64_t)head * q.head_stride;
  const T* zeros = (const T*)zero_row;
  V8<T> qf[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const uint32_t c = (k * 4 + quarter) * 8;
    qf[k] = load_row8(have && c < hd ? qp + c : zeros);
  }

  f32x4 o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  float top = -INFINITY, z = 0.f;

  const int32_t* table = b.table + (uint64_t)s * b.table_stride;
  const int32_t* list = kSelected ? sel + ((uint64_t)row * cache.n_heads + kh) * n_select : nullptr;
  const T* kbase = (const T*)cache.k + (uint64_t)kh * cache.head_stride;
  const T* vbase = (const T*)cache.v + (uint64_t)kh * cache.head_stride;
  T* sv = (T*)s_v[wave];

  // where key t0 + lane % 32 lies (elements); bit r of the result: some row sees key t0 + r
  auto locate = [&](int32_t t0, uint64_t& at) -> uint32_t {
    int32_t j = t0 + (int32_t)(lane % kTile);
    bool see = j < end;
    if (kSelected) {
      int32_t pg = -1;
      uint32_t e = 0;
      if (see) {
        e = cache.page.div((uint32_t)j);
        pg = list[e];
        if (e > 0 && list[e - 1] >= pg) pg = -1;
      }
      see = pg >= 0 && (uint32_t)pg < b.max_pages;
      j = see ? pg * (int32_t)cache.page.d + (j - (int32_t)(e * cache.page.d)) : 0;
    }
    see = see && j >= lo_a && j < hi_e;
    int32_t id = -1;
    uint32_t page = 0;
    if (see) {
      page = cache.page.div((uint32_t)j);
      id = table[page];
    }
    see = id >= 0 && (uint32_t)id < cache.n_pages;
    at = see ? (uint64_t)(uint32_t)id * cache.page_stride +
                   (uint64_t)((uint32_t)j - page * cache.page.d) * cache.token_stride
             : 0;
    return (uint32_t)__ballot(see);
  };
  // this lane's piece of row load_row + i * RPL: its offset (elements) from the pool's base
  const uint32_t load_row = lane / CH, load_c = lane % CH * 8;
  auto offset = [&](uint64_t at, int i) -> uint64_t {
    const int r = (int)load_row + i * RPL;
    return (((uint64_t)(uint32_t)__shfl((int)(uint32_t)(at >> 32), r) << 32) |
            (uint32_t)__shfl((int)(uint32_t)at, r)) + load_c;
  };
  auto loads = [&](uint32_t there, int i) {  // whether that row is there and has this piece
    return ((there >> (load_row + i * RPL)) & 1u) && load_c < hd;
  };
  T* put_at = sv + load_row * LD + load_c;
  const T* k_at = sv + col * LD + quarter * 8;
  // this lane's part of a transposed read of V
  const T* tr_at = sv + (4 * quarter + col / 4) * LD + 4 * (col % 4);
  bool odd = false;  // values that only some rows see and that are no numbers were left out

  for (int32_t t0 = begin + (int32_t)(wave / kHeads) * kTile; t0 < end; t0 += kBlockKeys) {
    V8<T> kf[NL], vf[NL];
    uint64_t at;
    const uint32_t there = locate(t0, at);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint64_t from_base = offset(at, i);
      const bool on = loads(there, i);
      kf[i] = load_row8(on ? kbase + from_base : zeros);
      vf[i] = load_row8(on ? vbase + from_base : zeros);
    }
    // every row sees every key of the tile?  (in lists, one row: `see` said all of it)
    bool plain = there == ~0u;
    if (!kSelected) plain = plain && t0 >= lo_e && t0 + kTile <= hi_a;

    // K to LDS, row = key of the tile
#pragma unroll
    for (int i = 0; i < NL; ++i) *(V8<T>*)(put_at + i * RPL * LD) = kf[i];
    wave_sync();
    f32x4 sc[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      sc[a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k)
        sc[a] = mfma16(*(const V8<T>*)(k_at + a * 16 * LD + k * 32), qf[k], sc[a]);
    }
    settle(sc[0], sc[1]);
    if (!kSelected && !plain) {  // (a list has one row: what it does not see is zeros)
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int32_t j = t0 + (int32_t)load_row + i * RPL;
        if (j < lo_e || j >= hi_a) {
          odd = odd || any_odd<T>(vf[i]);
          vf[i] = finite_part<T>(vf[i]);
        }
      }
    }
    // V in its place
    wave_sync();
#pragma unroll
    for (int i = 0; i < NL; ++i) *(V8<T>*)(put_at + i * RPL * LD) = vf[i];

    // lane's scores: keys t0 + 16 a + 4 quarter + r of its column's row
    float x[8];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int r = 0; r < 4; ++r) x[a * 4 + r] = sc[a][r] * scale_log2;
    if (!plain) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t kk = 4 * quarter + r;
          bool see = (there >> (a * 16 + kk)) & 1u;
          if (!kSelected) {
            const int32_t j = t0 + a * 16 + (int32_t)kk;
            see = see && j >= lo && j < hi;
          }
          if (!see) x[a * 4 + r] = -INFINITY;
        }
    }
    float most = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                       fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    most = max_half(max_quarter(most));
    // (any new maximum: its weight is then 2^kLift and rounds to itself, which is worth more here
    // than a rescaling; outputs in bf16 are off by 1.8e-3 instead of 2.1e-3)
    if (__any(most > top + Base<T>::kLift)) {
      const float next = next_base<T>(top, most);
      const float keep = exp2_raw(top - (next == -INFINITY ? 0.f : next));
      z *= keep;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[t][r] *= keep;
      top = next;
    }
    const float base = top == -INFINITY ? 0.f : top;
    V8<T> p;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
// (the product rounded as the base was: the largest of huge scores, too, is the base itself)
#pragma clang fp contract(off)
      const float y = exp2_raw(x[e] - base);
      z += y;
      p[e] = (T)y;  // half a step of the dtype, relative, as the output's own rounding
    }
    wave_sync();
#pragma unroll
    for (int t = 0; t < DT; ++t)
      o[t] = mfma16(join<T>(read_tr(tr_at + t * 16), read_tr(tr_at + t * 16 + 16 * LD)), p, o[t]);
    wave_sync();
  }

  settle(o);
  const bool all = __any(probe(o) != 0.f);  // (of every tile, else of those that some rows do not see)
  if (all || __any(odd)) {
    for (int32_t t0 = begin + (int32_t)(wave / kHeads) * kTile; t0 < end; t0 += kBlockKeys) {
      if (!all && t0 >= lo_e && t0 + kTile <= hi_a) continue;
      V8<T> sees;
      uint64_t at;
      const uint32_t there = locate(t0, at);
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int32_t mine = t0 + (int32_t)load_row + i * RPL;
        const bool some = all || mine < lo_e || mine >= hi_a;
        const uint64_t from_base = offset(at, i);
        *(V8<T>*)(put_at + i * RPL * LD) =
            odd_code<T>(load_row8(some && loads(there, i) ? vbase + from_base : zeros));
      }
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int32_t j = t0 + a * 16 + (int32_t)(4 * quarter) + r;
          bool see = (there >> (a * 16 + 4 * quarter + r)) & 1u;
          if (!kSelected) see = see && j >= lo && j < hi;
          sees[a * 4 + r] = (T)(see ? 1.f : 0.f);
        }
      wave_sync();
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        f32x4 n = f32x4{0.f, 0.f, 0.f, 0.f};
        n = mfma16(join<T>(read_tr(tr_at + t * 16), read_tr(tr_at + t * 16 + 16 * LD)), sees, n);
        settle(n);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[t][r] = add_odd(o[t][r], n[r]);
      }
      wave_sync();
    }
  }

  // the four waves' results together: rows of DP floats in the V tiles
  z = sum_half(sum_quarter(z));
  float* so = (float*)s_v[wave];
#pragma unroll
  for (int t = 0; t < DT; ++t) *(f32x4*)(so + col * DP + t * 16 + quarter * 4) = o[t];
  if (quarter == 0) {
    s_m[wave][col] = top;
    s_z[wave][col] = z;
  }
  __syncthreads();
  // a row of a head to 16 / kHeads threads; the head's waves are mine, mine + kHeads, ...
  constexpr uint32_t kOf = 256 / kHeads, kRowThreads = kOf / 16;
  const uint32_t mine = threadIdx.x / kOf, r = threadIdx.x % kOf / kRowThreads;
  const uint32_t first_c = threadIdx.x % kRowThreads;
  if (m0 + r >= m1) return;
  float mm = s_m[mine][r];
#pragma unroll
  for (int a = 1; a < kTurns; ++a) mm = fmaxf(mm, s_m[mine + a * kHeads][r]);
  float f[kTurns], zz = 0.f;
#pragma unroll
  for (int a = 0; a < kTurns; ++a) {
    f[a] = exp2_raw(s_m[mine + a * kHeads][r] - (mm == -INFINITY ? 0.f : mm));
    zz += f[a] * s_z[mine + a * kHeads][r];
  }
  const uint32_t rm = m0 + r;
  const uint32_t rrow = (uint32_t)(sq.row0 + i0) + rm / group;
  const uint32_t rhead = (kh - wave % kHeads + mine) * group + rm % group;
  const uint64_t unit = (uint64_t)rrow * q.n_heads + rhead;
  const bool whole = part.splits == 1;
  const float inv = zz == 0.f ? 0.f : 1.f / zz;
  T* op = (T*)out.p + rrow * out.token_stride + (uint64_t)rhead * out.head_stride;
  for (uint32_t c = first_c; c < hd / 8; c += kRowThreads) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = 0.f;
#pragma unroll
      for (int a = 0; a < kTurns; ++a) {
        const float x = ((const float*)s_v[mine + a * kHeads])[r * DP + c * 8 + e];
        y[e] += kTurns == 1 ? x : scaled(x, f[a]);
      }
    }
    if (whole) {
      V8<T> v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = mean<T>(y[e], inv);
      *(V8<T>*)(op + c * 8) = v;
    } else {
      float* to_ = part.row(unit, split) + c * 8;
      *(f32x4*)to_ = f32x4{y[0], y[1], y[2], y[3]};
      *(f32x4*)(to_ + 4) = f32x4{y[4], y[5], y[6], y[7]};
    }
  }
  if (first_c == 0) {
    if (!whole) part.ms[unit * part.splits + split] = make_float2(mm, zz);
    else if (lse) lse[unit] = zz == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(zz)) * kLn2;
  }
}

// The splits of a row together, few of them (of chunks, many rows): 16, 32 or 64 lanes a (row,
// head), four channels each; every lane forms the factors by itself.
constexpr uint32_t kFewSplits = 8;

template <typename T>
__global__ __launch_bounds__(256) void k_kv_join_few(Batch b, Rows out, Partial part, uint32_t lanes,
                                                     float* __restrict__ lse) {
  const uint32_t per = 256 / lanes;
  const uint64_t units = (uint64_t)b.n_rows * out.n_heads;
  const uint64_t unit = (uint64_t)blockIdx.x * per + threadIdx.x / lanes;
  if (unit >= units) return;
  const uint32_t row = (uint32_t)(unit / out.n_heads), head = (uint32_t)(unit % out.n_heads);
  if (seq_of_row(b, (int32_t)row) < 0) return;
  const uint32_t c = threadIdx.x % lanes * 4;
  const bool live = c < part.head_dim;
  float2 x[kFewSplits];
  f32x4 y[kFewSplits];
  float mm = -INFINITY;
#pragma unroll
  for (uint32_t e = 0; e < kFewSplits; ++e) {
    if (e >= part.splits) break;
    x[e] = part.ms[unit * part.splits + e];
    y[e] = live ? *(const f32x4*)(part.row(unit, e) + c) : f32x4{0.f, 0.f, 0.f, 0.f};
    mm = fmaxf(mm, x[e].x);
  }
  const float base = mm == -INFINITY ? 0.f : mm;
  f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
  float z = 0.f;
#pragma unroll
  for (uint32_t e = 0; e < kFewSplits; ++e) {
    if (e >= part.splits) break;
    const float f = exp2_raw(x[e].x - base);
    z += f * x[e].y;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] += scaled(y[e][r], f);
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  if (live) {
    typedef T t4 __attribute__((ext_vector_type(4)));
    t4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = mean<T>(o[r], inv);
    *(t4*)((T*)out.p + row * out.token_stride + (uint64_t)head * out.head_stride + c) = v;
  }
  if (lse && c == 0) lse[unit] = z == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(z)) * kLn2;
}

// The splits of a row together, many of them: a workgroup per (row, head).  Each split's factor first, from
// the maxima; then 16, 32 or 64 lanes (four channels each) a split, as many splits at
// a time as the workgroup holds.
template <typename T, uint32_t kJoinThreads>
__global__ __launch_bounds__(kJoinThreads) void k_kv_join(Batch b, Rows out, Partial part, uint32_t lanes,
                                                 float* __restrict__ lse) {
  __shared__ float s_f[kMaxSplits];
  constexpr uint32_t NW = kJoinThreads / kWave;
  __shared__ float s_red[NW];
  __shared__ f32x4 s_o[kJoinThreads];
  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const uint64_t unit = blockIdx.x;
  const uint32_t row = (uint32_t)(unit / out.n_heads), head = (uint32_t)(unit % out.n_heads);
  if (seq_of_row(b, (int32_t)row) < 0) return;
  const float2* ms = part.ms + unit * part.splits;
  float2 x[kMaxSplits / kJoinThreads];
  float mm = -INFINITY;
#pragma unroll
  for (uint32_t a = 0; a < kMaxSplits / kJoinThreads; ++a) {
    const uint32_t e = tid + a * kJoinThreads;
    x[a] = e < part.splits ? ms[e] : make_float2(-INFINITY, 0.f);
    mm = fmaxf(mm, x[a].x);
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) mm = fmaxf(mm, __shfl_xor(mm, d, kWave));
  if (lane == 0) s_red[wave] = mm;
  __syncthreads();
  for (uint32_t w = 0; w < NW; ++w) mm = fmaxf(mm, s_red[w]);
  __syncthreads();
  const float base = mm == -INFINITY ? 0.f : mm;
  float z = 0.f;
#pragma unroll
  for (uint32_t a = 0; a < kMaxSplits / kJoinThreads; ++a) {
    const uint32_t e = tid + a * kJoinThreads;
    const float f = exp2_raw(x[a].x - base);
    if (e < part.splits) {
      s_f[e] = f;
      z += f * x[a].y;
    }
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) z += __shfl_xor(z, d, kWave);
  if (lane == 0) s_red[wave] = z;
  __syncthreads();
  z = 0.f;
  for (uint32_t w = 0; w < NW; ++w) z += s_red[w];
  const uint32_t c = (tid % lanes) * 4;
  const uint32_t at_once = kJoinThreads / lanes;
  f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
  if (c < part.head_dim) {
#pragma unroll 4
    for (uint32_t e = tid / lanes; e < part.splits; e += at_once) {
      const float f = s_f[e];
      const f32x4 y = *(const f32x4*)(part.row(unit, e) + c);
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] += scaled(y[r], f);
    }
  }
  s_o[tid] = o;
  __syncthreads();
  for (uint32_t half = kJoinThreads / 2; half >= lanes; half /= 2) {
    if (tid < half) {
      const f32x4 y = s_o[tid + half];
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] += y[r];
      s_o[tid] = o;
    }
    __syncthreads();
  }
  if (tid < lanes && c < part.head_dim) {
    const float inv = z == 0.f ? 0.f : 1.f / z;
    typedef T t4 __attribute__((ext_vector_type(4)));
    t4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = mean<T>(o[r], inv);
    *(t4*)((T*)out.p + row * out.token_stride + (uint64_t)head * out.head_stride + c) = v;
  }
  if (lse && tid == 0) lse[unit] = z == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(z)) * kLn2;
}

template <typename T, int DP, bool kSelected, int kHeads>
hipError_t run_decode(const AttendPlan& p, const Cache& c, const Batch& b, const Rows& q,
                      const Rows& out, const int32_t* sel, uint32_t n_select, float scale,
                      uint32_t window, bool causal, float* lse, Partial part, hipStream_t s) {
  hipLaunchKernelGGL((k_kv_decode<T, DP, kSelected, kHeads>), dim3((uint32_t)p.blocks), dim3(256), 0, s, c,
                     b, q, out, sel, n_select, scale * kLog2e, window, causal, p.row_tiles, part, lse);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const AttendPlan& p, const Cache& c, uint32_t dtype, const Batch& b,
                         const Rows& q, const Rows& out, const int32_t* sel, uint32_t n_select,
                         float scale, uint32_t window, bool causal, float* lse, Partial part,
                         hipStream_t s) {
#define IBP_KV_DECODE(T, DP, SEL, HEADS) \
  run_decode<T, DP, SEL, HEADS>(p, c, b, q, out, sel, n_select, scale, window, causal, lse, part, s)
#define IBP_KV_DECODE_T(T, SEL, HEADS)                                          \
  (c.head_dim <= 64    ? IBP_KV_DECODE(T, 64, SEL, HEADS)                       \
   : c.head_dim <= 128 ? IBP_KV_DECODE(T, 128, SEL, HEADS)                      \
                       : IBP_KV_DECODE(T, 256, SEL, HEADS))
#define IBP_KV_DECODE_S(T)                                                      \
  (sel            ? IBP_KV_DECODE_T(T, true, 1)                                 \
   : p.heads == 4 ? IBP_KV_DECODE_T(T, false, 4) : IBP_KV_DECODE_T(T, false, 1))
  return dtype == IBP_KV_F16 ? IBP_KV_DECODE_S(_Float16) : IBP_KV_DECODE_S(__bf16);
#undef IBP_KV_DECODE_S
#undef IBP_KV_DECODE_T
#undef IBP_KV_DECODE
}

hipError_t launch_join(uint32_t dtype, const Batch& b, const Rows& out, Partial part, float* lse,
                       hipStream_t s) {
  const uint64_t units = (uint64_t)b.n_rows * out.n_heads;
  const uint32_t lanes = part.head_dim <= 64 ? 16 : part.head_dim <= 128 ? 32 : 64;
  // (11 splits of 800 rows and heads 5.8 us with 256 threads each, 10.6 with 1024; 256 splits of
  // 128 20 us with 256, 10 with 1024)
  const uint32_t threads = part.splits > 64 ? 1024 : 256;
  const bool few = part.splits <= kFewSplits;
  const uint32_t per = few ? 256 / lanes : 1;
  const dim3 grid((uint32_t)((units + per - 1) / per));
#define IBP_KV_JOIN(T)                                                                           \
  if (few)                                                                                       \
    hipLaunchKernelGGL(k_kv_join_few<T>, grid, dim3(256), 0, s, b, out, part, lanes, lse);       \
  else if (threads == 256)                                                                       \
    hipLaunchKernelGGL((k_kv_join<T, 256>), grid, dim3(256), 0, s, b, out, part, lanes, lse);    \
  else                                                                                           \
    hipLaunchKernelGGL((k_kv_join<T, 1024>), grid, dim3(1024), 0, s, b, out, part, lanes, lse);
  if (dtype == IBP_KV_F16) {
    IBP_KV_JOIN(_Float16)
  } else {
    IBP_KV_JOIN(__bf16)
  }
#undef IBP_KV_JOIN
  return hipGetLastError();
}

}  // namespace kv
}  // namespace ibp
