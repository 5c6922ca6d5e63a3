// kv8_decode.hip -- attention of few rows that share their keys over a cache in 8 bits: one new token
// (or a few) of a sequence with the query heads of one key head.
#include "kv8_attend.h"
#include "kv8_share.h"

namespace ibp {
namespace kv {

namespace {

constexpr int kTile = 32;   // keys of a wave's step
constexpr int kWaves = 4;
constexpr uint32_t kManyRows = 8192;  // as the GPU holds waves

// As k_kv_decode: a workgroup per (up to 16 NC rows that share a key head, split of their keys; all rows of
// a sequence), its four waves over four key heads of the same tokens or over one head's keys in turn, each with a
// running maximum and sum of its own.  A wave reads 32 keys' codes of K and of V at a time, neighbouring lanes
// neighbouring pieces of 16 codes, makes 16-bit rows of them in its registers (two codes an instruction,
// which applies the block's power of two too) and passes those through its own part of LDS, K first,
// then V in its place: the first product reads rows, the second one transposed.
//
// Where keys are shared out (plan.shares), each workgroup finds its part from all lengths by itself, in its
// first microsecond; one workgroup a sequence else.
//
// Bound by the reading of K and V, 2 * D bytes a key.  Measured (with the join): 20 sequences of up to
// 2,048 tokens, 40 heads (408 MB) 87 to 88 us, 4.7 TB/s; 4 sequences of up to 131,072 tokens, 32 query heads on 8
// key heads (806 MB) 151 to 156 us, 5.2 to 5.3 TB/s, as a large copy runs; 24 sequences of 5 tokens over 1,638 to
// 8,192 tokens (244 MB, two columns) 68 us.  Four workgroups a CU with one column (two 99 and 173 us for the
// first two; three, each with its next tile on the way, 95 and 168).
template <typename T, int DP, int kHeads, int NC>  // NC: columns of 16 rows
__global__ __launch_bounds__(256, decode8_groups(DP, NC)) void k_kv8_decode(
    Cache8 cache, Batch b, Rows q, Rows out, float scale_log2, uint32_t window, bool causal,
    Plan8 plan, float* __restrict__ lse) {
  constexpr int KS = DP / 32;   // products of the scores
  constexpr int DT = DP / 16;   // tiles of the output
  constexpr int LD = DP + 16;   // LDS row, elements
  constexpr int CH = DP / 16;   // 16 B pieces of a row of codes
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

  // block -> (its place among the head's workgroups, key head), heads innermost: the heads of a
  // token lie side by side in memory
  const uint32_t head_blocks = cache.n_heads / kHeads;
  const uint32_t kh = blockIdx.x % head_blocks * kHeads + wave % kHeads;
  const uint32_t place = blockIdx.x / head_blocks;
  const int32_t w = (int32_t)window;
  // keys that the first and the last row of a sequence see, [lo, hi); whole tiles of the workgroup
  auto first_lo = [&](const Seq& sq) { return w ? max(max(sq.first, -1) - w + 1, 0) : 0; };
  auto last_hi = [&](const Seq& sq) {
    return causal ? min(max(sq.first + sq.q_len - 1, -1) + 1, sq.n_keys) : sq.n_keys;
  };
  auto tiles_of = [&](const Seq& sq) {
    const int32_t from = first_lo(sq) / kBlockKeys * kBlockKeys;
    return max(last_hi(sq) - from + kBlockKeys - 1, 0) / kBlockKeys;
  };
  Part8 at_ = {(int32_t)place, 0, 1, 0};
  Seq sq;
  if (plan.shares) {
    // sequences past the first 64: their lengths where the rows of V will lie
    static_assert(kMaxShared <= kWaves * WORDS, "the lengths fit");
    uint32_t* s_tiles = (uint32_t*)s_v;
    auto length = [&](const Seq& x) { return x.q_len > 0 ? (uint32_t)tiles_of(x) << 1 | 1u : 0u; };
    Seq mine = {0, 0, 0, 0};
    if (lane < b.n_seqs) mine = load_seq(b, lane);
    if (b.n_seqs > (uint32_t)kWave) {
      for (uint32_t j = kWave + threadIdx.x; j < b.n_seqs; j += 256) s_tiles[j] = length(load_seq(b, j));
      __syncthreads();
    }
    at_ = part_of(length(mine), s_tiles, b.n_seqs, plan.shares, place, lane);
    if (b.n_seqs > (uint32_t)kWave) __syncthreads();
    if (at_.s < 0) return;
    if (at_.split == 0 && blockIdx.x % head_blocks == 0 && threadIdx.x == 0)
      plan.heads[at_.s] = make_int2(at_.place, at_.splits);
    if (at_.s < kWave)
      sq = Seq{(int32_t)lane_u32((uint32_t)mine.row0, at_.s), (int32_t)lane_u32((uint32_t)mine.q_len, at_.s),
               (int32_t)lane_u32((uint32_t)mine.first, at_.s), (int32_t)lane_u32((uint32_t)mine.n_keys, at_.s)};
    else
      sq = load_seq(b, (uint32_t)at_.s);
  } else {
    sq = load_seq(b, place);
  }
  const uint32_t s = (uint32_t)at_.s;
  const uint32_t n_m = (uint32_t)max(sq.q_len, 0) * group;  // rows: m = i * group + g
  if (n_m == 0) return;
  const uint32_t m1 = min(n_m, 16u * NC);

  const int32_t pos_e = max(sq.first + sq.q_len - 1, -1);
  const int32_t lo_a = first_lo(sq);                      // least lo of a row
  const int32_t lo_e = w ? max(pos_e - w + 1, 0) : 0;     // greatest
  const int32_t hi_a = causal ? min(max(sq.first, -1) + 1, sq.n_keys) : sq.n_keys;  // least hi
  const int32_t hi_e = last_hi(sq);                       // greatest

  // the split's keys, whole tiles of the workgroup
  const int32_t from = lo_a / kBlockKeys * kBlockKeys;
  const int32_t tiles = tiles_of(sq);
  const int32_t per = part_tiles(at_, tiles);
  const int32_t begin = from + min(at_.split * per, tiles) * kBlockKeys;
  const int32_t end = min(from + min((at_.split + 1) * per, tiles) * kBlockKeys, hi_e);

  // of this lane's rows, one in each column: queries, keys seen [lo, hi)
  const T* zeros = (const T*)zero_row;
  V8<T> qf[NC][KS];
  int32_t lo[NC], hi[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const bool have = n * 16 + col < m1;
    const uint32_t m = have ? n * 16 + col : m1 - 1;
    const int32_t i = (int32_t)(m / group);
    const int32_t pos = max(sq.first + i, -1);
    lo[n] = w ? max(pos - w + 1, 0) : 0;
    hi[n] = causal ? min(pos + 1, sq.n_keys) : sq.n_keys;
    const T* qp = (const T*)q.p + (uint32_t)(sq.row0 + i) * q.token_stride +
                  (uint64_t)(kh * group + m % group) * q.head_stride;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const uint32_t c = (k * 4 + quarter) * 8;
      qf[n][k] = load_row8(have && c < hd ? qp + c : zeros);
    }
  }

  f32x4 o[NC][DT];
  float top[NC], z[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    top[n] = -INFINITY;
    z[n] = 0.f;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t* table = b.table + (uint64_t)s * b.table_stride;
  const uint8_t* kbase = cache.k + (uint64_t)kh * cache.head_stride;
  const uint8_t* vbase = cache.v + (uint64_t)kh * cache.head_stride;
  T* sv = (T*)s_v[wave];

  // page id of key t0 + lane % 32 (-1: no row sees it)
  auto lookup = [&](int32_t t0) -> int32_t {
    const int32_t j = t0 + (int32_t)(lane % kTile);
    return j < end && j >= lo_a ? table[cache.page.div((uint32_t)j)] : -1;
  };
  // Where that key lies (bytes) and its block's exponents (of K, of V); bit r of the result: some
  // row sees key t0 + r.
  auto locate = [&](int32_t t0, int32_t id, uint64_t& at, uint32_t& ke, uint32_t& ve) -> uint32_t {
    const bool see = id >= 0 && (uint32_t)id < cache.n_pages;
    at = 0;
    ke = ve = 0;
    if (see) {
      const uint32_t j = (uint32_t)t0 + lane % kTile, in = j - cache.page.div(j) * cache.page.d;
      at = (uint64_t)(uint32_t)id * cache.page_stride + (uint64_t)in * cache.token_stride;
      const uint64_t e = ((uint64_t)(uint32_t)id * cache.page_blocks + cache.block.div(in)) * cache.n_heads + kh;
      ke = cache.k_exp[e];
      ve = cache.v_exp[e];
    }
    return (uint32_t)__ballot(see);
  };
  // this lane's piece of row load_row + i * RPL: its offset (bytes) from the pool's base
  const uint32_t load_row = lane / CH, load_c = lane % CH * 16;
  auto offset = [&](uint64_t at, int i) -> uint64_t {
    const int r = (int)load_row + i * RPL;
    return (((uint64_t)(uint32_t)__shfl((int)(uint32_t)(at >> 32), r) << 32) |
            (uint32_t)__shfl((int)(uint32_t)at, r)) + load_c;
  };
  auto loads = [&](uint32_t there, int i) {  // whether that row is there and has this piece
    return ((there >> (load_row + i * RPL)) & 1u) && load_c < hd;
  };
  auto power = [&](uint32_t e, int i) { return Read8<T>::power((uint32_t)__shfl((int)e, (int)load_row + i * RPL)); };
  auto codes = [&](const uint8_t* p) -> uint4 { return load_global((const uint4*)p); };
  T* put_at = sv + load_row * LD + load_c;
  const T* k_at = sv + col * LD + quarter * 8;
  // this lane's part of a transposed read of V
  const T* tr_at = sv + (4 * quarter + col / 4) * LD + 4 * (col % 4);
  bool odd = false;  // values that only some rows see and that are no numbers were left out

  const int32_t first = begin + (int32_t)(wave / kHeads) * kTile;
  // a tile's codes, its blocks' exponents, which of its keys are there
  struct Tile {
    uint4 k[NL], v[NL];
    uint32_t ke, ve, there;
  };
  // With two columns the next tile's codes are on their way while this one is computed (24 requests of 5
  // drafted tokens 74 -> 68 us); with one, four workgroups a CU do better than three that do so (87 and 95).
  constexpr bool kAhead = NC == 2 && DP <= 128;
  // page ids are looked up a step ahead: the rows' requests wait for nothing
  int32_t id = lookup(first);
  auto fetch = [&](int32_t t0, Tile& to) {
    uint64_t at;
    to.there = locate(t0, id, at, to.ke, to.ve);
    if (!kAhead) id = lookup(t0 + kBlockKeys);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint64_t from_base = offset(at, i);
      const bool on = loads(to.there, i);
      to.k[i] = codes(on ? kbase + from_base : (const uint8_t*)zeros);
      to.v[i] = codes(on ? vbase + from_base : (const uint8_t*)zeros);
    }
    if (kAhead) id = lookup(t0 + kBlockKeys);
  };
  Tile now, next;
  if (kAhead) fetch(first, now);
  for (int32_t t0 = first; t0 < end; t0 += kBlockKeys) {
    if (kAhead) fetch(t0 + kBlockKeys, next);
    else fetch(t0, now);
    const uint4 (&kc)[NL] = now.k, (&vc)[NL] = now.v;
    const uint32_t there = now.there, ke = now.ke, ve = now.ve;
    // every row sees every key of the tile?
    const bool plain = there == ~0u && t0 >= lo_e && t0 + kTile <= hi_a;

    // K to LDS, row = key of the tile
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const float p = power(ke, i);
      T* to = put_at + i * RPL * LD;
      *(V8<T>*)to = Read8<T>::eight(kc[i].x, kc[i].y, p);
      *(V8<T>*)(to + 8) = Read8<T>::eight(kc[i].z, kc[i].w, p);
    }
    wave_sync();
    f32x4 sc[NC][2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int n = 0; n < NC; ++n) sc[n][a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const V8<T> kf = *(const V8<T>*)(k_at + a * 16 * LD + k * 32);
#pragma unroll
        for (int n = 0; n < NC; ++n) sc[n][a] = mfma16(kf, qf[n][k], sc[n][a]);
      }
    }
#pragma unroll
    for (int n = 0; n < NC; ++n) settle(sc[n][0], sc[n][1]);
    // V in its place
    wave_sync();
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const float p = power(ve, i);
      V8<T> x = Read8<T>::eight(vc[i].x, vc[i].y, p), y = Read8<T>::eight(vc[i].z, vc[i].w, p);
      if (!plain) {
        const int32_t j = t0 + (int32_t)load_row + i * RPL;
        if (j < lo_e || j >= hi_a) {
          odd = odd || any_odd<T>(x) || any_odd<T>(y);
          x = finite_part<T>(x);
          y = finite_part<T>(y);
        }
      }
      T* to = put_at + i * RPL * LD;
      *(V8<T>*)to = x;
      *(V8<T>*)(to + 8) = y;
    }

    // lane's scores: keys t0 + 16 a + 4 quarter + r of its column's row
    V8<T> p[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float x[8];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[a * 4 + r] = sc[n][a][r] * scale_log2;
      if (!plain) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t kk = 4 * quarter + r;
            const int32_t j = t0 + a * 16 + (int32_t)kk;
            if (!((there >> (a * 16 + kk)) & 1u) || j < lo[n] || j >= hi[n]) x[a * 4 + r] = -INFINITY;
          }
      }
      float most = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                         fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      most = max_half(max_quarter(most));
      // (any new maximum, as in k_kv_decode: its weight is then 2^kLift and rounds to itself)
      if (__any(most > top[n] + Base<In8<T>>::kLift)) {
        const float next = next_base<In8<T>>(top[n], most);
        const float keep = exp2_raw(top[n] - (next == -INFINITY ? 0.f : next));
        z[n] *= keep;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[n][t][r] *= keep;
        top[n] = next;
      }
      float base = top[n] == -INFINITY ? 0.f : top[n];
      if (Base<In8<T>>::kBeside != 0.f) {
#pragma clang fp contract(off)
        if (__any(fabsf(base) >= 0x1p20f)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] -= base;
          base = 0.f;
        }
        base += Base<In8<T>>::kBeside;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
// (the product rounded as the base was: the largest of huge scores, too, is the base itself)
#pragma clang fp contract(off)
        const float y = exp2_raw(x[e] - base);
        z[n] += y;
        p[n][e] = (T)y;  // half a step of the dtype, relative, as the output's own rounding
      }
    }
    wave_sync();
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const V8<T> vf = join<T>(read_tr(tr_at + t * 16), read_tr(tr_at + t * 16 + 16 * LD));
#pragma unroll
      for (int n = 0; n < NC; ++n) o[n][t] = mfma16(vf, p[n], o[n][t]);
    }
    wave_sync();
    if (kAhead) now = next;
  }

  float bad = 0.f;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    settle(o[n]);
    bad += probe(o[n]) != 0.f ? 1.f : 0.f;
  }
  const bool all = __any(bad != 0.f);  // (of every tile, else of those that some rows do not see)
  if (all || __any(odd)) {
    for (int32_t t0 = first; t0 < end; t0 += kBlockKeys) {
      if (!all && t0 >= lo_e && t0 + kTile <= hi_a) continue;
      V8<T> sees[NC];
      uint64_t at;
      uint32_t ke, ve;
      const uint32_t there = locate(t0, lookup(t0), at, ke, ve);
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int32_t mine = t0 + (int32_t)load_row + i * RPL;
        const bool some = all || mine < lo_e || mine >= hi_a;
        const uint64_t from_base = offset(at, i);
        const uint4 c = codes(some && loads(there, i) ? vbase + from_base : (const uint8_t*)zeros);
        const float p = power(ve, i);
        T* to = put_at + i * RPL * LD;
        *(V8<T>*)to = odd_code<T>(Read8<T>::eight(c.x, c.y, p));
        *(V8<T>*)(to + 8) = odd_code<T>(Read8<T>::eight(c.z, c.w, p));
      }
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int32_t j = t0 + a * 16 + (int32_t)(4 * quarter) + r;
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const bool see = ((there >> (a * 16 + 4 * quarter + r)) & 1u) && j >= lo[n] && j < hi[n];
            sees[n][a * 4 + r] = (T)(see ? 1.f : 0.f);
          }
        }
      wave_sync();
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const V8<T> vf = join<T>(read_tr(tr_at + t * 16), read_tr(tr_at + t * 16 + 16 * LD));
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          f32x4 count = f32x4{0.f, 0.f, 0.f, 0.f};
          count = mfma16(vf, sees[n], count);
          settle(count);
#pragma unroll
          for (int r = 0; r < 4; ++r) o[n][t][r] = add_odd(o[n][t][r], count[r]);
        }
      }
      wave_sync();
    }
  }

  // the four waves' results together, a column of rows at a time: rows of DP floats in the V tiles
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    if (n > 0) __syncthreads();
    const float zn = sum_half(sum_quarter(z[n]));
    float* so = (float*)s_v[wave];
#pragma unroll
    for (int t = 0; t < DT; ++t) *(f32x4*)(so + col * DP + t * 16 + quarter * 4) = o[n][t];
    if (quarter == 0) {
      s_m[wave][col] = top[n];
      s_z[wave][col] = zn;
    }
    __syncthreads();
    // a row of a head to 16 / kHeads threads; the head's waves are mine, mine + kHeads, ...
    constexpr uint32_t kOf = 256 / kHeads, kRowThreads = kOf / 16;
    const uint32_t mine = threadIdx.x / kOf, r = threadIdx.x % kOf / kRowThreads;
    const uint32_t first_c = threadIdx.x % kRowThreads;
    const uint32_t rm = n * 16 + r;
    if (rm >= m1) continue;
    float mm = s_m[mine][r];
#pragma unroll
    for (int a = 1; a < kTurns; ++a) mm = fmaxf(mm, s_m[mine + a * kHeads][r]);
    float f[kTurns], zz = 0.f;
#pragma unroll
    for (int a = 0; a < kTurns; ++a) {
      f[a] = exp2_raw(s_m[mine + a * kHeads][r] - (mm == -INFINITY ? 0.f : mm));
      zz += f[a] * s_z[mine + a * kHeads][r];
    }
    const uint32_t rrow = (uint32_t)sq.row0 + rm / group;
    const uint32_t rhead = (kh - wave % kHeads + mine) * group + rm % group;
    const uint64_t unit = (uint64_t)rrow * q.n_heads + rhead;
    const bool whole = at_.splits == 1;
    // of this (place, key head, row)
    const uint64_t slot = ((uint64_t)place * cache.n_heads + (kh - wave % kHeads + mine)) * plan.rows + rm;
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
        y[e] *= Read8<T>::kScale;
      }
      if (whole) {
        V8<T> v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mean<T>(y[e], inv);
        *(V8<T>*)(op + c * 8) = v;
      } else {
        float* to_ = plan.o + slot * hd + c * 8;
        *(f32x4*)to_ = f32x4{y[0], y[1], y[2], y[3]};
        *(f32x4*)(to_ + 4) = f32x4{y[4], y[5], y[6], y[7]};
      }
    }
    if (first_c == 0) {
      if (!whole) plan.ms[slot] = make_float2(mm, zz);
      else if (lse) lse[unit] = zz == 0.f ? -INFINITY : (log_of_base<In8<T>>(mm) + __builtin_amdgcn_logf(zz)) * kLn2;
    }
  }
}

// What a place of the joins' grids has to join: `rows` rows from m0 of the item's, `n` results each (n <= 1: none).
struct Parts8 {
  Seq sq;
  uint32_t m0, rows, n, first;  // first: the place of the first result
};
__device__ __forceinline__ Parts8 parts_of(const Batch& b, const Plan8& plan, uint32_t group, uint32_t u) {
  Parts8 p = {};
  int2 of;  // (of no meaning where the item has no rows)
  uint32_t item = u;
  p.first = u;
  if (plan.row_tiles == 1) {
    if (item >= b.n_seqs) return p;
    of = plan.heads[item];
    p.first = (uint32_t)of.x;
  } else {  // (of the tiles of the longest sequence's rows most may have none)
    if (u >= plan.places) return p;
    of = plan.firsts[u];
    if (of.y <= 1) return p;
    item = (uint32_t)of.x;
  }
  p.sq = load_seq(b, item % b.n_seqs);
  const uint32_t n_m = (uint32_t)max(p.sq.q_len, 0) * group;
  p.m0 = (plan.row_tiles - 1 - item / b.n_seqs) * plan.rows;
  if (p.m0 >= n_m) return p;
  p.rows = min(plan.rows, n_m - p.m0);
  if ((uint64_t)p.first + (uint32_t)of.y <= plan.places) p.n = (uint32_t)of.y;  // (else: overlapping sequences)
  return p;
}
template <typename T>
__device__ __forceinline__ void finish(const Rows& out, uint32_t row, uint32_t head, uint32_t c, bool live,
                                       const f32x4& o, float z, float mm, float* lse) {
  if (live) {
    const float inv = z == 0.f ? 0.f : 1.f / z;
    typedef T t4 __attribute__((ext_vector_type(4)));
    t4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = mean<T>(o[r], inv);
    *(t4*)((T*)out.p + row * out.token_stride + (uint64_t)head * out.head_stride + c) = v;
  }
  if (lse && c == 0)
    lse[(uint64_t)row * out.n_heads + head] =
        z == 0.f ? -INFINITY : (log_of_base<In8<T>>(mm) + __builtin_amdgcn_logf(z)) * kLn2;
}

// The splits of rows together: a wave to one row of an item and key head, 64 splits' factors in its lanes, then
// `lanes` lanes (four channels each) a split; or, where rows are many (kMany), to four rows for each
// `lanes` lanes, so that what a wave looks up first serves them all (2 splits of 32,768 rows 12 us).  The
// first turns' results are asked for beside the factors: 800 rows of about 6 splits 4.3 us (5.3 in turn).
template <typename T, bool kMany>
__global__ __launch_bounds__(256) void k_kv8_join(Batch b, Rows out, Plan8 plan, uint32_t n_heads,
                                                  uint32_t head_dim, uint32_t lanes, float* __restrict__ lse) {
  const uint32_t lane = threadIdx.x % kWave, at_once = kWave / lanes;
  const uint32_t n_r = kMany ? 4 * at_once : 1, parts = (plan.rows + n_r - 1) / n_r;  // rows of a wave
  uint32_t u = blockIdx.x * 4 + uniform(threadIdx.x / kWave);
  const uint32_t r0 = u % parts * n_r;
  u /= parts;
  const uint32_t kh = u % n_heads;
  u /= n_heads;
  const uint32_t group = out.n_heads / n_heads;
  const Parts8 p = parts_of(b, plan, group, u);
  const uint32_t n = p.n;
  if (n <= 1 || r0 >= p.rows) return;
  const uint32_t rows = min(n_r, p.rows - r0);
  const uint64_t step = (uint64_t)n_heads * plan.rows, slot = p.first * step + (uint64_t)kh * plan.rows + r0;
  const uint32_t c = lane % lanes * 4, sub = lane / lanes;
  const bool live = c < head_dim;
  // a turn: four rows' parts of one split, or one row's of at_once splits
  constexpr int kR = kMany ? 4 : 1;
  constexpr uint32_t kAhead = kMany ? 2 : 4;
  auto split_of = [&](uint32_t t) { return kMany ? t : t * at_once + sub; };
  auto row_of = [&](int j) { return kMany ? sub * kR + j : 0; };
  auto part = [&](uint32_t e, int j) -> f32x4 {
    const uint64_t at = slot + min(row_of(j), rows - 1) + min(e, n - 1) * step;
    return live ? *(const f32x4*)(plan.o + at * head_dim + c) : f32x4{0.f, 0.f, 0.f, 0.f};
  };
  // factors: lane `lane` has row lane % n_r of split (lane / n_r) of every kWave / n_r; the first turns'
  // results are on their way beside them
  const uint32_t fr = lane % n_r, fe = lane / n_r, f_step = kWave / n_r;
  const float2* ms = plan.ms + slot + min(fr, rows - 1);
  const float2 nothing = make_float2(-INFINITY, 0.f);
  float2 x = fe < n ? ms[fe * step] : nothing;
  f32x4 ahead[kAhead][kR];
#pragma unroll
  for (uint32_t t = 0; t < kAhead; ++t)
#pragma unroll
    for (int j = 0; j < kR; ++j) ahead[t][j] = part(split_of(t), j);
  float mm = x.x;
  for (uint32_t e = fe + f_step; e < n; e += f_step) mm = fmaxf(mm, ms[e * step].x);
  for (uint32_t d = n_r; d < (uint32_t)kWave; d <<= 1) mm = fmaxf(mm, __shfl_xor(mm, (int)d));
  const float base = mm == -INFINITY ? 0.f : mm;
  f32x4 o[kR];
#pragma unroll
  for (int j = 0; j < kR; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float z = 0.f;
  for (uint32_t e0 = 0; e0 < n; e0 += f_step) {
    if (e0) x = e0 + fe < n ? ms[(e0 + fe) * step] : nothing;
    const float f = exp2_raw(x.x - base);
    z += f * x.y;
    const uint32_t some = min(n - e0, f_step);
    auto add = [&](uint32_t t, int j, const f32x4& y) {
      const uint32_t e = split_of(t);
      const float fj = __shfl(f, (int)min(e * n_r + row_of(j), (uint32_t)kWave - 1));
      if (e >= some) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] += scaled(y[i], fj);
    };
    const uint32_t turns = kMany ? some : (some + at_once - 1) / at_once;
    for (uint32_t t0 = 0; t0 < turns; t0 += kAhead) {
#pragma unroll
      for (uint32_t t = 0; t < kAhead; ++t)
#pragma unroll
        for (int j = 0; j < kR; ++j) add(t0 + t, j, ahead[t][j]);
      const bool last = t0 + kAhead >= turns;
      if (last && e0 + f_step >= n) break;
      const uint32_t next = last ? e0 + f_step : e0, nt = last ? 0 : t0 + kAhead;
#pragma unroll
      for (uint32_t t = 0; t < kAhead; ++t)
#pragma unroll
        for (int j = 0; j < kR; ++j) ahead[t][j] = part(next + split_of(nt + t), j);
    }
  }
  for (uint32_t d = n_r; d < (uint32_t)kWave; d <<= 1) z += __shfl_xor(z, (int)d);
  if (!kMany)
    for (uint32_t d = lanes; d < (uint32_t)kWave; d <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[0][i] += __shfl_xor(o[0][i], (int)d);
#pragma unroll
  for (int j = 0; j < kR; ++j) {
    const uint32_t r = row_of(j), m = p.m0 + r0 + r;
    const float zj = kMany ? __shfl(z, (int)r) : z, mj = kMany ? __shfl(mm, (int)r) : mm;
    const bool mine = kMany ? r < rows : sub == 0;
    finish<T>(out, (uint32_t)p.sq.row0 + m / group, kh * group + m % group, c, live && mine, o[j], zj, mj,
              mine ? lse : nullptr);
  }
}

// The same with a workgroup of 1024 for each (row, head), where the splits are many and the rows few (128 rows and
// heads of 128 splits 8 us; 784 of 36 take 11 here, 7 with a wave each).
template <typename T>
__global__ __launch_bounds__(1024) void k_kv8_join_many(Batch b, Rows out, Plan8 plan, uint32_t n_heads,
                                                       uint32_t head_dim, uint32_t lanes,
                                                       float* __restrict__ lse) {
  constexpr uint32_t kThreads = 1024, NW = kThreads / kWave;
  static_assert(kMaxSplits <= kThreads, "a thread per split");
  __shared__ float s_f[kThreads];
  __shared__ float s_red[NW];
  __shared__ f32x4 s_o[kThreads];
  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const uint32_t r = blockIdx.x % plan.rows, kh = blockIdx.x / plan.rows % n_heads, group = out.n_heads / n_heads;
  const Parts8 p = parts_of(b, plan, group, blockIdx.x / plan.rows / n_heads);
  if (p.n <= 1 || r >= p.rows) return;
  const uint64_t step = (uint64_t)n_heads * plan.rows, slot = p.first * step + (uint64_t)kh * plan.rows + r;
  const float2 x = tid < p.n ? plan.ms[slot + tid * step] : make_float2(-INFINITY, 0.f);
  float mm = x.x;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) mm = fmaxf(mm, __shfl_xor(mm, d, kWave));
  if (lane == 0) s_red[wave] = mm;
  __syncthreads();
  for (uint32_t w = 0; w < NW; ++w) mm = fmaxf(mm, s_red[w]);
  __syncthreads();
  const float f = exp2_raw(x.x - (mm == -INFINITY ? 0.f : mm));
  s_f[tid] = f;
  float z = tid < p.n ? f * x.y : 0.f;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) z += __shfl_xor(z, d, kWave);
  if (lane == 0) s_red[wave] = z;
  __syncthreads();
  z = 0.f;
  for (uint32_t w = 0; w < NW; ++w) z += s_red[w];
  const uint32_t c = (tid % lanes) * 4, at_once = kThreads / lanes;
  const bool live = c < head_dim;
  f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
  if (live) {
#pragma unroll 4
    for (uint32_t e = tid / lanes; e < p.n; e += at_once) {
      const f32x4 y = *(const f32x4*)(plan.o + (slot + e * step) * head_dim + c);
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] += scaled(y[r], s_f[e]);
    }
  }
  s_o[tid] = o;
  __syncthreads();
  for (uint32_t half = kThreads / 2; half >= lanes; half /= 2) {
    if (tid < half) {
      const f32x4 y = s_o[tid + half];
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] += y[r];
      s_o[tid] = o;
    }
    __syncthreads();
  }
  const uint32_t m = p.m0 + r;
  if (tid < lanes) finish<T>(out, (uint32_t)p.sq.row0 + m / group, kh * group + m % group, c, live, o, z, mm, lse);
}

template <typename T>
hipError_t run_join8(const Plan8& p, const Cache8& c, const Batch& b, const Rows& out, float* lse, hipStream_t s) {
  const uint32_t lanes = c.head_dim <= 64 ? 16 : c.head_dim <= 128 ? 32 : 64;
  const uint64_t head_units = (uint64_t)(p.row_tiles == 1 ? b.n_seqs : p.places) * c.n_heads;
  if (p.wide_join) {
    hipLaunchKernelGGL(k_kv8_join_many<T>, dim3((uint32_t)(head_units * p.rows)), dim3(1024), 0, s, b, out, p,
                       c.n_heads, c.head_dim, lanes, lse);
    return hipGetLastError();
  }
  const bool many = (uint64_t)b.n_rows * out.n_heads >= kManyRows || p.row_tiles > 1;
  const uint32_t n_r = many ? 4 * kWave / lanes : 1;
  const dim3 grid((uint32_t)((head_units * ((p.rows + n_r - 1) / n_r) + 3) / 4));
  if (many)
    hipLaunchKernelGGL((k_kv8_join<T, true>), grid, dim3(256), 0, s, b, out, p, c.n_heads, c.head_dim, lanes, lse);
  else
    hipLaunchKernelGGL((k_kv8_join<T, false>), grid, dim3(256), 0, s, b, out, p, c.n_heads, c.head_dim, lanes, lse);
  return hipGetLastError();
}

template <typename T, int DP, int kHeads, int NC>
hipError_t run_decode8(const Plan8& p, const Cache8& c, const Batch& b, const Rows& q, const Rows& out,
                       float scale, uint32_t window, bool causal, float* lse, hipStream_t s) {
  hipLaunchKernelGGL((k_kv8_decode<T, DP, kHeads, NC>), dim3(p.places * (c.n_heads / kHeads)), dim3(256), 0, s,
                     c, b, q, out, scale * kLog2e * Read8<T>::kScale, window, causal, p, lse);
  hipError_t e = hipGetLastError();
  return e != hipSuccess || p.shares == 0 ? e : run_join8<T>(p, c, b, out, lse, s);
}

}  // namespace

hipError_t launch_join8(const Plan8& p, const Cache8& c, uint32_t dtype, const Batch& b, const Rows& out, float* lse,
                        hipStream_t s) {
  return dtype == IBP_KV_F16 ? run_join8<_Float16>(p, c, b, out, lse, s) : run_join8<__bf16>(p, c, b, out, lse, s);
}

hipError_t launch_decode8(const Plan8& p, const Cache8& c, uint32_t dtype, const Batch& b, const Rows& q,
                          const Rows& out, float scale, uint32_t window, bool causal, float* lse,
                          hipStream_t s) {
#define IBP_KV8_DECODE(T, DP, HEADS, NC) \
  run_decode8<T, DP, HEADS, NC>(p, c, b, q, out, scale, window, causal, lse, s)
#define IBP_KV8_DECODE_T(T, HEADS, NC)                                              \
  (c.head_dim <= 64    ? IBP_KV8_DECODE(T, 64, HEADS, NC)                           \
   : c.head_dim <= 128 ? IBP_KV8_DECODE(T, 128, HEADS, NC)                          \
                       : IBP_KV8_DECODE(T, 256, HEADS, NC))
#define IBP_KV8_DECODE_C(T, HEADS) (p.rows > 16 ? IBP_KV8_DECODE_T(T, HEADS, 2) : IBP_KV8_DECODE_T(T, HEADS, 1))
#define IBP_KV8_DECODE_S(T) (p.head_group == 4 ? IBP_KV8_DECODE_C(T, 4) : IBP_KV8_DECODE_C(T, 1))
  return dtype == IBP_KV_F16 ? IBP_KV8_DECODE_S(_Float16) : IBP_KV8_DECODE_S(__bf16);
#undef IBP_KV8_DECODE_S
#undef IBP_KV8_DECODE_C
#undef IBP_KV8_DECODE_T
#undef IBP_KV8_DECODE
}

}  // namespace kv
}  // namespace ibp
