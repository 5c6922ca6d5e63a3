// kv_chunk.hip -- attention of many rows that share their keys: a chunk of new
// tokens of a sequence with the query heads of one key head.
#include "ibp_device.h"
#include "kv_mfma.h"

namespace ibp {
namespace kv {

namespace {

constexpr int kKeys = 64;   // keys of a step
constexpr int kWaves = 4;
constexpr int kRows = kChunkRows;
static_assert(kRows == 32 * kWaves, "a wave holds 32 rows");
constexpr int kThreads = kWave * kWaves;

// Barrier of the workgroup that orders LDS only: loads from global memory stay
// in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// One wave's load of 64 pieces of 16 B from global memory straight into LDS, piece l to
// lds + 16 l: no register holds them on the way, so the compiler neither counts nor waits
// for them: whoever reads them has waited for vmcnt(0) and a barrier.  Inactive lanes'
// pieces are left as they are.
__device__ __forceinline__ void load_lds(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void load_lds(const void* base, uint32_t offset, uint32_t lds) {
  // The move fills the wait state after m0; and a base that came straight from a lane would need
  // five before the load, which the compiler does not see to in here, but none before a move.
  uint64_t scalar;
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(scalar) : "s"(lds), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  typedef __attribute__((address_space(3))) const void lds_void;
  return uniform((uint32_t)(uintptr_t)(lds_void*)p);
}

// A workgroup per (128 rows that share a key head, split of their keys); a
// wave holds 32 rows: their queries, and their outputs transposed.
//
// Steps of 64 keys, in a pipeline: while step t's scores become weights (the vector ALU: a
// multiply-add, an exponential, a sum and half a conversion a score), the matrix cores
// form step t+1's scores; then step t's weights meet its values.  Rows go from
// memory straight into LDS, K two steps ahead and V one, each into the half that the
// step before has left: one barrier a step.
//
// LDS rows are DL elements, their 16 B pieces in an order of their own (load_lds fills
// LDS in lane order, so the lane chooses which piece it brings): piece c of K row r lies at c ^
// swizzle_k(r), so that 16 rows read at one channel lie in 16 different 16 B slots of the
// banks; V pieces so that the four rows of half a transposed read lie in four 64 B windows.
//
// Measured (bf16, 32 query heads on 8 key heads, head_dim 128): one prompt of 16,384 tokens
// 2.09 to 2.26 ms from card to card, 0.97 to 1.05 PFLOP/s, where a library product of 16,384^3 reaches
// 1.31 to 1.37; the matrix cores are busy 52 % of the time, the vector ALU 56 %, at the 1.9 GHz that
// power leaves.  Without the pipeline (rows through registers, scores, weights and values in turn) it
// took 2.49 ms where it took 2.13 with it.  Ragged chunks of up to 511 rows over 9,001 to 2,701 tokens
// 243 us, 870 TFLOP/s; one prompt of 2,048 tokens 57 us, 600 TFLOP/s (too few tiles for all CUs).
// No faster: 64 rows a wave, one wave a SIMD (2.09 ms on a card where this took the same; ragged chunks
// 380 us where this then took 290), half of the weights beside the values instead of the scores (the same).
template <typename T, int DP, bool kExact>  // kExact: head_dim == DP == the LDS row
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void k_kv_chunk(
    Cache cache, Batch b, Rows q, Rows out, float scale, uint32_t window, bool causal,
    uint32_t row_tiles, bool by_length, Partial part, float* __restrict__ lse) {
  constexpr int KS = DP / 16;                            // products of a score
  constexpr int DT = DP / 32;                            // tiles of the output
  constexpr int DL = DP <= 64 ? 64 : DP <= 128 ? 128 : 256;  // LDS row, elements
  constexpr int CH = DL / 8;                             // pieces of a row
  constexpr int ST = kKeys * CH / kThreads;              // loads of a wave, of K and of V
  constexpr int RPL = kWave / CH;                        // rows of a load
  constexpr int RPR = kThreads / CH;                     // rows of the four waves' loads
  constexpr int TILE = kKeys * DL;
  __shared__ __align__(1024) uint16_t s_k[2][TILE];
  __shared__ __align__(1024) uint16_t s_v[2][TILE];
  __shared__ uint32_t s_odd, s_bad;

  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const uint32_t col = lane % 32, half = lane / 32;
  const uint32_t group = q.n_heads / cache.n_heads;
  const uint32_t hd = kExact ? DP : cache.head_dim;

  // block -> key head (innermost: blocks of one head meet in one XCD's L2 where the heads
  // are a multiple of eight), split, then sequence, row tile from the last (under a
  // causal mask the longest)
  uint32_t u = blockIdx.x;
  const uint32_t kh = u % cache.n_heads;
  u /= cache.n_heads;
  const uint32_t split = u % part.splits;
  u /= part.splits;
  uint32_t s, tile;
  Seq sq;
  if (!by_length) {
    s = u % b.n_seqs;
    tile = row_tiles - 1 - u / b.n_seqs;
    sq = load_seq(b, s);
  } else {
    // Chunks against longer contexts, whose tiles' times differ by sequence more than inside
    // one: the longest sequence's first (a lane per sequence), so that two long tiles seldom
    // share a CU and none begins late.
    Seq mine = Seq{0, 0, 0, 0};
    if (lane < b.n_seqs) mine = load_seq(b, lane);
    const uint32_t n_tiles = ((uint32_t)max(mine.q_len, 0) * group + kRows - 1) / kRows;
    uint32_t before = 0, total = 0;
    for (uint32_t j = 0; j < b.n_seqs; ++j) {
      const int32_t keys = __builtin_amdgcn_readlane(mine.n_keys, j);
      const uint32_t n = (uint32_t)__builtin_amdgcn_readlane((int)n_tiles, j);
      if (keys > mine.n_keys || (keys == mine.n_keys && j < lane)) before += n;
      total += n;
    }
    if (u >= total) return;
    s = (uint32_t)__builtin_ctzll(__ballot(u >= before && u - before < n_tiles));
    tile = (uint32_t)__builtin_amdgcn_readlane((int)(n_tiles - 1 - (u - before)), s);
    sq = Seq{__builtin_amdgcn_readlane(mine.row0, s), __builtin_amdgcn_readlane(mine.q_len, s),
             __builtin_amdgcn_readlane(mine.first, s), __builtin_amdgcn_readlane(mine.n_keys, s)};
  }
  const uint32_t n_m = (uint32_t)max(sq.q_len, 0) * group;
  const uint32_t m0 = tile * kRows;
  if (m0 >= n_m) return;
  const uint32_t m1 = min(m0 + kRows, n_m);

  // keys seen by rows m of the block or of a wave: [lo, hi) of the first and of the last
  const int32_t w = (int32_t)window;
  auto pos_of = [&](uint32_t m) { return max(sq.first + (int32_t)(m / group), -1); };
  auto lo_of = [&](int32_t pos) { return w ? max(pos - w + 1, 0) : 0; };
  auto hi_of = [&](int32_t pos) { return causal ? min(pos + 1, sq.n_keys) : sq.n_keys; };
  const int32_t blk_lo = lo_of(pos_of(m0)), blk_hi = hi_of(pos_of(m1 - 1));
  const int32_t edge_lo = lo_of(pos_of(m1 - 1)), edge_hi = hi_of(pos_of(m0));
  const bool active = m0 + wave * 32 < m1;
  const uint32_t wm0 = min(m0 + wave * 32, m1 - 1), wm1 = min(m0 + wave * 32 + 32, m1) - 1;
  const int32_t full_lo = lo_of(pos_of(active ? wm1 : wm0)), full_hi = hi_of(pos_of(wm0));
  const bool have = m0 + wave * 32 + col < m1;
  const uint32_t m = have ? m0 + wave * 32 + col : m1 - 1;
  const int32_t pos = pos_of(m), lo = lo_of(pos), hi = hi_of(pos);
  const uint32_t row = (uint32_t)sq.row0 + m / group, head = kh * group + m % group;

  const int32_t from = blk_lo / kKeys * kKeys;
  const int32_t tiles = max(blk_hi - from + kKeys - 1, 0) / kKeys;
  const int32_t per = (tiles + (int32_t)part.splits - 1) / (int32_t)part.splits;
  const int32_t begin = from + min((int32_t)split * per, tiles) * kKeys;
  const int32_t end = from + min(((int32_t)split + 1) * per, tiles) * kKeys;
  // a step with keys that some rows of the block see and others do not
  auto is_edge = [&](int32_t t0) { return t0 < edge_lo || t0 + kKeys > edge_hi; };

  // queries, their sign that of the scale (the maximum below is of unscaled scores)
  const T* qp = (const T*)q.p + row * q.token_stride + (uint64_t)head * q.head_stride;
  const T* zeros = (const T*)zero_row;
  V8<T> qf[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const uint32_t c = k * 16 + half * 8;
    qf[k] = load_row8(have && c < hd ? qp + c : zeros);
    if (scale < 0.f) qf[k] = -qf[k];
    if (scale == 0.f)  // (zeros, but for what is no number)
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[k][e] = isfinite((float)qf[k][e]) ? (T)0.f : (T)NAN;
  }
  const float sc2 = scale == 0.f ? 1.f : fabsf(scale) * kLog2e;

  f32x16 o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[t][r] = 0.f;
  float top = -INFINITY, z = 0.f;

  const int32_t* table = b.table + (uint64_t)s * b.table_stride;
  const T* kbase = (const T*)cache.k + (uint64_t)kh * cache.head_stride;
  const T* vbase = (const T*)cache.v + (uint64_t)kh * cache.head_stride;

  // this lane's piece in a load: row load_row (plus RPR for each further load) and place
  auto swizzle_k = [](uint32_t r) { return CH >= 16 ? r & 15u : (r >> 1) & 7u; };
  auto swizzle_v = [](uint32_t r) { return CH >= 16 ? (r & 3u) << 2 : (r & 2u) << 1; };
  const uint32_t load_row = wave * RPL + lane / CH, place = lane % CH;
  const uint32_t lds_k = lds_address(s_k), lds_v = lds_address(s_v);
  // a load's rows lie in one page, at offsets that 32 bits hold
  const bool same_page = cache.page.d % RPL == 0 && cache.token_stride <= (1u << 26);
  if (!kExact) {  // pieces past head_dim: never loaded, zeros
#pragma unroll
    for (int i = 0; i < 2 * ST; ++i) {
      ((uint4*)s_k)[tid + i * kThreads] = make_uint4(0, 0, 0, 0);
      ((uint4*)s_v)[tid + i * kThreads] = make_uint4(0, 0, 0, 0);
    }
  }

  // page id of key t0 + lane (-1: no row of the block sees it)
  auto lookup = [&](int32_t t0) -> int32_t {
    const int32_t j = t0 + (int32_t)lane;
    return t0 < end && j >= blk_lo && j < blk_hi ? table[cache.page.div((uint32_t)j)] : -1;
  };
  // where key t0 + lane lies (elements), and which of the 64 are there
  auto locate = [&](int32_t t0, int32_t id, uint64_t& at) -> uint64_t {
    const uint32_t j = (uint32_t)(t0 + (int32_t)lane);
    const bool see = id >= 0 && (uint32_t)id < cache.n_pages;
    at = see ? (uint64_t)(uint32_t)id * cache.page_stride +
                   (uint64_t)(j - cache.page.div(j) * cache.page.d) * cache.token_stride
             : 0;
    return __ballot(see);
  };
  auto bring = [&](const T* base, uint64_t at, uint64_t seen, uint32_t lds, bool is_k) {
    if (seen == ~0ull && same_page) {
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        const uint32_t c = place ^ (is_k ? swizzle_k(load_row + i * RPR) : swizzle_v(load_row + i * RPR));
        const uint32_t off = (uint32_t)((lane / CH) * cache.token_stride + c * 8) * 2;
        const uint64_t a = lane_u64(at, i * RPR + wave * RPL);
        if (kExact || c * 8 < hd) load_lds(base + a, off, lds + (i * RPR + wave * RPL) * DL * 2);
      }
    } else {
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        const uint32_t r = load_row + i * RPR;
        const uint32_t c = place ^ (is_k ? swizzle_k(r) : swizzle_v(r));
        const uint64_t a = ((uint64_t)(uint32_t)__shfl((int)(uint32_t)(at >> 32), (int)r) << 32) |
                           (uint32_t)__shfl((int)(uint32_t)at, (int)r);
        const T* p = (seen >> r) & 1u ? base + a + c * 8 : zeros;
        if (kExact || c * 8 < hd) load_lds(p, lds + (i * RPR + wave * RPL) * DL * 2);
      }
    }
  };

  bool odd = false;
  // no infinity or NaN of an edge step's values may enter the product (what they add to the
  // rows that see them comes after the loop)
  auto clean = [&](uint16_t* sv) {
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      V8<T>* p = (V8<T>*)sv + tid + i * kThreads;
      const V8<T> v = *p;
      if (any_odd<T>(v)) {
        odd = true;
        *p = finite_part<T>(v);
      }
    }
    lds_barrier();
  };

  // K pieces of row r: piece 2 k + half lies at (2 k) ^ (half ^ swizzle_k(r))
  const uint32_t k_at = col * DL, k_sw = half ^ swizzle_k(col);
  auto scores = [&](const uint16_t* sk, f32x16 (&sc)[2]) {
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int r = 0; r < 16; ++r) sc[a][r] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const V8<T> kf = *(const V8<T>*)(sk + a * 32 * DL + k_at + (((uint32_t)(2 * k) ^ k_sw) << 3));
        sc[a] = mfma32(kf, qf[k], sc[a]);
      }
  };
  // this lane's part of a transposed read: rows 16 k + v_row (+ 8), columns 32 t + ...
  const uint32_t v_row = 4 * half + (lane % 16) / 4;
  auto tr_at = [&](int t) {
    const uint32_t c = (uint32_t)t * 4 + 2 * ((lane / 16) % 2) + (lane % 4) / 2;
    return v_row * DL + ((c ^ swizzle_v(v_row)) << 3) + (lane % 2) * 4;
  };
  // Which keys of step t0 this lane's row sees, as the scores lie: bit 8 (r / 4) + r % 4 of
  // word a for register r of tile a (key t0 + 32 a + 8 (r / 4) + 4 half + r % 4).
  auto visible = [&](int32_t t0, uint64_t seen, uint32_t (&vis)[2]) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int32_t l = lo - t0 - 32 * a, h = hi - t0 - 32 * a;
      const uint32_t below_h = h <= 0 ? 0u : h >= 32 ? ~0u : (1u << h) - 1u;
      const uint32_t below_l = l <= 0 ? 0u : l >= 32 ? ~0u : (1u << l) - 1u;
      vis[a] = ((uint32_t)(seen >> (32 * a)) & below_h & ~below_l) >> (4 * half);
    }
  };
  // Scores of step t0 that the row does not see to -inf, where there may be any (`most`, the
  // largest one, is then found anew); then the base that the exponents are taken against: a
  // weight is 2^(score * mul + off).  Where a base is so large that its own rounding could lift
  // a weight past fp16's range, the scores are first made differences, each product
  // rounded as the base was.
  float mul = sc2, off = 0.f;
  auto bound = [&](int32_t t0, uint64_t seen, f32x16 (&sc)[2], float most) {
    if (!(seen == ~0ull && t0 >= full_lo && t0 + kKeys <= full_hi)) {
      uint32_t vis[2];
      visible(t0, seen, vis);
      most = -INFINITY;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (!(vis[a] & (1u << (8 * (r / 4) + r % 4)))) sc[a][r] = -INFINITY;
          most = fmaxf(most, sc[a][r]);
        }
    }
    most = max_half(most) * sc2;
    if (__any(most > top + Base<T>::kRoom)) {
      const float next = next_base<T>(top, most);
      const float keep = exp2_raw(top - (next == -INFINITY ? 0.f : next));
      settle(o);
      z *= keep;
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] *= keep;
      top = next;
    }
    mul = sc2;
    off = top == -INFINITY ? 0.f : -top;
    if (__any(fabsf(off) >= 0x1p20f)) {
#pragma clang fp contract(off)
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[a][r] = sc[a][r] * sc2 + off;
      mul = 1.f;
      off = 0.f;
    }
  };

  uint64_t at1, at2, seen0, seen1, seen2;
  {
    uint64_t at0;
    const int32_t id0 = lookup(begin), id1 = lookup(begin + kKeys);
    seen0 = locate(begin, id0, at0);
    seen1 = locate(begin + kKeys, id1, at1);
    if (tid == 0) s_odd = s_bad = 0;
    lds_barrier();
    if (begin < end) {
      bring(kbase, at0, seen0, lds_k, true);
      bring(vbase, at0, seen0, lds_v, false);
    }
    if (begin + kKeys < end) bring(kbase, at1, seen1, lds_k + TILE * 2, true);
  }
  int32_t id2 = lookup(begin + 2 * kKeys);
  wait_loads();
  lds_barrier();

  f32x16 sa[2], sb[2];
  if (begin < end) {
    scores(s_k[0], sa);
    // The first step loads into s_k[0] at once: every wave has to have read it.
    lds_barrier();
    settle(sa[0], sa[1]);
    float most = -INFINITY;
#pragma unroll
    for (int r = 0; r < 16; ++r) most = fmaxf(most, fmaxf(sa[0][r], sa[1][r]));
    bound(begin, seen0, sa, most);
  }

  // Step t0 (its scores in `cur`, masked, the base set; K of t0 + 64 and V of t0 in LDS):
  // buffer `buf` holds V of t0 and gets K of t0 + 128, the other one gets V of t0 + 64.  Both loads
  // begin on entry, so a barrier lies between it and the last reading of s_k[buf] (the scores of t0,
  // in the step before or ahead of the loop) and of s_v[buf ^ 1] (the values of t0 - 64).
  auto step = [&](int32_t t0, uint32_t buf, f32x16 (&cur)[2], f32x16 (&nxt)[2]) {
    seen2 = locate(t0 + 2 * kKeys, id2, at2);
    if (t0 + kKeys < end) bring(vbase, at1, seen1, lds_v + (buf ^ 1) * TILE * 2, false);
    if (t0 + 2 * kKeys < end) bring(kbase, at2, seen2, lds_k + buf * TILE * 2, true);
    id2 = lookup(t0 + 3 * kKeys);
    if (is_edge(t0)) clean(s_v[buf]);
    if (active) {
      // Step t0's weights and the next step's scores together, in a fixed order: a K piece two
      // products ahead, a product, its share of the weights.  (Past the last step: scores of
      // what lies in LDS, not used.)
      const uint16_t* sk = s_k[buf ^ 1] + k_at;
      auto k_piece = [&](int i) {
        return *(const V8<T>*)(sk + (i % 2) * 32 * DL + (((uint32_t)(i / 2 * 2) ^ k_sw) << 3));
      };
      V8<T> p[4], kf[3];
      float z0 = 0.f, z1 = 0.f;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) nxt[a][r] = 0.f;
      kf[0] = k_piece(0);
      kf[1] = k_piece(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) {
        if (i + 2 < 2 * KS) kf[(i + 2) % 3] = k_piece(i + 2);
        nxt[i % 2] = mfma32(kf[i % 3], qf[i / 2], nxt[i % 2]);
#pragma unroll
        for (int e = i * 16 / KS; e < (i + 1) * 16 / KS; ++e) {
          const float y = exp2_raw(fmaf(cur[e / 16][e % 16], mul, off));
          if (e % 2) z1 += y;
          else z0 += y;
          // half a step of the dtype, relative, as the output's own rounding
          p[e / 8][e % 8] = (T)y;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      z += z0 + z1;
      // Step t0's values, with the largest of the next step's scores on the side.
      const T* sv = (const T*)s_v[buf];
      uint32_t tr[DT];
#pragma unroll
      for (int t = 0; t < DT; ++t) tr[t] = tr_at(t);
      auto v_piece = [&](int i) {
        const T* v = sv + tr[i % DT] + 16 * (i / DT) * DL;
        return join<T>(read_tr(v), read_tr(v + 8 * DL));
      };
      V8<T> vf[3];
      vf[0] = v_piece(0);
      vf[1] = v_piece(1);
      float most = -INFINITY, most1 = -INFINITY;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4 * DT; ++i) {
        if (i + 2 < 4 * DT) vf[(i + 2) % 3] = v_piece(i + 2);
        o[i % DT] = mfma32(vf[i % 3], p[i / DT], o[i % DT]);
#pragma unroll
        for (int e = i * 8 / DT; e < (i + 1) * 8 / DT; ++e) {
          if (e % 2) most1 = fmaxf(most1, nxt[e / 16][e % 16]);
          else most = fmaxf(most, nxt[e / 16][e % 16]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (t0 + kKeys < end) bound(t0 + kKeys, seen1, nxt, fmaxf(most, most1));
    }
    wait_loads();
    lds_barrier();
    at1 = at2;
    seen1 = seen2;
  };
  for (int32_t t0 = begin; t0 < end; t0 += 2 * kKeys) {
    step(t0, 0, sa, sb);
    if (t0 + kKeys < end) step(t0 + kKeys, 1, sb, sa);
  }

  settle(o);
  if (odd) s_odd = 1;
  if (probe(o) != 0.f) s_bad = 1;
  lds_barrier();
  if (s_odd || s_bad) {
    for (int32_t t0 = begin; t0 < end; t0 += kKeys) {
      if (!s_bad && !is_edge(t0)) continue;
      uint64_t at;
      const uint64_t seen = locate(t0, lookup(t0), at);
      bring(vbase, at, seen, lds_v, false);
      wait_loads();
      lds_barrier();
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        V8<T>* p = (V8<T>*)s_v[0] + tid + i * kThreads;
        *p = odd_code<T>(*p);
      }
      lds_barrier();
      V8<T> sees[4];
      uint32_t vis[2];
      visible(t0, seen, vis);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        sees[e / 8][e % 8] = (T)(vis[e / 16] & (1u << (8 * ((e / 4) % 4) + e % 4)) ? 1.f : 0.f);
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        f32x16 n;
#pragma unroll
        for (int r = 0; r < 16; ++r) n[r] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const T* v = (const T*)s_v[0] + tr_at(t) + 16 * k * DL;
          n = mfma32(join<T>(read_tr(v), read_tr(v + 8 * DL)), sees[k], n);
        }
        settle(n);
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] = add_odd(o[t][r], n[r]);
      }
      lds_barrier();
    }
  }

  if (!have) return;
  z = sum_half(z);
  const uint64_t unit = (uint64_t)row * q.n_heads + head;
  if (part.splits > 1) {
    float* to = part.row(unit, split);
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t c = t * 32 + 8 * r + 4 * half;
        if (c < hd)
          *(f32x4*)(to + c) = f32x4{o[t][4 * r], o[t][4 * r + 1], o[t][4 * r + 2], o[t][4 * r + 3]};
      }
    if (half == 0) part.ms[unit * part.splits + split] = make_float2(top, z);
    return;
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  T* op = (T*)out.p + row * out.token_stride + (uint64_t)head * out.head_stride;
  typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t c = t * 32 + 8 * r + 4 * half;
      t4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = mean<T>(o[t][4 * r + e], inv);
      if (c < hd) *(t4*)(op + c) = v;
    }
  if (lse && half == 0) lse[unit] = z == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(z)) * kLn2;
}

template <typename T, int DP, bool kExact>
hipError_t run_chunk(const AttendPlan& p, const Cache& c, const Batch& b, const Rows& q,
                     const Rows& out, float scale, uint32_t window, bool causal, float* lse,
                     Partial part, hipStream_t s) {
  hipLaunchKernelGGL((k_kv_chunk<T, DP, kExact>), dim3((uint32_t)p.blocks), dim3(kThreads), 0, s, c, b, q,
                     out, scale, window, causal, p.row_tiles, p.by_length, part, lse);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk(const AttendPlan& p, const Cache& c, uint32_t dtype, const Batch& b,
                        const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                        float* lse, Partial part, hipStream_t s) {
#define IBP_KV_CHUNK(T, DP, E) \
  run_chunk<T, DP, E>(p, c, b, q, out, scale, window, causal, lse, part, s)
#define IBP_KV_CHUNK_T(T)                                                                      \
  (c.head_dim == 64    ? IBP_KV_CHUNK(T, 64, true)                                             \
   : c.head_dim < 64   ? IBP_KV_CHUNK(T, 64, false)                                            \
   : c.head_dim <= 96  ? IBP_KV_CHUNK(T, 96, false)                                            \
   : c.head_dim < 128  ? IBP_KV_CHUNK(T, 128, false)                                           \
   : c.head_dim == 128 ? IBP_KV_CHUNK(T, 128, true)                                            \
   : c.head_dim <= 192 ? IBP_KV_CHUNK(T, 192, false)                                           \
   : c.head_dim < 256  ? IBP_KV_CHUNK(T, 256, false)                                           \
                       : IBP_KV_CHUNK(T, 256, true))
  return dtype == IBP_KV_F16 ? IBP_KV_CHUNK_T(_Float16) : IBP_KV_CHUNK_T(__bf16);
#undef IBP_KV_CHUNK_T
#undef IBP_KV_CHUNK
}

}  // namespace kv
}  // namespace ibp
