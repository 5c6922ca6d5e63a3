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

// A workgroup per (128 rows that share a key head, split of their keys); a
// wave holds 32 rows: their queries, and their outputs transposed.  Steps of 64 keys:
// K and V rows of the next step are loaded into registers (one page lookup a lane, a
// step further ahead) while this one is worked on, then written to the other
// half of LDS; one barrier a step.
//
// LDS rows are padded: a K row by 16 B, so that the 16 rows a quarter of the wave reads at
// one channel lie in 16 different 16 B slots of the banks; a V row to an odd multiple of
// 64 B, so that the four rows of half a transposed read lie in four 64 B windows.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void k_kv_chunk(Cache cache, Batch b, Rows q, Rows out,
                                                       float scale, uint32_t window, bool causal,
                                                       uint32_t row_tiles, Partial part,
                                                       float* __restrict__ lse) {
  constexpr int KS = DP / 16;                   // products of a score
  constexpr int DT = DP / 32;                   // tiles of the output
  constexpr int CH = DP / 8;                    // 16 B pieces of a row
  constexpr int LK = DP + 8;                    // LDS rows, elements
  constexpr int LV = DP + (DP % 64 == 0 ? 32 : 0);
  constexpr int ST = kKeys * CH / kThreads;     // pieces a thread brings of K and of V
  static_assert(kKeys * CH % kThreads == 0, "pieces divide among the threads");
  __shared__ __align__(16) uint16_t s_k[2][kKeys * LK];
  __shared__ __align__(16) uint16_t s_v[2][kKeys * LV];
  __shared__ uint32_t s_odd;

  const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const uint32_t col = lane % 32, half = lane / 32;
  const uint32_t group = q.n_heads / cache.n_heads, hd = cache.head_dim;

  // block -> key head (innermost: blocks of one head meet in one XCD's L2 where the heads
  // are a multiple of eight), split, sequence, row tile from the last (under a
  // causal mask the longest)
  uint32_t u = blockIdx.x;
  const uint32_t kh = u % cache.n_heads;
  u /= cache.n_heads;
  const uint32_t split = u % part.splits;
  u /= part.splits;
  const uint32_t s = u % b.n_seqs;
  const uint32_t tile = row_tiles - 1 - u / b.n_seqs;

  const Seq sq = load_seq(b, s);
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
  const uint32_t wm0 = min(m0 + wave * 32, m1 - 1), wm1 = min(m0 + wave * 32 + 32, m1);
  const bool active = m0 + wave * 32 < m1;
  const int32_t w_lo = lo_of(pos_of(wm0)), w_hi = hi_of(pos_of(active ? wm1 - 1 : wm0));
  const int32_t full_lo = lo_of(pos_of(active ? wm1 - 1 : wm0)), full_hi = hi_of(pos_of(wm0));
  const bool have = m0 + wave * 32 + col < m1;
  const uint32_t m = have ? m0 + wave * 32 + col : m1 - 1;
  const int32_t pos = pos_of(m), lo = lo_of(pos), hi = hi_of(pos);
  const uint32_t row = (uint32_t)sq.row0 + m / group, head = kh * group + m % group;

  const int32_t from = blk_lo / kKeys * kKeys;
  const int32_t tiles = max(blk_hi - from + kKeys - 1, 0) / kKeys;
  const int32_t per = (tiles + (int32_t)part.splits - 1) / (int32_t)part.splits;
  const int32_t begin = from + min((int32_t)split * per, tiles) * kKeys;
  const int32_t end = from + min(((int32_t)split + 1) * per, tiles) * kKeys;

  // queries, their sign that of the scale (the maximum below is of unscaled scores)
  const T* qp = (const T*)q.p + row * q.token_stride + (uint64_t)head * q.head_stride;
  const T* zeros = (const T*)zero_row;
  V8<T> qf[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const uint32_t c = k * 16 + half * 8;
    qf[k] = load_row8(have && c < hd && scale != 0.f ? qp + c : zeros);
    if (scale < 0.f) qf[k] = -qf[k];
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

  // page id of key t0 + lane (-1: no row sees it)
  auto lookup = [&](int32_t t0) -> int32_t {
    const int32_t j = t0 + (int32_t)lane;
    return t0 < end && j >= blk_lo && j < blk_hi ? table[cache.page.div((uint32_t)j)] : -1;
  };
  V8<T> kr[ST], vr[ST];
  uint64_t there = 0;  // of the step whose rows are in the registers
  auto fetch = [&](int32_t t0, int32_t id) {
    const uint32_t j = (uint32_t)(t0 + (int32_t)lane);
    const bool see = id >= 0 && (uint32_t)id < cache.n_pages;
    const uint64_t at = (uint64_t)(uint32_t)id * cache.page_stride +
                        (uint64_t)(j - cache.page.div(j) * cache.page.d) * cache.token_stride;
    there = __ballot(see);
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      const uint32_t e = tid + i * kThreads;
      const uint32_t r = e / CH, c = (e % CH) * 8;
      const uint64_t a = ((uint64_t)(uint32_t)__shfl((int)(uint32_t)(at >> 32), (int)r) << 32) |
                         (uint32_t)__shfl((int)(uint32_t)at, (int)r);
      const bool ok = ((there >> r) & 1u) && c < hd;
      kr[i] = load_row8(ok ? kbase + a + c : zeros);
      vr[i] = load_row8(ok ? vbase + a + c : zeros);
    }
  };

  int32_t id = lookup(begin);
  if (begin < end) fetch(begin, id);
  id = lookup(begin + kKeys);
  if (tid == 0) s_odd = 0;
  bool odd = false;
  auto is_edge = [&](int32_t t0) { return t0 < edge_lo || t0 + kKeys > edge_hi; };
  // this lane's part of a transposed read of V
  const uint32_t tr_at = (4 * half + (lane % 16) / 4) * LV + 16 * ((lane / 16) % 2) + 4 * (lane % 4);
  uint32_t buf = 0;
  for (int32_t t0 = begin; t0 < end; t0 += kKeys, buf ^= 1) {
    uint16_t *sk = s_k[buf], *sv = s_v[buf];
    // a key that some rows see and others do not: no infinity or NaN of its values
    // may enter the product (what they add comes after the loop)
    if (is_edge(t0)) {
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        odd = odd || any_odd<T>(vr[i]);
        vr[i] = finite_part<T>(vr[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      const uint32_t e = tid + i * kThreads;
      const uint32_t r = e / CH, c = (e % CH) * 8;
      *(V8<T>*)(sk + r * LK + c) = kr[i];
      *(V8<T>*)(sv + r * LV + c) = vr[i];
    }
    const uint64_t seen = there;
    if (t0 + kKeys < end) fetch(t0 + kKeys, id);
    id = lookup(t0 + 2 * kKeys);
    lds_barrier();

    if (active && t0 < w_hi && t0 + kKeys > w_lo) {
      f32x16 sc[2];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[a][r] = 0.f;
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const V8<T> kf = *(const V8<T>*)(sk + (a * 32 + col) * LK + k * 16 + half * 8);
          sc[a] = mfma32(kf, qf[k], sc[a]);
        }
      __builtin_amdgcn_s_setprio(0);
      settle(sc[0], sc[1]);
      // register r of tile a: key t0 + 32 a + 8 (r / 4) + 4 half + r % 4
      if (!(seen == ~0ull && t0 >= full_lo && t0 + kKeys <= full_hi)) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const uint32_t kk = a * 32 + 8 * (r / 4) + 4 * half + r % 4;
            const int32_t j = t0 + (int32_t)kk;
            if (!((seen >> kk) & 1u) || j < lo || j >= hi) sc[a][r] = -INFINITY;
          }
      }
      float most = sc[0][0];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) most = fmaxf(most, sc[a][r]);
      most = max_half(most) * sc2;
      // The base that exponents are taken against follows the maximum only when it is
      // passed by 2^8: weights then stay below 2^8 (as exact in the dtype as below 1,
      // and far from its largest number), and most steps need no rescaling.
      if (__any(most > top + 8.f)) {
        const float next = fmaxf(top, most);
        const float keep = exp2_raw(top - (next == -INFINITY ? 0.f : next));
        z *= keep;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[t][r] *= keep;
        top = next;
      }
      const float base = top == -INFINITY ? 0.f : top;
      V8<T> p[4];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float y = exp2_raw(fmaf(sc[a][r], sc2, -base));
          z += y;
          // half a step of the dtype, relative, as the output's own rounding
          p[a * 2 + r / 8][r % 8] = (T)y;
        }
      const uint16_t* at = sv + tr_at;
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int t = 0; t < DT; ++t) {
          const T* v = (const T*)at + 16 * k * LV + t * 32;
          o[t] = mfma32(join<T>(read_tr(v), read_tr(v + 8 * LV)), p[k], o[t]);
        }
      __builtin_amdgcn_s_setprio(0);
    }
  }

  settle(o);
  lds_barrier();
  if (odd) s_odd = 1;
  lds_barrier();
  if (s_odd) {
    for (int32_t t0 = begin; t0 < end; t0 += kKeys) {
      if (!is_edge(t0)) continue;
      fetch(t0, lookup(t0));
      uint16_t* sv = s_v[0];
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        const uint32_t e = tid + i * kThreads;
        *(V8<T>*)(sv + (e / CH) * LV + (e % CH) * 8) = odd_code<T>(vr[i]);
      }
      lds_barrier();
      V8<T> sees[4];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const uint32_t kk = 32 * (e / 16) + 8 * ((e / 4) % 4) + 4 * half + e % 4;
        const int32_t j = t0 + (int32_t)kk;
        sees[e / 8][e % 8] = (T)(((there >> kk) & 1u) && j >= lo && j < hi ? 1.f : 0.f);
      }
      const uint16_t* at = sv + tr_at;
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        f32x16 n;
#pragma unroll
        for (int r = 0; r < 16; ++r) n[r] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const T* v = (const T*)at + 16 * k * LV + t * 32;
          n = mfma32(join<T>(read_tr(v), read_tr(v + 8 * LV)), sees[k], n);
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
      for (int e = 0; e < 4; ++e) v[e] = (T)(o[t][4 * r + e] * inv);
      if (c < hd) *(t4*)(op + c) = v;
    }
  if (lse && half == 0) lse[unit] = z == 0.f ? -INFINITY : (top + __builtin_amdgcn_logf(z)) * kLn2;
}

template <typename T, int DP>
hipError_t run_chunk(const AttendPlan& p, const Cache& c, const Batch& b, const Rows& q,
                     const Rows& out, float scale, uint32_t window, bool causal, float* lse,
                     Partial part, hipStream_t s) {
  hipLaunchKernelGGL((k_kv_chunk<T, DP>), dim3((uint32_t)p.blocks), dim3(kThreads), 0, s, c, b, q,
                     out, scale, window, causal, p.row_tiles, part, lse);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk(const AttendPlan& p, const Cache& c, uint32_t dtype, const Batch& b,
                        const Rows& q, const Rows& out, float scale, uint32_t window, bool causal,
                        float* lse, Partial part, hipStream_t s) {
#define IBP_KV_CHUNK(T, DP) \
  run_chunk<T, DP>(p, c, b, q, out, scale, window, causal, lse, part, s)
#define IBP_KV_CHUNK_T(T)                                                                     \
  (c.head_dim <= 64    ? IBP_KV_CHUNK(T, 64)                                                  \
   : c.head_dim <= 96  ? IBP_KV_CHUNK(T, 96)                                                  \
   : c.head_dim <= 128 ? IBP_KV_CHUNK(T, 128)                                                 \
   : c.head_dim <= 192 ? IBP_KV_CHUNK(T, 192)                                                 \
                       : IBP_KV_CHUNK(T, 256))
  return dtype == IBP_KV_F16 ? IBP_KV_CHUNK_T(_Float16) : IBP_KV_CHUNK_T(__bf16);
#undef IBP_KV_CHUNK_T
#undef IBP_KV_CHUNK
}

}  // namespace kv
}  // namespace ibp
