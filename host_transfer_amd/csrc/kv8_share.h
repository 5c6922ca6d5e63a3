// kv8_share.h -- the keys of all sequences shared out over workgroups by their number, in the kernel.
#pragma once

#include "kv8.h"
#include "kv_wave.h"

namespace ibp {
namespace kv {

// The item (a sequence, or a tile of its rows) and split of workgroup `place` of its head group: with
// n_s = max(ceil(tiles_s / size), 1) workgroups for an item that has rows, size the least length from `least` on
// with which all items' are at most `shares` (or the longest's, where the items are more); items in their
// order.  s < 0: there is none for it.
//   mine    2 * tiles + 1 of item `lane`, 0 where it has no rows; others', past 64, in `tiles`
struct Part8 {
  int32_t s, split, splits, place;  // place: the item's first workgroup
};
__device__ __forceinline__ Part8 part_of(uint32_t mine, const uint32_t* tiles, uint32_t n_seqs, uint32_t shares,
                                         uint32_t place, uint32_t lane, uint32_t least = 1) {
  auto at = [&](uint32_t j0) -> uint32_t { return j0 == 0 ? mine : j0 + lane < n_seqs ? tiles[j0 + lane] : 0; };
  uint32_t total = 0, most = 0, active = 0;
  for (uint32_t j0 = 0; j0 < n_seqs; j0 += kWave) {
    const uint32_t t = at(j0);
    total += wave_sum(t >> 1);
    most = max(most, wave_max(t >> 1));
    active += (uint32_t)__builtin_popcountll(__ballot(t & 1u));
  }
  // lo may be too short, hi is not: sum of ceil(t / hi) <= total / hi + active
  uint32_t lo = max((total + shares - 1) / shares, least), hi = max(most, 1u);
  if (shares > active) hi = min(hi, (total + shares - active - 1) / (shares - active));
  hi = max(hi, lo);
  auto splits = [&](uint32_t t, uint32_t size) { return t ? max(((t >> 1) + size - 1) / size, 1u) : 0u; };
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    uint32_t n = 0;
    for (uint32_t j0 = 0; j0 < n_seqs; j0 += kWave) n += wave_sum(splits(at(j0), mid));
    if (n <= shares) hi = mid;
    else lo = mid + 1;
  }
  Part8 p = {-1, 0, 0, 0};
  uint32_t before = 0;
  for (uint32_t j0 = 0; j0 < n_seqs && p.s < 0; j0 += kWave) {
    const uint32_t n = splits(at(j0), hi), upto = before + wave_prefix_sum(n);
    const uint64_t here = __ballot(n && place >= upto - n && place < upto);
    if (here) {
      const uint32_t l = (uint32_t)__builtin_ctzll(here);
      p.s = (int32_t)(j0 + l);
      p.splits = (int32_t)lane_u32(n, l);
      p.place = (int32_t)(lane_u32(upto, l) - lane_u32(n, l));
      p.split = (int32_t)place - p.place;
    }
    before = lane_u32(upto, kWave - 1);
  }
  return p;
}
// Tiles of a part of an item of `tiles`: its parts are as even as they can be, none longer than `size`.
__device__ __forceinline__ int32_t part_tiles(const Part8& p, int32_t tiles) {
  return (tiles + p.splits - 1) / p.splits;
}

}  // namespace kv
}  // namespace ibp
