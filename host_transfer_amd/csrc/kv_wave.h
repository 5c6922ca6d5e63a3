// kv_wave.h -- sums over a wave's lanes without LDS, for the planning parts of the serving kernels.
#pragma once

#include "ibp_device.h"

namespace ibp {

// Lane moves of the vector ALU, a few cycles each (through LDS some 100): x of the lane that kCtrl names,
// 0 where there is none; rows of 16 lanes outside kRows get 0.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xf, false);
}
// Combines every lane's value with those of the lanes before it; 0 has to be neutral.
template <typename F>
__device__ __forceinline__ uint32_t wave_prefix(uint32_t x, F op) {
  x = op(x, moved<0x111, 0xf>(x));  // within rows, 1, 2, 4 and 8 lanes further
  x = op(x, moved<0x112, 0xf>(x));
  x = op(x, moved<0x114, 0xf>(x));
  x = op(x, moved<0x118, 0xf>(x));
  x = op(x, moved<0x142, 0xa>(x));  // a row's last lane to the next row, the second's to the last two
  x = op(x, moved<0x143, 0xc>(x));
  return x;
}
__device__ __forceinline__ uint32_t wave_prefix_sum(uint32_t x) {
  return wave_prefix(x, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ uint32_t wave_sum(uint32_t x) { return lane_u32(wave_prefix_sum(x), kWave - 1); }
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  return lane_u32(wave_prefix(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; }), kWave - 1);
}

}  // namespace ibp
