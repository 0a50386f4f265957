// wave_ops.h -- reductions over the 64 lanes of a wave by data-parallel moves (a shuffle through
// LDS costs over a hundred cycles).
#pragma once

#include "common.h"

namespace int8w {

// The moved value, or `v` itself where the move has no source.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_self(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp((int)__float_as_uint(v), (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_self(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  u32x2 m;
  m.x = (uint32_t)__builtin_amdgcn_update_dpp((int)w.x, (int)w.x, CTRL, ROWS, 0xF, false);
  m.y = (uint32_t)__builtin_amdgcn_update_dpp((int)w.y, (int)w.y, CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, m);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_zero(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xF, true));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  u32x2 w = __builtin_bit_cast(u32x2, v);
  w.x = (uint32_t)__builtin_amdgcn_readlane((int)w.x, 63);
  w.y = (uint32_t)__builtin_amdgcn_readlane((int)w.y, 63);
  return __builtin_bit_cast(double, w);
}

// Maximum over the wave, in every lane.
template <class T>
__device__ __forceinline__ T wave_max(T v) {
  v = fmax(v, dpp_or_self<0x111, 0xF>(v));  // row_shr:1
  v = fmax(v, dpp_or_self<0x112, 0xF>(v));
  v = fmax(v, dpp_or_self<0x114, 0xF>(v));
  v = fmax(v, dpp_or_self<0x118, 0xF>(v));
  v = fmax(v, dpp_or_self<0x142, 0xA>(v));  // row_bcast:15
  v = fmax(v, dpp_or_self<0x143, 0xC>(v));  // row_bcast:31
  return last_lane(v);
}

// Sum over the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_add(float v) {
  v += dpp_or_zero<0x111, 0xF>(v);
  v += dpp_or_zero<0x112, 0xF>(v);
  v += dpp_or_zero<0x114, 0xF>(v);
  v += dpp_or_zero<0x118, 0xF>(v);
  v += dpp_or_zero<0x142, 0xA>(v);
  v += dpp_or_zero<0x143, 0xC>(v);
  return last_lane(v);
}

}  // namespace int8w
