// wave.h -- reductions over a 64-lane wavefront or groups of its lanes by DPP.
// Every lane of the group has to be active. The order of a sum is fixed.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace wt {

// Max over the L lanes of each aligned L-lane group (DPP within 16-lane rows;
// lanes read from outside the group take no part), left in every lane.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x0B1, 0xF, 0xF, false));  // quad_perm [1,0,3,2]
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x04E, 0xF, 0xF, false));  // quad_perm [2,3,0,1]
  if (L >= 8) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));  // row_half_mirror
  if (L >= 16) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));  // row_mirror
  return m;
}

// Over the whole wavefront; the result is uniform.

template <int Ctrl, int RowMask>
__device__ __forceinline__ float dpp_f32(float old, float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), Ctrl, RowMask, 0xF, false));
}

__device__ __forceinline__ float lane63(float x) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Lane i's value (i uniform).
__device__ __forceinline__ float lane_value(float x, int i) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), i));
}

// A NaN takes no part in the maximum (of a number and a NaN the number wins).
__device__ __forceinline__ float wave_max(float m) {
  m = fmaxf(m, dpp_f32<0x0B1, 0xF>(m, m));  // quad_perm [1,0,3,2]
  m = fmaxf(m, dpp_f32<0x04E, 0xF>(m, m));  // quad_perm [2,3,0,1]
  m = fmaxf(m, dpp_f32<0x141, 0xF>(m, m));  // row_half_mirror
  m = fmaxf(m, dpp_f32<0x140, 0xF>(m, m));  // row_mirror: every row of 16 has its maximum
  m = fmaxf(m, dpp_f32<0x142, 0xA>(m, m));  // rows 1 and 3 take in rows 0 and 2
  m = fmaxf(m, dpp_f32<0x143, 0xC>(m, m));  // rows 2 and 3 take in row 1
  return lane63(m);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t m) {
  m = lanes_max<16>(m);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x142, 0xA, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x143, 0xC, 0xF, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)m, 63);
}

// Orders a wave's accesses to shared memory that only this wave touches: what
// its lanes wrote before is what any of them reads behind.
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

__device__ __forceinline__ float wave_sum(float x) {
  x += dpp_f32<0x0B1, 0xF>(0.0f, x);
  x += dpp_f32<0x04E, 0xF>(0.0f, x);
  x += dpp_f32<0x141, 0xF>(0.0f, x);
  x += dpp_f32<0x140, 0xF>(0.0f, x);
  x += dpp_f32<0x142, 0xA>(0.0f, x);
  x += dpp_f32<0x143, 0xC>(0.0f, x);
  return lane63(x);
}

}  // namespace wt
