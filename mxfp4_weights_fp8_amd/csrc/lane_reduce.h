// Reductions over 16 or 64 neighbouring lanes without LDS, and the ordering of LDS
// accesses between the lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Reductions over the LPR lanes of a row, the result in all of them: within 16 lanes
// by DPP (xor 1, xor 2, then mirrored halves and rows, which cost no LDS access as a
// shuffle does), then gfx950's lane-half swaps.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, true);
}
template <int LPR, typename F>
__device__ __forceinline__ int row_reduce(int v, F f) {
  static_assert(LPR == 16 || LPR == 64, "lanes per row");
  v = f(v, dpp<0xB1>(v));    // quad_perm [1, 0, 3, 2]
  v = f(v, dpp<0x4E>(v));    // quad_perm [2, 3, 0, 1]
  v = f(v, dpp<0x141>(v));   // row_half_mirror
  v = f(v, dpp<0x140>(v));   // row_mirror
  if constexpr (LPR == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
    v = f((int)a[0], (int)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    v = f((int)b[0], (int)b[1]);
  }
  return v;
}
template <int LPR>
__device__ __forceinline__ int row_max(int v) {
  return row_reduce<LPR>(v, [](int a, int b) { return max(a, b); });
}
template <int LPR>
__device__ __forceinline__ int row_min(int v) {
  return row_reduce<LPR>(v, [](int a, int b) { return min(a, b); });
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  return __int_as_float(row_reduce<LPR>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  return __int_as_float(row_reduce<LPR>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

// LDS accesses of the wave's lanes before this are seen by all of its lanes after it: a
// wave's LDS operations complete in order, so this only keeps the compiler from moving
// them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace moe
