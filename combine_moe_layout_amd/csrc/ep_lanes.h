// ep_lanes.h -- exchanges and reductions between neighbouring lanes of a wave,
// in registers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

// All-reductions over L neighbouring lanes (a power of two, 4 to 64).  Within a row of
// 16 lanes the DPP controls are exchanges: neighbours, pairs, the mirrored half row and the
// mirrored row (the lanes of a half are equal by then); gfx950 swaps rows and half waves by
// v_permlane16_swap and v_permlane32_swap.  Every lane of the wave must be active.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, true);
}
template <int kStep>
__device__ __forceinline__ void exchange(uint32_t v, uint32_t& a, uint32_t& b) {
  a = v;
  if constexpr (kStep == 0) b = dpp<0xB1>(v);        // quad_perm [1, 0, 3, 2]
  else if constexpr (kStep == 1) b = dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  else if constexpr (kStep == 2) b = dpp<0x141>(v);  // row_half_mirror
  else if constexpr (kStep == 3) b = dpp<0x140>(v);  // row_mirror
  else if constexpr (kStep == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  }
}
template <int kStep, typename T>
__device__ __forceinline__ void exchange_any(T v, T& a, T& b) {
  if constexpr (sizeof(T) == 4) {
    uint32_t x, y;
    exchange<kStep>(__builtin_bit_cast(uint32_t, v), x, y);
    a = __builtin_bit_cast(T, x);
    b = __builtin_bit_cast(T, y);
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t xl, yl, xh, yh;
    exchange<kStep>((uint32_t)u, xl, yl);
    exchange<kStep>((uint32_t)(u >> 32), xh, yh);
    a = __builtin_bit_cast(T, (uint64_t)xh << 32 | xl);
    b = __builtin_bit_cast(T, (uint64_t)yh << 32 | yl);
  }
}
template <int L, int kStep = 0, typename T, typename F>
__device__ __forceinline__ T reduce(T v, F op) {
  if constexpr ((1 << kStep) >= L) {
    return v;
  } else {
    T a, b;
    exchange_any<kStep>(v, a, b);
    return reduce<L, kStep + 1>(op(a, b), op);
  }
}
template <int L, typename T>
__device__ __forceinline__ T reduce_max(T v) {
  return reduce<L>(v, [](T a, T b) { return a > b ? a : b; });
}
template <int L, typename T>
__device__ __forceinline__ T reduce_sum(T v) {
  return reduce<L>(v, [](T a, T b) { return a + b; });
}

}  // namespace ep
