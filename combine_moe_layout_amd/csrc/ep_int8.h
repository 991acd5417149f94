// ep_int8.h -- launchers of the 8-bit integer rows (ep_int8.hip) and products
// (ep_gemm_int8.hip).
#pragma once

#include "ep_gemm.h"
#include "ep_lanes.h"

namespace ep {

hipError_t launch_dispatch_int8(const void* x, const ep_layout_t& L, int32_t hidden, void* recv_x,
                                void* recv_scales, hipStream_t stream);

// The used rows of `groups` (a layout's, or one dense group).
hipError_t launch_quantize_int8(const void* x, const RowGroups& groups, int32_t n, bool f16, void* q,
                                float* scales, hipStream_t stream);

// Sums of codes' products are at most 2^30, so that times a row's scale past 2^98 one may leave fp32's range
// where the result does not.  A row's large scale is taken in two factors: the results get 2^32 at the end
// (before that they are in the normal range, for the smaller factor is at least 2^58).
constexpr float kLargeScale = 0x1p90f, kLargePart = 0x1p32f;
__device__ __forceinline__ bool split_scale(float& row) {
  const bool large = fabsf(row) > kLargeScale;
  row = large ? row * (1.0f / kLargePart) : row;
  return large;
}

// a, b: int8; a_scales [rows] and b_scales [E, columns of the product] fp32.
hipError_t launch_gemm_int8(const GemmArgs& g, hipStream_t stream);
// Tiles of 16, 32 or 64 rows and as many columns.
hipError_t launch_gemm_int8_few(const GemmArgs& g, int32_t height, int32_t width, hipStream_t stream);

}  // namespace ep
