// ep_route.h -- the router's launchers (ep_route.hip).
#pragma once

#include <type_traits>

#include "ep_gemm.h"
#include "ep_lanes.h"

namespace ep {

struct RouteArgs {
  int32_t E, k;
  int32_t groups, topk_groups, group_top;
  int32_t softmax;      // scores: softmax, else sigmoid
  int32_t renormalize;
  float scale;
  int32_t group_shift;  // set by the launcher: a group is 2^group_shift whole lanes, or -1: not so
  int32_t shared;       // set by the launcher: bytes of LDS of one token for the groups
};

// dtype: EP_F32, EP_BF16 or EP_F16.
hipError_t launch_route(const void* logits, const float* bias, int64_t tokens, RouteArgs a, int32_t dtype,
                        int64_t* idx, float* weights, hipStream_t stream);
hipError_t launch_route_grad(const float* dweights, const void* logits, const int64_t* idx, int64_t tokens,
                             const RouteArgs& a, int32_t dtype, void* dlogits, hipStream_t stream);

}  // namespace ep
