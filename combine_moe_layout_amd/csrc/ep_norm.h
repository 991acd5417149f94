// ep_norm.h -- the block norms' launchers (ep_norm.hip).
#pragma once

#include "ep_gemm.h"
#include "ep_lanes.h"

namespace ep {

struct NormArgs {
  const void* y;            // the block's output, or NULL
  const void* post_weight;  // its norm's weight, or NULL: y as it is
  const float* gate;        // of every row, or NULL: 1
  const void* residual;     // or NULL
  float residual_scale;
  const void* pre_weight;   // the next norm's weight, or NULL
  int64_t rows;
  int32_t hidden;
  float eps;
  // forward
  void* out;
  void* normed;
  // gradient (outputs may be NULL)
  const void* d_out;
  const void* d_normed;
  void* d_y;
  void* d_residual;
  float* d_gate;
  void* d_post_weight;
  void* d_pre_weight;
  bool grad_f32, accumulate;
  float* partial;           // [2][norm_partials(rows, hidden)][hidden]
};

// Partial sums of each weight's gradient.
int64_t norm_partials(int64_t rows, int32_t hidden);

hipError_t launch_block_norm(const NormArgs& a, bool f16, hipStream_t stream);
hipError_t launch_block_norm_grad(const NormArgs& a, bool f16, hipStream_t stream);

}  // namespace ep
