// ep_norm.hip -- the norm after a block with its gate and residual scale, the norm before the
// next block, and their gradients.
//
//   s = (mean(y^2) + eps)^-1/2,  b = y s post        (without a post weight: b = y)
//   x = alpha residual + gate_t b                    -> out, rounded
//   r = (mean(x^2) + eps)^-1/2,  normed = x r pre    (of the unrounded x) -> normed, rounded
//
// Bound by HBM: y and the residual are read once, out and normed written once.  A row stays in
// the registers of its lanes, V vectors of 8 channels each, through both sums.
//
// Gradient, with D = sum(dx post y), everything recomputed from the forward's inputs:
//   dx = d_out + r (pre dn) - x r^3 mean(pre dn x)        d_residual = alpha dx
//   d_gate = s D       d_y = gate (s post dx - y s^3 D / hidden)
//   d_post = sum over rows of gate dx y s                 d_pre = sum over rows of dn x r
// A workgroup walks rows and keeps its sums of d_post and d_pre in registers; they meet in a
// second kernel in a fixed order, so the result does not depend on timing.
#include <type_traits>

#include "ep_norm.h"

namespace ep {

namespace {

constexpr int kMaxLanes = 1024;
constexpr int kMaxWaves = kMaxLanes / 64;

template <bool kF16>
__device__ __forceinline__ void unpack8(const u32x4& d, float* f) {
  const uint32_t u[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = elem_low<kF16>(u[i]);
    f[2 * i + 1] = elem_high<kF16>(u[i]);
  }
}
template <bool kF16>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  return u32x4{elem_rne2<kF16>(f[0], f[1]), elem_rne2<kF16>(f[2], f[3]), elem_rne2<kF16>(f[4], f[5]),
               elem_rne2<kF16>(f[6], f[7])};
}

// Sums of N values over the `lanes` threads of a row (whole waves), the same in each of them
// and added in a fixed order.  `part`: the row's floats in LDS, N to a wave, that nobody else
// uses until the next barrier after this one.  Rows of one wave need neither.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int lanes, float* part) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = reduce_sum<64>(v[i]);
  if (lanes == 64) return;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[wave * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < lanes / 64; ++w) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += part[w * N + i];
  }
}
__device__ __forceinline__ float inverse_rms(float squares, int32_t hidden, float eps) {
  return 1.0f / sqrtf(squares / (float)hidden + eps);
}

// lanes: threads of one row; the block holds blockDim / lanes rows (one, if lanes > 64).
template <bool kF16, int V>
__global__ __launch_bounds__(kMaxLanes) void block_norm_kernel(NormArgs a, int32_t lanes) {
  __shared__ float part[2][kMaxWaves];
  const int lane = threadIdx.x % lanes, local = threadIdx.x / lanes;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / lanes) + local;
  if (row >= a.rows) return;  // a whole wave, and no barrier follows in such a block
  const int32_t vecs = a.hidden / 8;
  const u32x4* const y = static_cast<const u32x4*>(a.y) + row * vecs;
  const u32x4* const res = static_cast<const u32x4*>(a.residual) + row * vecs;
  const u32x4* const post = static_cast<const u32x4*>(a.post_weight);
  const u32x4* const pre = static_cast<const u32x4*>(a.pre_weight);
  const u32x4 zero = {0, 0, 0, 0};
  u32x4 yv[V], rv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = lane + i * lanes;
    yv[i] = a.y != nullptr && v < vecs ? y[v] : zero;
    rv[i] = a.residual != nullptr && v < vecs ? res[v] : zero;
  }
  float scale = a.gate != nullptr ? a.gate[row] : 1.0f;
  float s = 1.0f;
  if (a.post_weight != nullptr) {
    float squares[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8<kF16>(yv[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) squares[0] = fmaf(f[k], f[k], squares[0]);
    }
    row_sums(squares, lanes, part[0]);
    s = inverse_rms(squares[0], a.hidden, a.eps);
  }
  float x[V][8], squares[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = lane + i * lanes;
    float f[8], r[8];
    unpack8<kF16>(yv[i], f);
    unpack8<kF16>(rv[i], r);
    if (a.post_weight != nullptr) {
      float w[8];
      unpack8<kF16>(v < vecs ? post[v] : zero, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = f[k] * s * w[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[i][k] = fmaf(scale, f[k], a.residual_scale * r[k]);
      squares[0] = fmaf(x[i][k], x[i][k], squares[0]);
    }
    if (a.out != nullptr && v < vecs) static_cast<u32x4*>(a.out)[row * vecs + v] = pack8<kF16>(x[i]);
  }
  if (a.normed == nullptr) return;
  row_sums(squares, lanes, part[1]);
  const float r = inverse_rms(squares[0], a.hidden, a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = lane + i * lanes;
    if (v >= vecs) continue;
    float w[8];
    unpack8<kF16>(pre[v], w);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] *= x[i][k] * r;
    static_cast<u32x4*>(a.normed)[row * vecs + v] = pack8<kF16>(w);
  }
}

// One block walks rows blockIdx, blockIdx + gridDim, .. (times its rows).  `partials`: how many
// sums of the weights' gradients there are; block b's row group writes number b * rows + group.
template <bool kF16, int V>
__global__ __launch_bounds__(kMaxLanes) void block_norm_grad_kernel(NormArgs a, int32_t lanes, int64_t partials) {
  __shared__ float part[2][3][2 * kMaxWaves];
  const int lane = threadIdx.x % lanes, local = threadIdx.x / lanes;
  const int64_t here = blockDim.x / lanes;
  const int32_t vecs = a.hidden / 8;
  const u32x4 *const y = static_cast<const u32x4*>(a.y), *const res = static_cast<const u32x4*>(a.residual);
  const u32x4 *const dout = static_cast<const u32x4*>(a.d_out), *const dn = static_cast<const u32x4*>(a.d_normed);
  const u32x4* const post = static_cast<const u32x4*>(a.post_weight);
  const u32x4* const pre = static_cast<const u32x4*>(a.pre_weight);
  const bool has_pre = dn != nullptr, has_post = post != nullptr;
  const u32x4 zero = {0, 0, 0, 0};
  const float mean = 1.0f / (float)a.hidden;
  float sum_post[V][8] = {}, sum_pre[V][8] = {};
  int turn = 0;
  for (int64_t row = blockIdx.x * here + local; row < a.rows; row += gridDim.x * here, turn ^= 1) {
    const int64_t at = row * vecs;
    u32x4 yv[V], nv[V];
    float x[V][8], dx[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = lane + i * lanes;
      const bool ok = v < vecs;
      yv[i] = y != nullptr && ok ? y[at + v] : zero;
      nv[i] = has_pre && ok ? dn[at + v] : zero;
      unpack8<kF16>(has_pre && res != nullptr && ok ? res[at + v] : zero, x[i]);
      unpack8<kF16>(dout != nullptr && ok ? dout[at + v] : zero, dx[i]);
    }
    const float gate = a.gate != nullptr ? a.gate[row] : 1.0f;
    float s = 1.0f;
    if (has_post) {
      float squares[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8<kF16>(yv[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) squares[0] = fmaf(f[k], f[k], squares[0]);
      }
      row_sums(squares, lanes, part[turn][0]);
      s = inverse_rms(squares[0], a.hidden, a.eps);
    }
    if (has_pre) {
      float sums[2] = {0.0f, 0.0f};  // x^2, pre dn x
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = lane + i * lanes;
        float f[8], w[8], d[8];
        unpack8<kF16>(yv[i], f);
        if (has_post) {
          unpack8<kF16>(v < vecs ? post[v] : zero, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = f[k] * s * w[k];
        }
        unpack8<kF16>(v < vecs ? pre[v] : zero, w);
        unpack8<kF16>(nv[i], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[i][k] = fmaf(gate, f[k], a.residual_scale * x[i][k]);
          sums[0] = fmaf(x[i][k], x[i][k], sums[0]);
          sums[1] = fmaf(d[k] * w[k], x[i][k], sums[1]);
        }
      }
      row_sums(sums, lanes, part[turn][1]);
      const float r = inverse_rms(sums[0], a.hidden, a.eps);
      const float back = r * r * r * (sums[1] * mean);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = lane + i * lanes;
        float w[8], d[8];
        unpack8<kF16>(v < vecs ? pre[v] : zero, w);
        unpack8<kF16>(nv[i], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sum_pre[i][k] = fmaf(d[k], x[i][k] * r, sum_pre[i][k]);
          dx[i][k] += fmaf(r, d[k] * w[k], -x[i][k] * back);
        }
      }
    }
    if (a.d_residual != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = lane + i * lanes;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = a.residual_scale * dx[i][k];
        if (v < vecs) static_cast<u32x4*>(a.d_residual)[at + v] = pack8<kF16>(o);
      }
    }
    if (y == nullptr) continue;
    float dot[1] = {0.0f};
    if (has_post || a.d_gate != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = lane + i * lanes;
        float f[8], w[8];
        unpack8<kF16>(yv[i], f);
        if (has_post) {
          unpack8<kF16>(v < vecs ? post[v] : zero, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sum_post[i][k] = fmaf(gate * dx[i][k], f[k] * s, sum_post[i][k]);
            dx[i][k] *= w[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) dot[0] = fmaf(dx[i][k], f[k], dot[0]);
      }
      row_sums(dot, lanes, part[turn][2]);
      if (a.d_gate != nullptr && lane == 0) a.d_gate[row] = s * dot[0];
    }
    if (a.d_y == nullptr) continue;
    const float along = gate * s, back = has_post ? gate * (s * s * s) * (dot[0] * mean) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = lane + i * lanes;
      float f[8];
      unpack8<kF16>(yv[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = fmaf(along, dx[i][k], -f[k] * back);
      if (v < vecs) static_cast<u32x4*>(a.d_y)[at + v] = pack8<kF16>(f);
    }
  }
  const int64_t mine = blockIdx.x * here + local;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.d_post_weight : a.d_pre_weight) == nullptr) continue;
    float* const to = a.partial + (which * partials + mine) * a.hidden;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = lane + i * lanes;
      const float* const f = which == 0 ? sum_post[i] : sum_pre[i];
      if (v < vecs) {
        reinterpret_cast<f32x4*>(to)[2 * v] = f32x4{f[0], f[1], f[2], f[3]};
        reinterpret_cast<f32x4*>(to)[2 * v + 1] = f32x4{f[4], f[5], f[6], f[7]};
      }
    }
  }
}

// The weights' gradients from their partial sums: a workgroup takes 64 channels of one of
// them, its 16 waves share out the partials and meet in LDS.
template <bool kF16>
__global__ __launch_bounds__(kMaxLanes) void norm_weights_kernel(const float* __restrict__ partial, int64_t partials,
                                                                 int32_t hidden, void* d_post, void* d_pre,
                                                                 bool f32, bool accumulate) {
  __shared__ float sums[kMaxWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t col = blockIdx.x * 64 + lane;
  void* const to = blockIdx.y == 0 ? d_post : d_pre;
  if (to == nullptr) return;
  float s = 0.0f;
  if (col < hidden)
    for (int64_t p = wave; p < partials; p += kMaxWaves) s += partial[(blockIdx.y * partials + p) * hidden + col];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= hidden) return;
  for (int w = 1; w < kMaxWaves; ++w) s += sums[w][lane];
  if (f32) {
    float* const p = static_cast<float*>(to) + col;
    *p = accumulate ? *p + s : s;
  } else {
    static_cast<uint16_t*>(to)[col] = elem_rne<kF16>(accumulate ? elem_at<kF16>(to, col) + s : s);
  }
}

// Threads of a row and vectors of each.
struct RowShape {
  int lanes, vectors;
  int rows_per_block() const { return lanes == 64 ? 4 : 1; }
};
RowShape row_shape(int32_t hidden, int most_vectors) {
  const int vecs = hidden / 8;
  int vectors = most_vectors;
  while (vectors > 1 && vecs <= 64 * (vectors / 2)) vectors /= 2;
  int lanes = ((vecs + vectors - 1) / vectors + 63) / 64 * 64;
  while (lanes > kMaxLanes) {
    vectors *= 2;
    lanes = ((vecs + vectors - 1) / vectors + 63) / 64 * 64;
  }
  return {lanes, vectors};
}
constexpr int kForwardVectors = 2, kGradVectors = 2;
constexpr int64_t kGradBlocks = 2 * kChipCUs;

template <bool kF16>
hipError_t forward(const NormArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.hidden, kForwardVectors);
  const int64_t blocks = (a.rows + s.rows_per_block() - 1) / s.rows_per_block();
  const int threads = s.lanes * s.rows_per_block();
  if (!grid_fits(blocks, threads)) return hipErrorInvalidValue;
  const auto run = [&](auto kernel) { kernel<<<(uint32_t)blocks, threads, 0, stream>>>(a, s.lanes); };
  if (s.vectors == 1) run(block_norm_kernel<kF16, 1>);
  else if (s.vectors == 2) run(block_norm_kernel<kF16, 2>);
  else if (s.vectors == 4) run(block_norm_kernel<kF16, 4>);
  else run(block_norm_kernel<kF16, 8>);
  return hipGetLastError();
}

int64_t grad_blocks(int64_t rows, const RowShape& s) {
  const int64_t most = (rows + s.rows_per_block() - 1) / s.rows_per_block();
  return most < kGradBlocks ? most : kGradBlocks;
}

template <bool kF16>
hipError_t gradient(const NormArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.hidden, kGradVectors);
  const int64_t blocks = grad_blocks(a.rows, s), partials = blocks * s.rows_per_block();
  const int threads = s.lanes * s.rows_per_block();
  if (blocks > 0) {
    const auto run = [&](auto kernel) { kernel<<<(uint32_t)blocks, threads, 0, stream>>>(a, s.lanes, partials); };
    if (s.vectors == 1) run(block_norm_grad_kernel<kF16, 1>);
    else if (s.vectors == 2) run(block_norm_grad_kernel<kF16, 2>);
    else if (s.vectors == 4) run(block_norm_grad_kernel<kF16, 4>);
    else run(block_norm_grad_kernel<kF16, 8>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.d_post_weight != nullptr || a.d_pre_weight != nullptr) {
    norm_weights_kernel<kF16><<<dim3((a.hidden + 63) / 64, 2), kMaxLanes, 0, stream>>>(
        a.partial, partials, a.hidden, a.d_post_weight, a.d_pre_weight, a.grad_f32, a.accumulate);
  }
  return hipGetLastError();
}

}  // namespace

int64_t norm_partials(int64_t rows, int32_t hidden) {
  const RowShape s = row_shape(hidden, kGradVectors);
  return grad_blocks(rows, s) * s.rows_per_block();
}

hipError_t launch_block_norm(const NormArgs& a, bool f16, hipStream_t stream) {
  return f16 ? forward<true>(a, stream) : forward<false>(a, stream);
}
hipError_t launch_block_norm_grad(const NormArgs& a, bool f16, hipStream_t stream) {
  return f16 ? gradient<true>(a, stream) : gradient<false>(a, stream);
}

}  // namespace ep
