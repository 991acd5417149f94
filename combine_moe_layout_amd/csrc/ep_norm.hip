// ep_norm.hip -- the norm after a block with its gate and residual scale, the norm before the
// next block, and their gradients.
//
//   s = (mean(y^2) + eps)^-1/2,  b = y s post        (without a post weight: b = y)
//   x = alpha residual + gate_t b                    -> out, rounded
//   r = (mean(x^2) + eps)^-1/2,  normed = x r pre    (of the unrounded x) -> normed, rounded
//
// Bound by HBM: y and the residual are read once, out and normed written once.  A row stays in
// the registers of its lanes, V vectors of 8 channels each, through both sums.  Loads and stores
// past the caches: 8192 rows of 7168 in 84 us (5.6 TB/s), 109 us through them; no size was slower.
// Two vectors to a lane (8192 x 7168: one vector 95 us, four 84; 2048 x 4096: 15.6, 13.1 with two, 12.1).
//
// Gradient, with D = sum(dx post y), everything recomputed from the forward's inputs:
//   dx = d_out + r (pre dn - x r (r mean(pre dn x)))      d_residual = alpha dx
//   d_gate = s D       d_y = gate s (post dx - y s (s D / hidden))
//   d_post = sum over rows of gate dx y s                 d_pre = sum over rows of dn x r
// s and r are applied one at a time: their cubes leave fp32's range where rows' roots of mean squares
// are past 1e12, and where they and eps are small.
// A workgroup walks rows and keeps its sums of d_post and d_pre; they meet in a second kernel in a
// fixed order, so the result does not depend on timing.  16,384 rows of 4096: 145 us (5.5 TB/s),
// 344 us without the next row's loads in flight, 234 us with them but with the weights loaded for
// each row, behind them.  More than 8192 channels leave no registers for that, and up to 16,384 the
// sums are in LDS (2048 x 16,384: 121 us; 176 in registers, which spilled; 300 by the wide rows'
// kernel, which more channels go to).
#include "ep_norm.h"

namespace ep {

namespace {

constexpr int kMaxLanes = 1024;
constexpr int kMaxWaves = kMaxLanes / 64;
constexpr int kRowsPerBlock = 4;  // of one wave each

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
    yv[i] = a.y != nullptr && v < vecs ? load_nt(y + v) : zero;
    rv[i] = a.residual != nullptr && v < vecs ? load_nt(res + v) : zero;
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
    if (a.out != nullptr && v < vecs) store_nt(static_cast<u32x4*>(a.out) + row * vecs + v, pack8<kF16>(x[i]));
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
    store_nt(static_cast<u32x4*>(a.normed) + row * vecs + v, pack8<kF16>(w));
  }
}

// A thread's sums over rows of a weight's gradient, of its V vectors of channels: in registers, or
// (kLds) in LDS, 16 bytes of a vector's 32 at a time, so that neighbouring lanes' are neighbours.
template <int V, bool kLds>
struct ChannelSums {
  float f[V][8];
  __device__ __forceinline__ void clear(f32x4*, int, int) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) f[i][k] = 0.0f;
  }
  __device__ __forceinline__ void add(int i, const float (&a)[8], const float (&b)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[i][k] = fmaf(a[k], b[k], f[i][k]);
  }
  __device__ __forceinline__ void get(int i, float (&to)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) to[k] = f[i][k];
  }
};
constexpr int kLdsVecs = 2 * kMaxLanes;  // channels / 8 that ChannelSums in LDS hold
template <int V>
struct ChannelSums<V, true> {
  f32x4* at;  // of the thread's first vector
  int step;   // to its next
  __device__ __forceinline__ void clear(f32x4* sums, int lane, int lanes) {
    at = sums + lane;
    step = lanes;
#pragma unroll
    for (int i = 0; i < V; ++i) at[i * step] = at[i * step + kLdsVecs] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  __device__ __forceinline__ void add(int i, const float (&a)[8], const float (&b)[8]) {
    f32x4 lo = at[i * step], hi = at[i * step + kLdsVecs];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = fmaf(a[k], b[k], lo[k]);
      hi[k] = fmaf(a[4 + k], b[4 + k], hi[k]);
    }
    at[i * step] = lo;
    at[i * step + kLdsVecs] = hi;
  }
  __device__ __forceinline__ void get(int i, float (&to)[8]) const {
    const f32x4 lo = at[i * step], hi = at[i * step + kLdsVecs];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      to[k] = lo[k];
      to[4 + k] = hi[k];
    }
  }
};

// One block walks rows blockIdx, blockIdx + gridDim, .. (times its rows), and writes sums number
// blockIdx of `partials` of each weight's gradient.
template <bool kF16, int V, bool kPrefetch>
__global__ __launch_bounds__(kPrefetch ? kMaxLanes / 2 : kMaxLanes) void block_norm_grad_kernel(
    NormArgs a, int32_t lanes, int64_t partials) {
  __shared__ float part[2][3][2 * kMaxWaves];
  const int lane = threadIdx.x % lanes, local = threadIdx.x / lanes;
  const int64_t here = blockDim.x / lanes, step = gridDim.x * here;
  const int32_t vecs = a.hidden / 8;
  const u32x4 *const y = static_cast<const u32x4*>(a.y), *const res = static_cast<const u32x4*>(a.residual);
  const u32x4 *const dout = static_cast<const u32x4*>(a.d_out), *const dn = static_cast<const u32x4*>(a.d_normed);
  const u32x4* const post = static_cast<const u32x4*>(a.post_weight);
  const u32x4* const pre = static_cast<const u32x4*>(a.pre_weight);
  const bool has_pre = dn != nullptr, has_post = post != nullptr;
  const u32x4 zero = {0, 0, 0, 0};
  const float mean = 1.0f / (float)a.hidden;
  // kPrefetch: the next row's vectors are on their way while this row is worked on, and the
  // weights stay in registers (a load of them would wait for the next row's, issued before it).
  u32x4 post_w[V], pre_w[V];
  const auto weights = [&] {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = lane + i * lanes;
      post_w[i] = has_post && v < vecs ? post[v] : zero;
      pre_w[i] = has_pre && v < vecs ? pre[v] : zero;
    }
  };
  if (kPrefetch) weights();
  constexpr bool kLds = V == 2 && !kPrefetch;
  __shared__ f32x4 channel_sums[kLds ? 2 : 1][kLds ? 2 * kLdsVecs : 1];
  ChannelSums<V, kLds> sum_post, sum_pre;
  sum_post.clear(channel_sums[0], lane, lanes);
  sum_pre.clear(channel_sums[kLds], lane, lanes);
  struct Row {
    u32x4 y[V], dn[V], res[V], dout[V];
    float gate;
  };
  const auto load = [&](Row& r, int64_t row) {
    const int64_t at = row * vecs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = lane + i * lanes;
      const bool ok = v < vecs;
      r.y[i] = y != nullptr && ok ? load_nt(y + at + v) : zero;
      r.dn[i] = has_pre && ok ? load_nt(dn + at + v) : zero;
      r.res[i] = has_pre && res != nullptr && ok ? load_nt(res + at + v) : zero;
      r.dout[i] = dout != nullptr && ok ? load_nt(dout + at + v) : zero;
    }
    r.gate = a.gate != nullptr ? a.gate[row] : 1.0f;
  };
  int turn = 0;
  Row now, next;
  int64_t row = blockIdx.x * here + local;
  if (row < a.rows) load(now, row);
  for (; row < a.rows; row += step, turn ^= 1) {
    const int64_t at = row * vecs;
    if (kPrefetch && row + step < a.rows) load(next, row + step);
    if (!kPrefetch) weights();
    u32x4* const yv = now.y;
    u32x4* const nv = now.dn;
    float x[V][8], dx[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack8<kF16>(now.res[i], x[i]);
      unpack8<kF16>(now.dout[i], dx[i]);
    }
    const float gate = now.gate;
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
        float f[8], w[8], d[8];
        unpack8<kF16>(yv[i], f);
        if (has_post) {
          unpack8<kF16>(post_w[i], w);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = f[k] * s * w[k];
        }
        unpack8<kF16>(pre_w[i], w);
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
      const float along = r * (sums[1] * mean);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float w[8], d[8];
        unpack8<kF16>(pre_w[i], w);
        unpack8<kF16>(nv[i], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[i][k] *= r;
          dx[i][k] = fmaf(r, fmaf(-x[i][k], along, d[k] * w[k]), dx[i][k]);
        }
        sum_pre.add(i, d, x[i]);
      }
    }
    if (a.d_residual != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = lane + i * lanes;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = a.residual_scale * dx[i][k];
        if (v < vecs) store_nt(static_cast<u32x4*>(a.d_residual) + at + v, pack8<kF16>(o));
      }
    }
    const bool has_y = y != nullptr;
    float dot[1] = {0.0f};
    if (has_y && (has_post || a.d_gate != nullptr)) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8], w[8];
        unpack8<kF16>(yv[i], f);
        if (has_post) {
          unpack8<kF16>(post_w[i], w);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[i][k] = gate * s * f[k];
          sum_post.add(i, dx[i], x[i]);
#pragma unroll
          for (int k = 0; k < 8; ++k) dx[i][k] *= w[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) dot[0] = fmaf(dx[i][k], f[k], dot[0]);
      }
      row_sums(dot, lanes, part[turn][2]);
      if (a.d_gate != nullptr && lane == 0) a.d_gate[row] = s * dot[0];
    }
    if (has_y && a.d_y != nullptr) {
      const float along = s * (dot[0] * mean);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = lane + i * lanes;
        float f[8];
        unpack8<kF16>(yv[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // (without its norm y has no part in it: it may be infinite)
          f[k] = gate * s * (has_post ? fmaf(-f[k] * s, along, dx[i][k]) : dx[i][k]);
        if (v < vecs) store_nt(static_cast<u32x4*>(a.d_y) + at + v, pack8<kF16>(f));
      }
    }
    if (kPrefetch) now = next;
    else if (row + step < a.rows) load(now, row + step);
  }
  // The block's rows meet in LDS, in order, and its sums go to the workspace.
  constexpr bool kSmall = kPrefetch;
  __shared__ float sums[kSmall ? kRowsPerBlock : 1][kSmall ? 64 * V * 8 : 1];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.d_post_weight : a.d_pre_weight) == nullptr) continue;
    const ChannelSums<V, kLds>& mine = which == 0 ? sum_post : sum_pre;
    float* const to = a.partial + (which * partials + blockIdx.x) * a.hidden;
    if constexpr (kSmall) {
      if (lanes == 64) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float f[8];
          mine.get(i, f);
#pragma unroll
          for (int k = 0; k < 8; ++k) sums[local][k * (64 * V) + i * 64 + lane] = f[k];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.hidden; c += blockDim.x) {
          const int at = c % 8 * (64 * V) + c / 8;
          float f = sums[0][at];
          for (int r = 1; r < kRowsPerBlock; ++r) f += sums[r][at];
          to[c] = f;
        }
        continue;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = lane + i * lanes;
      float f[8];
      mine.get(i, f);
      if (v < vecs) {
        reinterpret_cast<f32x4*>(to)[2 * v] = f32x4{f[0], f[1], f[2], f[3]};
        reinterpret_cast<f32x4*>(to)[2 * v + 1] = f32x4{f[4], f[5], f[6], f[7]};
      }
    }
  }
}

// More than kLdsVecs * 8 channels: a row's vectors do not fit its lanes' registers (kept there, they
// spilled: 2048 rows of 32,768 in 811 us, of 65,536 in 2777 us).  A workgroup goes over its row four
// times, for y's sum of squares, x's sums, D and the outputs, and computes x and dx anew each time; the
// row comes from the caches after the first (589 us, 1230 us; two workgroups to a CU no better).  Its sums of the weights' gradients are
// kept in the workspace.
template <bool kF16>
__global__ __launch_bounds__(kMaxLanes) void block_norm_grad_wide_kernel(NormArgs a, int64_t partials) {
  __shared__ float part[2][3][2 * kMaxWaves];
  const int32_t vecs = a.hidden / 8, lanes = blockDim.x;
  const u32x4* const post = static_cast<const u32x4*>(a.post_weight);
  const u32x4* const pre = static_cast<const u32x4*>(a.pre_weight);
  const bool has_y = a.y != nullptr, has_pre = a.d_normed != nullptr, has_post = post != nullptr;
  const bool weights = a.d_post_weight != nullptr || a.d_pre_weight != nullptr;
  const float mean = 1.0f / (float)a.hidden;
  float* const own_post = a.d_post_weight != nullptr ? a.partial + (int64_t)blockIdx.x * a.hidden : nullptr;
  float* const own_pre = a.d_pre_weight != nullptr ? a.partial + (partials + blockIdx.x) * a.hidden : nullptr;
  const u32x4 zero = {0, 0, 0, 0};
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const bool first = row == blockIdx.x;
    const int64_t at = row * vecs;
    const auto vector = [&](const void* p, int v, float (&f)[8]) {
      unpack8<kF16>(p != nullptr ? static_cast<const u32x4*>(p)[at + v] : zero, f);
    };
    const float gate = a.gate != nullptr ? a.gate[row] : 1.0f;
    float s = 1.0f, r = 0.0f, along = 0.0f;
    if (has_post) {
      float squares[1] = {0.0f};
#pragma unroll 4
      for (int v = threadIdx.x; v < vecs; v += lanes) {
        float f[8];
        vector(a.y, v, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) squares[0] = fmaf(f[k], f[k], squares[0]);
      }
      row_sums(squares, lanes, part[turn][0]);
      s = inverse_rms(squares[0], a.hidden, a.eps);
    }
    // x, and pre dn
    const auto hidden = [&](int v, float (&x)[8], float (&d)[8]) {
      float f[8], w[8];
      vector(a.y, v, f);
      vector(a.residual, v, x);
      vector(a.d_normed, v, d);
      if (has_post) {
        unpack8<kF16>(post[v], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * s * w[k];
      }
      unpack8<kF16>(pre[v], w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[k] = fmaf(gate, f[k], a.residual_scale * x[k]);
        d[k] *= w[k];
      }
    };
    if (has_pre) {
      float sums[2] = {0.0f, 0.0f};  // x^2, pre dn x
#pragma unroll 2
      for (int v = threadIdx.x; v < vecs; v += lanes) {
        float x[8], d[8];
        hidden(v, x, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sums[0] = fmaf(x[k], x[k], sums[0]);
          sums[1] = fmaf(d[k], x[k], sums[1]);
        }
      }
      row_sums(sums, lanes, part[turn][1]);
      r = inverse_rms(sums[0], a.hidden, a.eps);
      along = r * (sums[1] * mean);
    }
    const auto gradient = [&](int v, float (&x)[8], float (&dx)[8]) {
      vector(a.d_out, v, dx);
      if (!has_pre) return;
      float d[8];
      hidden(v, x, d);
#pragma unroll
      for (int k = 0; k < 8; ++k) dx[k] = fmaf(r, fmaf(-x[k] * r, along, d[k]), dx[k]);
    };
    const auto add = [&](float* own, int v, const float (&p)[8], const float (&q)[8]) {
      f32x4* const to = reinterpret_cast<f32x4*>(own) + 2 * v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        if (!first) sum = to[h];
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = fmaf(p[4 * h + k], q[4 * h + k], sum[k]);
        to[h] = sum;
      }
    };
    float dot[1] = {0.0f};
    if (weights || (has_y && (has_post || a.d_gate != nullptr))) {
#pragma unroll 2
      for (int v = threadIdx.x; v < vecs; v += lanes) {
        float x[8], dx[8], f[8], w[8];
        gradient(v, x, dx);
        if (own_pre != nullptr) {
          vector(a.d_normed, v, f);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] *= r;
          add(own_pre, v, f, x);
        }
        vector(a.y, v, f);
        if (has_post) {
          if (own_post != nullptr) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = gate * s * f[k];
            add(own_post, v, dx, x);
          }
          unpack8<kF16>(post[v], w);
#pragma unroll
          for (int k = 0; k < 8; ++k) dx[k] *= w[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) dot[0] = fmaf(dx[k], f[k], dot[0]);
      }
      row_sums(dot, lanes, part[turn][2]);
      if (a.d_gate != nullptr && threadIdx.x == 0) a.d_gate[row] = s * dot[0];
    }
    if (a.d_y == nullptr && a.d_residual == nullptr) continue;
    const float along_y = s * (dot[0] * mean);
#pragma unroll 2
    for (int v = threadIdx.x; v < vecs; v += lanes) {
      float x[8], dx[8], f[8], w[8];
      gradient(v, x, dx);
      vector(a.y, v, f);
      if (a.d_residual != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = a.residual_scale * dx[k];
        store_nt(static_cast<u32x4*>(a.d_residual) + at + v, pack8<kF16>(x));
      }
      if (a.d_y == nullptr) continue;
      if (has_post) {
        unpack8<kF16>(post[v], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) dx[k] *= w[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = gate * s * (has_post ? fmaf(-f[k] * s, along_y, dx[k]) : dx[k]);
      store_nt(static_cast<u32x4*>(a.d_y) + at + v, pack8<kF16>(f));
    }
  }
}

// The weights' gradients from the blocks' sums: a workgroup takes 64 channels of one of them, four
// to a thread; its 64 groups of 16 threads share out the blocks and meet in LDS.
template <bool kF16>
__global__ __launch_bounds__(kMaxLanes) void norm_weights_kernel(const float* __restrict__ partial, int64_t partials,
                                                                 int32_t hidden, void* d_post, void* d_pre,
                                                                 bool f32, bool accumulate) {
  __shared__ f32x4 sums[64][16];
  void* const to = blockIdx.y == 0 ? d_post : d_pre;
  if (to == nullptr) return;
  const int quad = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int32_t col = blockIdx.x * 64 + quad * 4;  // (hidden is a multiple of 8)
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (col < hidden) {
    const float* const from = partial + blockIdx.y * partials * hidden + col;
#pragma unroll 8
    for (int64_t p = group; p < partials; p += 64) s += *reinterpret_cast<const f32x4*>(from + p * hidden);
  }
  sums[group][quad] = s;
  __syncthreads();
  const int32_t mine = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || mine >= hidden) return;
  float f = 0.0f;
  for (int g = 0; g < 64; ++g) f += sums[g][threadIdx.x / 4][threadIdx.x % 4];
  if (f32) {
    float* const p = static_cast<float*>(to) + mine;
    *p = accumulate ? *p + f : f;
  } else {
    static_cast<uint16_t*>(to)[mine] = elem_rne<kF16>(accumulate ? elem_at<kF16>(to, mine) + f : f);
  }
}

// Threads of a row and vectors of each.
struct RowShape {
  int lanes, vectors;
  int rows_per_block() const { return lanes == 64 ? kRowsPerBlock : 1; }
};
RowShape row_shape(int32_t hidden) {
  const int vecs = hidden / 8;
  int vectors = vecs <= 64 ? 1 : 2;
  while ((vecs + vectors - 1) / vectors > kMaxLanes) vectors *= 2;
  return {((vecs + vectors - 1) / vectors + 63) / 64 * 64, vectors};
}

template <bool kF16>
hipError_t forward(const NormArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.hidden);
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

// As many blocks as run at one time: two waves to a SIMD, by registers (one block where it has
// more than four waves).
int64_t grad_blocks(int64_t rows, const RowShape& s) {
  const int64_t most = (rows + s.rows_per_block() - 1) / s.rows_per_block();
  const int64_t run = s.lanes * s.rows_per_block() <= 256 ? 2 * kChipCUs : kChipCUs;
  return most < run ? most : run;
}

template <bool kF16>
hipError_t gradient(const NormArgs& a, hipStream_t stream) {
  const RowShape s = row_shape(a.hidden);
  const int64_t blocks = grad_blocks(a.rows, s);
  const int threads = s.lanes * s.rows_per_block();
  if (blocks > 0) {
    const auto run = [&](auto kernel) { kernel<<<(uint32_t)blocks, threads, 0, stream>>>(a, s.lanes, blocks); };
    if (s.vectors == 1) run(block_norm_grad_kernel<kF16, 1, true>);
    else if (s.vectors == 2 && s.lanes <= kMaxLanes / 2) run(block_norm_grad_kernel<kF16, 2, true>);
    else if (s.vectors == 2) run(block_norm_grad_kernel<kF16, 2, false>);
    else block_norm_grad_wide_kernel<kF16><<<(uint32_t)blocks, threads, 0, stream>>>(a, blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.d_post_weight != nullptr || a.d_pre_weight != nullptr) {
    norm_weights_kernel<kF16><<<dim3((a.hidden + 63) / 64, 2), kMaxLanes, 0, stream>>>(
        a.partial, blocks, a.hidden, a.d_post_weight, a.d_pre_weight, a.grad_f32, a.accumulate);
  }
  return hipGetLastError();
}

}  // namespace

int64_t norm_partials(int64_t rows, int32_t hidden) {
  return grad_blocks(rows, row_shape(hidden));
}

hipError_t launch_block_norm(const NormArgs& a, bool f16, hipStream_t stream) {
  return f16 ? forward<true>(a, stream) : forward<false>(a, stream);
}
hipError_t launch_block_norm_grad(const NormArgs& a, bool f16, hipStream_t stream) {
  return f16 ? gradient<true>(a, stream) : gradient<false>(a, stream);
}

}  // namespace ep
