// ep_grad.hip -- the gradients that are not matrix products: the weighted
// combine's, and an activation's.
//
// Combine: out[t] = sum_j w[t,j] y[slot[t,j]], so
//   dy[slot[t,j]] = w[t,j] dout[t]          (rounded once)
//   dw[t,j]       = sum_h dout[t,h] y[slot[t,j],h]   (fp32; 0 for a pair without a row)
// Bound by HBM: dout is read once, every used row of y read once and of dy
// written once.  A workgroup holds a token's dout row in registers, 16 bytes
// to a lane, and takes up to four of its pairs, all of whose y rows are loaded
// before the first is used (dout comes from L2 for the others); the dot products
// meet in LDS in a fixed order, so the result does not depend on timing.
#include <type_traits>

#include "ep_gemm.h"

namespace ep {

namespace {

constexpr int kMaxLanes = 1024;
constexpr int kMostPairs = 4;

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
__device__ __forceinline__ u32x4 pack8_rne(const float* f) {
  return u32x4{elem_rne2<kF16>(f[0], f[1]), elem_rne2<kF16>(f[2], f[3]), elem_rne2<kF16>(f[4], f[5]),
               elem_rne2<kF16>(f[6], f[7])};
}

// Sums of N values (a power of two) over the 64 lanes of a wave.  In the first
// log2(N) steps the two lanes of a pair hand each other half of their values, so
// N - 1 exchanges leave one value to a lane, and the other steps take one each (7
// exchanges for 4 values instead of 24).  Returns the sum of value `index`.
template <int N, int kMask = 1>
__device__ __forceinline__ float wave_sums(const float (&v)[N], int& index) {
  if constexpr (N == 1) {
    index = 0;
    float s = v[0];
#pragma unroll
    for (int mask = kMask; mask < 64; mask *= 2) s += __shfl_xor(s, mask, 64);
    return s;
  } else {
    const bool high = threadIdx.x & kMask;
    float half[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float keep = high ? v[N / 2 + i] : v[i], give = high ? v[i] : v[N / 2 + i];
      half[i] = keep + __shfl_xor(give, kMask, 64);
    }
    const float s = wave_sums<N / 2, kMask * 2>(half, index);
    index += high ? N / 2 : 0;
    return s;
  }
}

// lanes: threads of one token (a multiple of 64); the block holds blockDim / lanes
// tokens.  kPairs: pairs of one workgroup, splits: workgroups per token.
// kStream: y does not stay in the last-level cache.
template <bool kF16, bool kDw, bool kStream, int kPairs>
__global__ __launch_bounds__(kMaxLanes) void combine_grad_kernel(
    const u32x4* __restrict__ dout, const u32x4* __restrict__ y, const float* __restrict__ w,
    const int32_t* __restrict__ slot, int64_t tokens, int32_t k, int32_t vecs, int32_t lanes,
    int32_t splits, u32x4* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float part[kMaxLanes / 64][kPairs];
  const int local = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int64_t block = blockIdx.x;
  const int64_t t = block / splits * (blockDim.x / lanes) + local;
  const int j0 = (int)(block % splits) * kPairs;
  const int n = t < tokens ? min(kPairs, k - j0) : 0;
  float dot[kPairs] = {};
  if (n > 0) {
    // All slots and weights at once: a pair past the last reads the last one's.
    int64_t row[kPairs];
    float weight[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int64_t p = t * k + j0 + min(j, n - 1);
      row[j] = slot[p];
      weight[j] = w[p];
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
      if (j >= n) row[j] = -1;
    for (int v = lane; v < vecs; v += lanes) {
      const u32x4 mine = dout[t * vecs + v];
      u32x4 rows[kPairs];
      if constexpr (kDw) {  // a pair without a row reads row 0, and its sum is dropped
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const u32x4* const from = y + max(row[j], (int64_t)0) * vecs + v;
          if constexpr (kStream) rows[j] = load_nt(from);
          else rows[j] = *from;
        }
      }
      float d[8];
      unpack8<kF16>(mine, d);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        if constexpr (kDw) {
          float f[8], sum = dot[j];
          unpack8<kF16>(rows[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(d[i], f[i], sum);
          dot[j] = row[j] >= 0 ? sum : 0.f;
        }
        if (row[j] >= 0) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = weight[j] * d[i];
          store_nt(dy + row[j] * vecs + v, pack8_rne<kF16>(o));
        }
      }
    }
  }
  if constexpr (kDw) {
    const int wave = threadIdx.x >> 6, waves = lanes >> 6;
    constexpr int kSums = kPairs == 3 ? 4 : kPairs;
    float sums[kSums] = {};
#pragma unroll
    for (int j = 0; j < kPairs; ++j) sums[j] = dot[j];
    int index;
    const float total = wave_sums<kSums>(sums, index);
    if ((threadIdx.x & 63) < kSums && index < kPairs) part[wave][index] = total;
    __syncthreads();
    if (lane < n) {
      float s = 0.f;
      for (int i = 0; i < waves; ++i) s += part[local * waves + i][lane];
      dw[t * k + j0 + lane] = s;
    }
  }
}

// dz = dy act'(z), 8 columns to a lane; swiglu: z and dz rows are 2n wide.
// (dz may be dy or z: no __restrict__.)
template <bool kF16>
__global__ __launch_bounds__(256) void act_grad_kernel(const u32x4* dy, const u32x4* z, int64_t vecs,
                                                       int32_t row_vecs, int32_t act, u32x4* dz) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vecs; i += (int64_t)gridDim.x * 256) {
    float d[8], a[8];
    unpack8<kF16>(dy[i], d);
    if (act != EP_ACT_SWIGLU) {
      unpack8<kF16>(z[i], a);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = act_backward<true>(act, d[k], a[k]);
      dz[i] = pack8_rne<kF16>(d);
    } else {
      const int64_t at = i / row_vecs * row_vecs * 2 + i % row_vecs;
      float up[8], du[8];
      unpack8<kF16>(z[at], a);
      unpack8<kF16>(z[at + row_vecs], up);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        du[k] = d[k] * a[k] * sigmoid<true>(a[k]);
        d[k] = silu_backward_exact(d[k] * up[k], a[k]);
      }
      dz[at] = pack8_rne<kF16>(d);
      dz[at + row_vecs] = pack8_rne<kF16>(du);
    }
  }
}

template <bool kF16>
hipError_t combine_grad(const void* dout, const void* y, const float* w, const ep_layout_t& L,
                        int32_t hidden, void* dy, float* dw, hipStream_t stream) {
  const int32_t vecs = hidden / 8;
  int32_t lanes = (vecs + 63) / 64 * 64;
  if (lanes > kMaxLanes) lanes = kMaxLanes;
  const int32_t tokens_per_block = lanes >= 256 ? 1 : 256 / lanes;
  const int64_t token_blocks = (L.num_tokens + tokens_per_block - 1) / tokens_per_block;
  // At most four pairs to a workgroup, shared out evenly; one for the smallest
  // batches.  Measured at hidden 7168, top-8: 128 tokens 13.1 us with one pair,
  // 10.6 with two, 9.5 with four; 512 tokens 29 us with up to four, 36 with eight;
  // 8192 tokens 384 us with four, 389 with two, 387 with eight; 8 tokens 4.4 us
  // with one, 5.3 with four.
  int32_t pairs = 1;
  if (token_blocks >= 64) {
    const int32_t parts = (L.num_topk + kMostPairs - 1) / kMostPairs;
    pairs = (L.num_topk + parts - 1) / parts;
  }
  const int32_t splits = (L.num_topk + pairs - 1) / pairs;
  const int64_t blocks = token_blocks * splits;
  if (!grid_fits(blocks, lanes * tokens_per_block)) return hipErrorInvalidValue;
  const auto args = [&](auto kernel) {
    kernel<<<(uint32_t)blocks, lanes * tokens_per_block, 0, stream>>>(
        static_cast<const u32x4*>(dout), static_cast<const u32x4*>(y), w, L.slot_idx, L.num_tokens,
        L.num_topk, vecs, lanes, splits, static_cast<u32x4*>(dy), dw);
  };
  const auto sized = [&](auto with_dw, auto streams) {
    constexpr bool kDw = decltype(with_dw)::value, kStream = decltype(streams)::value;
    if (pairs == 4) args(combine_grad_kernel<kF16, kDw, kStream, 4>);
    else if (pairs == 3) args(combine_grad_kernel<kF16, kDw, kStream, 3>);
    else if (pairs == 2) args(combine_grad_kernel<kF16, kDw, kStream, 2>);
    else args(combine_grad_kernel<kF16, kDw, kStream, 1>);
  };
  // y is loaded past the caches where y and dy together outgrow the last-level
  // cache's 256 MiB.  Past against through them, hidden 7168, top-8: 128 tokens 7.9
  // against 6.1 us, 1024 (112 MiB of y) 54 and 50, 1536 (168 MiB) 78 and 79, 4096
  // 194 and 210, 8192 387 and 408.
  const bool stream_y = L.num_tokens * (int64_t)L.num_topk * hidden * 2 > (int64_t)128 << 20;
  if (dw == nullptr) sized(std::false_type(), std::false_type());  // y is not read
  else if (stream_y) sized(std::true_type(), std::true_type());
  else sized(std::true_type(), std::false_type());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_grad(const void* dout, const void* y, const float* w, const ep_layout_t& L,
                               int32_t hidden, bool f16, void* dy, float* dw, hipStream_t stream) {
  return f16 ? combine_grad<true>(dout, y, w, L, hidden, dy, dw, stream)
             : combine_grad<false>(dout, y, w, L, hidden, dy, dw, stream);
}

hipError_t launch_act_grad(const void* dy, const void* z, int64_t rows, int32_t n, bool f16,
                           int32_t act, void* dz, hipStream_t stream) {
  const int64_t vecs = rows * (n / 8);
  const int64_t need = (vecs + 255) / 256;
  const uint32_t blocks = (uint32_t)(need < 16 * kChipCUs ? need : 16 * kChipCUs);
  const u32x4 *d = static_cast<const u32x4*>(dy), *a = static_cast<const u32x4*>(z);
  u32x4* o = static_cast<u32x4*>(dz);
  if (f16) act_grad_kernel<true><<<blocks, 256, 0, stream>>>(d, a, vecs, n / 8, act, o);
  else act_grad_kernel<false><<<blocks, 256, 0, stream>>>(d, a, vecs, n / 8, act, o);
  return hipGetLastError();
}

}  // namespace ep
