// ep_gemm_few.hip -- bf16 and fp16 products of few rows (a decode step's dense
// layer, experts with a handful of rows each): reading the matrix once is all
// that counts.
//
//   out[r, n] = act(sum_k a[r, k] b[e, n, k] + bias[e, n]) + residual[r, n]
//
// A workgroup takes 16 rows of the matrix (for swiglu 8 gates and the 8 ups of
// the same columns) against 16 TM rows of a, and its 8 waves share out the
// reduction in chunks of 128 (64 for 64 rows), so that a product of 4096 columns has a workgroup
// for every CU, each with 64 KB on its way: a wave's lanes hold two chunks of
// both operands in registers while they work on a third, and there is no barrier
// before the end.  The waves' sums meet in LDS and are added in wave order, so
// the result does not depend on timing.
#include "ep_gemm.h"

namespace ep {

namespace {

constexpr int kWaves = 8;

template <bool kF16>
struct FewFrag {
  typedef bf16x8 type;
  static __device__ __forceinline__ f32x4 mfma(type a, type b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct FewFrag<true> {
  typedef f16x8 type;
  static __device__ __forceinline__ f32x4 mfma(type a, type b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

template <bool kF16, bool kGlu, int TM>
__global__ __launch_bounds__(kWaves * 64, 2) void gemm_few_kernel(GemmArgs g) {
  typedef typename FewFrag<kF16>::type F;
  constexpr int kChunk = TM == 4 ? 64 : 128;  // reduction elements of one wave at a time
  constexpr int kSteps = kChunk / 32;         // matrix instructions deep
  constexpr int kOut = kGlu ? 8 : 16;         // result columns of a workgroup
  constexpr int kPitch = 17;                // LDS row of 16 sums
  __shared__ float sums[kWaves][16 * TM * kPitch];
  Tile t;
  if (!find_tile<1>(g.groups, 16 * TM, (g.out_cols + kOut - 1) / kOut, blockIdx.x, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  // This lane's row of the matrix and rows of a; 8 elements at 8 q of every 32.
  const int first = t.col * kOut;
  const int n = kGlu ? min(first + (m & 7), g.out_cols - 1) + (m >= 8 ? g.out_cols : 0)
                     : min(first + m, g.out_cols - 1);
  const uint16_t* const b = static_cast<const uint16_t*>(g.b) + t.e * g.b_stride + (int64_t)n * g.ldb + q * 8;
  const uint16_t* a[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i)
    a[i] = static_cast<const uint16_t*>(g.a) + (t.row0 + min(i * 16 + m, t.rows - 1)) * g.lda + q * 8;

  const int chunks = (g.reduce + kChunk - 1) / kChunk, whole = g.reduce / kChunk;
  f32x4 acc[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Chunk {
    F b[kSteps], a[TM][kSteps];
  };
  Chunk ring[3];
  const auto load = [&](Chunk& c, int i) {
    const int k = i * kChunk;
    if (i < whole) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) c.b[s] = *reinterpret_cast<const F*>(b + k + s * 32);
#pragma unroll
      for (int r = 0; r < TM; ++r)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) c.a[r][s] = *reinterpret_cast<const F*>(a[r] + k + s * 32);
    } else {  // past the reduction: zeros
      const F zero = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bool in = k + s * 32 + q * 8 < g.reduce;
        c.b[s] = zero;
        if (in) c.b[s] = *reinterpret_cast<const F*>(b + k + s * 32);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          c.a[r][s] = zero;
          if (in) c.a[r][s] = *reinterpret_cast<const F*>(a[r] + k + s * 32);
        }
      }
    }
  };
  const auto multiply = [&](const Chunk& c) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int r = 0; r < TM; ++r) acc[r] = FewFrag<kF16>::mfma(c.b[s], c.a[r][s], acc[r]);
  };
  // Chunks wave, wave + 8, ..: two loaded ahead.
  if (wave < chunks) load(ring[0], wave);
  if (wave + kWaves < chunks) load(ring[1], wave + kWaves);
  for (int i = wave; i < chunks; i += 3 * kWaves) {
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const int c = i + s * kWaves;
      if (c >= chunks) break;
      if (c + 2 * kWaves < chunks) load(ring[(s + 2) % 3], c + 2 * kWaves);
      multiply(ring[s]);
    }
  }
  // Lane 16 q + m holds columns 4 q .. 4 q + 3 of row m of each block.
#pragma unroll
  for (int r = 0; r < TM; ++r)
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[wave][(r * 16 + m) * kPitch + q * 4 + k] = acc[r][k];
  __syncthreads();
  const int32_t out_n = g.out_cols, width = kGlu ? 2 * out_n : out_n;
  uint16_t* const out = static_cast<uint16_t*>(g.out);
  uint16_t* const pre = static_cast<uint16_t*>(g.preact);
  for (int i = threadIdx.x; i < 16 * TM * kOut; i += kWaves * 64) {
    const int r = i / kOut, c = i % kOut, col = first + c;
    if (r >= t.rows || col >= out_n) continue;
    const int64_t row = t.row0 + r;
    float z = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      z += sums[w][r * kPitch + c];
      if constexpr (kGlu) up += sums[w][r * kPitch + 8 + c];
    }
    if (g.bias != nullptr) {
      z += elem_at<kF16>(g.bias, (int64_t)t.e * width + col);
      if constexpr (kGlu) up += elem_at<kF16>(g.bias, (int64_t)t.e * width + out_n + col);
    }
    if (pre != nullptr) {
      pre[row * width + col] = elem_rne<kF16>(z);
      if constexpr (kGlu) pre[row * width + out_n + col] = elem_rne<kF16>(up);
    }
    float v = kGlu ? silu(z) * up : act_value(g.act, z);
    if (g.residual != nullptr) v += elem_at<kF16>(g.residual, row * out_n + col);
    out[row * out_n + col] = elem_rne<kF16>(v);
  }
}

template <bool kF16, bool kGlu, int TM>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  constexpr int kOut = kGlu ? 8 : 16;
  const int64_t ct = (g.out_cols + kOut - 1) / kOut;
  const int64_t blocks = (max_row_tiles(g.groups, 16 * TM) * ct + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, kWaves * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_few_kernel<kF16, kGlu, TM><<<(uint32_t)blocks, kWaves * 64, 0, stream>>>(g);
  return hipGetLastError();
}
template <bool kF16, bool kGlu>
hipError_t launch_rows(const GemmArgs& g, int64_t rows, hipStream_t stream) {
  if (rows <= 16) return launch<kF16, kGlu, 1>(g, stream);
  if (rows <= 32) return launch<kF16, kGlu, 2>(g, stream);
  return launch<kF16, kGlu, 4>(g, stream);
}

}  // namespace

hipError_t launch_gemm_few(const GemmArgs& g, int64_t rows, bool f16, hipStream_t stream) {
  if (g.act == EP_ACT_SWIGLU)
    return f16 ? launch_rows<true, true>(g, rows, stream) : launch_rows<false, true>(g, rows, stream);
  return f16 ? launch_rows<true, false>(g, rows, stream) : launch_rows<false, false>(g, rows, stream);
}

}  // namespace ep
