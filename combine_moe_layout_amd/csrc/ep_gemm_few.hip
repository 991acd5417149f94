// ep_gemm_few.hip -- bf16 and fp16 products with few tiles (a decode step's dense
// layer, a small batch, a small matrix' gradient): what counts is to have the
// whole GPU read the operands.
//
//   forward        out[r, n] = act(sum_k a[r, k] b[e, n, k] + bias[e, n]) + residual[r, n]
//   rows' gradient out[r, k] = (sum_n a[r, n] b[e, n, k]) act'(preact[r, k])
//   weights'       out[e, n, k] (+)= sum_{r in e} a[r, n] b[r, k]
//
// A workgroup takes 16 TN columns of the result (forward: rows of the matrix; for
// swiglu half of them gates and half the ups of the same columns) and 16 TM rows,
// and its waves share out the reduction in chunks of 64.  TN = 1: a product of
// 4096 columns has a workgroup for every CU; TM = TN = 4 for more rows, and for
// the gradients.  Each wave has a ring of chunks of both operands in LDS to
// itself, so there is no barrier before the end, and a workgroup has 8 chunks or
// more on their way, where tiles whose waves share every chunk have two.  (LDS is
// for the address unit: a load costs it 2.6 cycles for each 128-byte line that it
// touches.  In the order of the matrix instruction a load touches 16 lines;
// through LDS it takes 8 whole ones.)  The waves' sums meet in LDS and are added
// in wave order, so the result does not depend on timing.
//
// Measured, reduction 7168 and 4096 columns: 1 row 11.8 us (58.7 MB, 5.0 TB/s), 16
// rows 14, 32 rows 17, 64 rows 22; 256 rows 40 us (TN = 4).  Before the rings, with
// fragments loaded straight into registers: 14.3, 18.5, 23 and 35 us.  What bounds
// the long gradients is latency: 9689 rows, 184 x 840 are 42 workgroups, and a
// chunk takes a wave 1.6 us with the next one on its way.
#include <type_traits>

#include "ep_gemm.h"

namespace ep {

namespace {

constexpr int kChunk = 64;  // reduction elements of one wave at a time: 128 bytes of a row
// Waves of a workgroup and chunks in a wave's ring: what LDS holds.
constexpr int waves_of(int TM) { return TM < 4 ? 8 : 4; }
constexpr int slots_of(int TM, int TN) { return TN > 1 ? 2 : TM == 2 ? 3 : 4; }

// One weight's or bias' gradient.
template <bool kF16>
__device__ __forceinline__ void store_gradient(const GemmArgs& g, void* to, int64_t at, float v) {
  if (g.grad_f32) {
    float* const p = static_cast<float*>(to) + at;
    *p = g.accumulate ? *p + v : v;
  } else {
    uint16_t* const p = static_cast<uint16_t*>(to) + at;
    *p = elem_rne<kF16>(g.accumulate ? elem_at<kF16>(to, at) + v : v);
  }
}

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

// Where the reduction is the slow dimension of an operand, a chunk of it is 64
// rows of 64 elements: pair p of the 16-byte chunks of row k lies at p ^ f(k), so
// that the eight rows which one half wave of a transposing read touches lie in
// different banks.
__device__ __forceinline__ int slow_swizzle(int k) { return ((k >> 1) & 1) | ((k >> 3) & 1) * 2; }

template <int kMode, bool kF16, bool kGlu, int TM, int TN>
__global__ __launch_bounds__(waves_of(TM) * 64, waves_of(TM) / 4) void gemm_few_kernel(GemmArgs g) {
  typedef typename FewFrag<kF16>::type F;
  constexpr bool kASlow = kMode == kWeightsGrad, kBSlow = kMode != kForward;
  static_assert((!kASlow || TM == 4) && (!kBSlow || TN == 4), "slow operands come in 64 columns");
  constexpr bool kHalves = kGlu && kMode == kForward;  // gates and ups
  constexpr int kWaves = waves_of(TM), kSlots = slots_of(TM, TN);
  constexpr int kOut = kHalves ? 8 * TN : 16 * TN;  // result columns of a workgroup
  constexpr int kPitch = 16 * TN + 1;               // floats of a row's sums in LDS (one more: the bias')
  constexpr int kLoads = 2 * TN + 2 * TM;           // of a chunk: 8 rows each
  constexpr int kSlotBytes = kLoads * 1024, kRingBytes = kSlots * kSlotBytes;
  __shared__ __align__(1024) char lds[kWaves * kRingBytes];
  static_assert(16 * TM * kPitch * 4 <= kRingBytes, "the sums take the ring's place");
  Tile t;
  int64_t group_row = 0;
  int32_t reduce = g.reduce;
  if constexpr (kMode == kWeightsGrad) {
    const int32_t rt = (g.out_rows + 16 * TM - 1) / (16 * TM), ct = (g.out_cols + kOut - 1) / kOut;
    t.e = blockIdx.x / (rt * ct);
    const int32_t rem = blockIdx.x % (rt * ct);
    t.row0 = (int64_t)(rem / ct) * (16 * TM);
    t.col = rem % ct;
    t.rows = (int32_t)min((int64_t)(16 * TM), g.out_rows - t.row0);
    group_row = group_first(g.groups, t.e);
    reduce = __builtin_amdgcn_readfirstlane(group_count(g.groups, t.e));
  } else {
    if (!find_tile<1>(g.groups, 16 * TM, (g.out_cols + kOut - 1) / kOut, blockIdx.x, t)) return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  const int first = t.col * kOut;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  const uint32_t ring = lds0 + wave * kRingBytes;

  // Load j brings rows 8 j .. 8 j + 7 of a chunk (the first 16 TN are the
  // matrix's): lane l row l / 8; 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7),
  // so that the fragment reads below touch every bank once in each of their phases.
  const char* const b0 = static_cast<const char*>(g.b) + t.e * g.b_stride * 2 +
                         (kBSlow ? group_row * g.ldb + first : (int64_t)first * g.ldb) * 2;
  const char* const ups = b0 + (int64_t)g.out_cols * g.ldb * 2;
  const char* const a0 = static_cast<const char*>(g.a) +
                         (kASlow ? group_row * g.lda + t.row0 : t.row0 * g.lda) * 2;
  const int64_t a_step = kASlow ? (int64_t)kChunk * g.lda * 2 : kChunk * 2;
  const int64_t b_step = kBSlow ? (int64_t)kChunk * g.ldb * 2 : kChunk * 2;
  uint32_t offset[kLoads];
  int place[kLoads];  // of the load's 8 elements in the chunk's reduction
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const bool of_b = j < 2 * TN;
    const int row = j * 8 + (lane >> 3), r = of_b ? row : row - 16 * TN;
    const int32_t ld = of_b ? g.ldb : g.lda;
    const int last = of_b ? g.out_cols - 1 - first : t.rows - 1;  // row, or column
    if (of_b ? kBSlow : kASlow) {
      const int chunk = (lane & 7) ^ (slow_swizzle(r) << 1);
      place[j] = r;
      offset[j] = (uint32_t)r * (uint32_t)ld * 2u + min(chunk * 8, last - 7) * 2;
    } else {
      const int chunk = (lane & 7) ^ ((row >> 1) & 7);
      place[j] = chunk * 8;
      offset[j] = (uint32_t)min(of_b ? r % kOut : r, last) * (uint32_t)ld * 2u + chunk * 16;
    }
  }
  const int chunks = tiles_of(reduce, kChunk), whole = reduce / kChunk;
  const auto load = [&](int c, int slot) {
    const uint32_t to = ring + slot * kSlotBytes;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const char* const from = j >= 2 * TN ? a0 + c * a_step : (kHalves && j >= TN ? ups : b0) + c * b_step;
      if (c < whole)
        load16_to_lds(from, offset[j], to + j * 1024);
      else  // past the reduction: zeros
        load16_to_lds(c * kChunk + place[j] < reduce ? from + offset[j] : reinterpret_cast<const char*>(g_zero16),
                      to + j * 1024);
    }
  };
  f32x4 acc[TM][TN], bias_acc[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    bias_acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < TN; ++n) acc[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // Biases' gradient: products with ones, in the workgroups of the first columns.
  const bool bias_tile = kMode == kWeightsGrad && g.bias_grad != nullptr && t.col == 0;
  F ones;
#pragma unroll
  for (int k = 0; k < 8; ++k) ones[k] = 1;
  // Chunks wave, wave + kWaves, ..: every slot of the ring is filled, and a slot is
  // filled again as soon as its chunk has been read.
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (wave + i * kWaves < chunks) load(wave + i * kWaves, i);
  const uint32_t in_row = m * 128 + ((q ^ ((m >> 1) & 7)) << 4);
  const int k0 = q * 8 + (m >> 2);
  const uint32_t in_slow = k0 * 128 + (slow_swizzle(k0) << 5) + ((m & 2) << 3) + ((m & 1) << 3);
  // Fragment of 32 elements (half h) of block n of an operand whose chunk begins at `base`.
  const auto fragment = [&](auto slow, uint32_t base, int n, int h) -> F {
    if constexpr (decltype(slow)::value) {
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const uint32_t at = lds0 + base + (in_slow ^ (uint32_t)(n << 5)) + h * 4096;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)(at + 512));
      return __builtin_bit_cast(F, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const F*>(lds + base + (in_row ^ (h * 64)) + n * 2048);
    }
  };
  int slot = 0;
  for (int c = wave; c < chunks; c += kWaves) {
    // Chunk c has landed: only those after it are on their way.
    const int later = (chunks - 1 - c) / kWaves;
    if (later >= kSlots - 1) wait_loads<(kSlots - 1) * kLoads>();
    else if (later == 2 && kSlots > 3) wait_loads<2 * kLoads>();
    else if (later == 1) wait_loads<kLoads>();
    else wait_loads<0>();
    const uint32_t now = wave * kRingBytes + slot * kSlotBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      F b[TN];
#pragma unroll
      for (int n = 0; n < TN; ++n) b[n] = fragment(std::bool_constant<kBSlow>(), now, n, h);
#pragma unroll
      for (int r = 0; r < TM; ++r) {
        const F a = fragment(std::bool_constant<kASlow>(), now + TN * 2048, r, h);
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[r][n] = FewFrag<kF16>::mfma(b[n], a, acc[r][n]);
        if (bias_tile) bias_acc[r] = FewFrag<kF16>::mfma(ones, a, bias_acc[r]);
      }
    }
    // The slot's reads are back; it takes the chunk that comes a ring later.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (c + kSlots * kWaves < chunks) load(c + kSlots * kWaves, slot);
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  float* const mine = reinterpret_cast<float*>(lds + wave * kRingBytes);
  // Lane 16 q + m holds columns 4 q .. 4 q + 3 of row m of each block.
#pragma unroll
  for (int r = 0; r < TM; ++r)
#pragma unroll
    for (int k = 0; k < 4 * TN; ++k)
      mine[(r * 16 + m) * kPitch + k / 4 * 16 + q * 4 + k % 4] = acc[r][k / 4][k % 4];
  if (bias_tile && q == 0) {
#pragma unroll
    for (int r = 0; r < TM; ++r) mine[(r * 16 + m) * kPitch + 16 * TN] = bias_acc[r][0];
  }
  __syncthreads();
  const int32_t out_n = g.out_cols, width = kHalves ? 2 * out_n : out_n;
  uint16_t* const out = static_cast<uint16_t*>(g.out);
  uint16_t* const pre = static_cast<uint16_t*>(g.preact);
  for (int i = threadIdx.x; i < 16 * TM * kOut; i += kWaves * 64) {
    const int r = i / kOut, c = i % kOut, col = first + c;
    if (r >= t.rows || col >= out_n) continue;
    const int64_t row = t.row0 + r;
    float z = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float* const sums = reinterpret_cast<const float*>(lds + w * kRingBytes) + r * kPitch;
      z += sums[c];
      if constexpr (kHalves) up += sums[kOut + c];
    }
    if constexpr (kMode == kWeightsGrad) {
      store_gradient<kF16>(g, g.out, ((int64_t)t.e * g.out_rows + row) * out_n + col, z);
    } else if constexpr (kMode == kRowsGrad) {
      if constexpr (kGlu) {
        const int64_t at = row * 2 * out_n + col;
        const float gate = elem_at<kF16>(pre, at);
        out[at] = elem_rne<kF16>(z * elem_at<kF16>(pre, at + out_n) * silu_slope(gate));
        out[at + out_n] = elem_rne<kF16>(z * silu(gate));
      } else {
        const int64_t at = row * out_n + col;
        if (g.act != EP_ACT_NONE) z = act_backward(g.act, z, elem_at<kF16>(pre, at));
        out[at] = elem_rne<kF16>(z);
      }
    } else {
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
  if (bias_tile && (int)threadIdx.x < t.rows) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      sum += reinterpret_cast<const float*>(lds + w * kRingBytes)[threadIdx.x * kPitch + 16 * TN];
    store_gradient<kF16>(g, g.bias_grad, (int64_t)t.e * g.out_rows + t.row0 + threadIdx.x, sum);
  }
}

template <int kMode, bool kF16, bool kGlu, int TM, int TN>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  constexpr int kOut = kGlu && kMode == kForward ? 8 * TN : 16 * TN;
  const int64_t ct = (g.out_cols + kOut - 1) / kOut;
  const int64_t blocks = kMode == kWeightsGrad
                             ? g.groups.E * ((g.out_rows + 16 * TM - 1) / (16 * TM)) * ct
                             : (max_row_tiles(g.groups, 16 * TM) * ct + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, waves_of(TM) * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_few_kernel<kMode, kF16, kGlu, TM, TN><<<(uint32_t)blocks, waves_of(TM) * 64, 0, stream>>>(g);
  return hipGetLastError();
}
template <bool kF16, bool kGlu>
hipError_t launch_mode(const GemmArgs& g, int mode, int64_t rows, bool wide, hipStream_t stream) {
  if (mode == kWeightsGrad) return launch<kWeightsGrad, kF16, false, 4, 4>(g, stream);
  if (mode == kRowsGrad) return launch<kRowsGrad, kF16, kGlu, 4, 4>(g, stream);
  if (wide) return launch<kForward, kF16, kGlu, 4, 4>(g, stream);
  if (rows <= 16) return launch<kForward, kF16, kGlu, 1, 1>(g, stream);
  if (rows <= 32) return launch<kForward, kF16, kGlu, 2, 1>(g, stream);
  return launch<kForward, kF16, kGlu, 4, 1>(g, stream);
}

}  // namespace

hipError_t launch_gemm_few(const GemmArgs& g, int mode, int64_t rows, bool wide, bool f16, hipStream_t stream) {
  if (g.act == EP_ACT_SWIGLU)
    return f16 ? launch_mode<true, true>(g, mode, rows, wide, stream)
               : launch_mode<false, true>(g, mode, rows, wide, stream);
  return f16 ? launch_mode<true, false>(g, mode, rows, wide, stream)
             : launch_mode<false, false>(g, mode, rows, wide, stream);
}

}  // namespace ep
