// ep_gemm_few.hip -- bf16 and fp16 products with few tiles (a decode step's dense
// layer, a small batch): what counts is to have the whole GPU read the matrix.
//
//   out[r, n] = act(sum_k a[r, k] b[e, n, k] + bias[e, n]) + residual[r, n]
//
// A workgroup takes 16 TN rows of the matrix (for swiglu half of them gates and
// half the ups of the same columns) against 16 TM rows of a, and its waves share
// out the reduction in chunks of 64.  TN = 1: a product of 4096 columns has a
// workgroup for every CU; TM = TN = 4 for more rows.  Each wave has a ring of
// chunks of both operands in LDS to itself, so there is no barrier before the
// end, and a workgroup has 8 chunks or more on their way, where tiles whose waves
// share every chunk have two.  (LDS is for the address unit: a load costs it 2.6
// cycles for each 128-byte line that it touches.  In the order of the matrix
// instruction a load touches 16 lines; through LDS it takes 8 whole ones.)  The
// waves' sums meet in LDS and are added in wave order, so the result does not
// depend on timing.
//
// Measured, reduction 7168 and 4096 columns: 1 row 11.8 us (58.7 MB, 5.0 TB/s), 16
// rows 14, 32 rows 17, 64 rows 22; 256 rows 40 us (TN = 4).  Before the rings, with
// fragments loaded straight into registers: 14.3, 18.5, 23 and 35 us.
#include "ep_gemm.h"

namespace ep {

namespace {

constexpr int kChunk = 64;  // reduction elements of one wave at a time: 128 bytes of a row
// Waves of a workgroup and chunks in a wave's ring: what LDS holds.
constexpr int waves_of(int TM) { return TM < 4 ? 8 : 4; }
constexpr int slots_of(int TM, int TN) { return TN > 1 ? 2 : TM == 2 ? 3 : 4; }

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

template <bool kF16, bool kGlu, int TM, int TN>
__global__ __launch_bounds__(waves_of(TM) * 64, waves_of(TM) / 4) void gemm_few_kernel(GemmArgs g) {
  typedef typename FewFrag<kF16>::type F;
  constexpr int kWaves = waves_of(TM), kSlots = slots_of(TM, TN);
  constexpr int kOut = kGlu ? 8 * TN : 16 * TN;   // result columns of a workgroup
  constexpr int kPitch = 16 * TN + 1;             // floats of a row's sums in LDS
  constexpr int kLoads = 2 * TN + 2 * TM;         // of a chunk: 8 rows each
  constexpr int kSlotBytes = kLoads * 1024, kRingBytes = kSlots * kSlotBytes;
  __shared__ __align__(1024) char lds[kWaves * kRingBytes];
  static_assert(16 * TM * kPitch * 4 <= kRingBytes, "the sums take the ring's place");
  Tile t;
  if (!find_tile<1>(g.groups, 16 * TM, (g.out_cols + kOut - 1) / kOut, blockIdx.x, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  const int first = t.col * kOut;
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_address(lds)) + wave * kRingBytes;

  // Load j brings rows 8 j .. 8 j + 7 of a chunk (the first 16 TN are the
  // matrix's): lane l row l / 8; 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7),
  // so that the fragment reads below touch every bank once in each of their phases.
  const char* const b0 = static_cast<const char*>(g.b) + t.e * g.b_stride * 2 + (int64_t)first * g.ldb * 2;
  const char* const ups = b0 + (int64_t)g.out_cols * g.ldb * 2;
  const char* const a0 = static_cast<const char*>(g.a) + t.row0 * g.lda * 2;
  uint32_t offset[kLoads];
  int piece[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int row = j * 8 + (lane >> 3);
    piece[j] = (lane & 7) ^ ((row >> 1) & 7);
    offset[j] = (j < 2 * TN ? (uint32_t)min(row % kOut, g.out_cols - 1 - first) * (uint32_t)g.ldb
                            : (uint32_t)min(row - 16 * TN, t.rows - 1) * (uint32_t)g.lda) * 2u + piece[j] * 16;
  }
  const int chunks = (g.reduce + kChunk - 1) / kChunk, whole = g.reduce / kChunk;
  const auto load = [&](int c, int slot) {
    const uint32_t to = ring + slot * kSlotBytes;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const char* const from = (j >= 2 * TN ? a0 : kGlu && j >= TN ? ups : b0) + (int64_t)c * (kChunk * 2);
      if (c < whole)
        load16_to_lds(from, offset[j], to + j * 1024);
      else  // past the reduction: zeros
        load16_to_lds(c * kChunk + piece[j] * 8 < g.reduce ? from + offset[j] : reinterpret_cast<const char*>(g_zero16),
                      to + j * 1024);
    }
  };
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM * TN; ++i) acc[i / TN][i % TN] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Chunks wave, wave + kWaves, ..: all but one of the ring's slots ahead.
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (wave + i * kWaves < chunks) load(wave + i * kWaves, i);
  const uint32_t in_row = m * 128 + ((q ^ ((m >> 1) & 7)) << 4);
  int slot = 0;
  for (int c = wave; c < chunks; c += kWaves) {
    // Chunk c has landed: only those after it are on their way.
    const int later = (chunks - 1 - c) / kWaves;
    if (later >= kSlots - 1) wait_loads<(kSlots - 1) * kLoads>();
    else if (later == 2 && kSlots > 3) wait_loads<2 * kLoads>();
    else if (later == 1) wait_loads<kLoads>();
    else wait_loads<0>();
    const uint32_t now = wave * kRingBytes + slot * kSlotBytes + in_row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 32 elements each: chunks q and q + 4 of the rows
      const char* const at = lds + (now ^ (h * 64));
      F b[TN];
#pragma unroll
      for (int n = 0; n < TN; ++n) b[n] = *reinterpret_cast<const F*>(at + n * 2048);
#pragma unroll
      for (int r = 0; r < TM; ++r) {
        const F a = *reinterpret_cast<const F*>(at + (TN + r) * 2048);
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[r][n] = FewFrag<kF16>::mfma(b[n], a, acc[r][n]);
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
      const float* const sums = reinterpret_cast<const float*>(lds + w * kRingBytes) + r * kPitch;
      z += sums[c];
      if constexpr (kGlu) up += sums[kOut + c];
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

template <bool kF16, bool kGlu, int TM, int TN>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  constexpr int kOut = kGlu ? 8 * TN : 16 * TN;
  const int64_t ct = (g.out_cols + kOut - 1) / kOut;
  const int64_t blocks = (max_row_tiles(g.groups, 16 * TM) * ct + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, waves_of(TM) * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_few_kernel<kF16, kGlu, TM, TN><<<(uint32_t)blocks, waves_of(TM) * 64, 0, stream>>>(g);
  return hipGetLastError();
}
template <bool kF16, bool kGlu>
hipError_t launch_rows(const GemmArgs& g, int64_t rows, bool wide, hipStream_t stream) {
  if (wide) return launch<kF16, kGlu, 4, 4>(g, stream);
  if (rows <= 16) return launch<kF16, kGlu, 1, 1>(g, stream);
  if (rows <= 32) return launch<kF16, kGlu, 2, 1>(g, stream);
  return launch<kF16, kGlu, 4, 1>(g, stream);
}

}  // namespace

hipError_t launch_gemm_few(const GemmArgs& g, int64_t rows, bool wide, bool f16, hipStream_t stream) {
  if (g.act == EP_ACT_SWIGLU)
    return f16 ? launch_rows<true, true>(g, rows, wide, stream) : launch_rows<false, true>(g, rows, wide, stream);
  return f16 ? launch_rows<true, false>(g, rows, wide, stream) : launch_rows<false, false>(g, rows, wide, stream);
}

}  // namespace ep
