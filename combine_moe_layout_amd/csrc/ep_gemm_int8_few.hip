// ep_gemm_int8_few.hip -- products of 8-bit integers with few tiles (a decode step's dense layer, a
// small batch): what counts is to have the whole GPU read the operands.
//
// A workgroup takes 16 TN columns of the product (for swiglu half of them gates and half the ups of
// the same columns) and 16 TM rows, and its waves share out the reduction in chunks of 128.  Each
// wave has a ring of chunks of both operands in LDS to itself, filled by loads that go there
// directly: no barrier before the end, and 8 chunks or more of a workgroup on their way.  The
// waves' sums are exact, so it does not matter in which order they meet.
//
// Bound by what a CU takes in, about 46 GB/s for what it has on its way.  Matrices from
// HBM, 7168 channels: 16 rows, 4096 columns 8.2 us; 8192 columns 12.6; 16,384 columns 22.2 (5.3 TB/s).
#include "ep_int8.h"

namespace ep {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

constexpr int kChunk = 128;  // channels, and bytes of a row, of one wave at a time
// Waves of a workgroup and chunks in a wave's ring: what LDS holds, in 2 (TM + TN) KiB each.
constexpr int waves_of(int TM, int TN) { return TM < 4 && TM + TN < 6 ? 8 : 4; }
constexpr int slots_of(int TM, int TN) {
  const int fit = 80 / (waves_of(TM, TN) * (TM + TN));
  return fit < 4 ? fit : 4;
}

template <bool kGlu, int TM, int TN>
__global__ __launch_bounds__(waves_of(TM, TN) * 64, waves_of(TM, TN) / 4) void gemm_int8_few_kernel(GemmArgs g) {
  constexpr int kWaves = waves_of(TM, TN), kSlots = slots_of(TM, TN);
  constexpr int kOut = kGlu ? 8 * TN : 16 * TN;  // result columns of a workgroup
  constexpr int kPitch = 16 * TN + 1;            // ints of a row's sums in LDS
  constexpr int kLoads = 2 * TN + 2 * TM;        // of a chunk: 8 rows each, the matrix's first
  constexpr int kSlotBytes = kLoads * 1024, kRingBytes = kSlots * kSlotBytes;
  __shared__ __align__(1024) char lds[kWaves * kRingBytes];
  static_assert(16 * TM * kPitch * 4 <= kRingBytes, "the sums take the ring's place");
  // Up to four row tiles of a group at a column, so that an XCD reads that part of the matrix once: 256
  // rows, 7168 x 4096, 22.6 us, row tile by row tile 24.7.
  Tile t;
  if (!find_tile<4, true>(g.groups, 16 * TM, (g.out_cols + kOut - 1) / kOut, blockIdx.x, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, q = lane >> 4;
  const int first = t.col * kOut;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
  const uint32_t ring = lds0 + wave * kRingBytes;

  // Load j: lane l row 8 j + l / 8; 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7), so that
  // the fragment reads below touch every bank once in each of their phases.
  const char* const b0 = static_cast<const char*>(g.b) + t.e * g.b_stride + (int64_t)first * g.ldb;
  const char* const ups = b0 + (int64_t)g.out_cols * g.ldb;
  const char* const a0 = static_cast<const char*>(g.a) + t.row0 * g.lda;
  uint32_t offset[kLoads];
  int place[kLoads];  // first of the load's 16 channels in the chunk
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const bool of_b = j < 2 * TN;
    const int row = j * 8 + (lane >> 3), r = of_b ? row % kOut : row - 16 * TN;
    const int last = of_b ? g.out_cols - 1 - first : t.rows - 1;
    place[j] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    offset[j] = (uint32_t)min(r, last) * (uint32_t)(of_b ? g.ldb : g.lda) + place[j];
  }
  const int chunks = tiles_of(g.reduce, kChunk), whole = g.reduce / kChunk;
  const auto load = [&](int c, int slot) {
    const uint32_t to = ring + slot * kSlotBytes;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const char* const from = (j >= 2 * TN ? a0 : kGlu && j >= TN ? ups : b0) + c * kChunk;
      if (c < whole)
        load16_to_lds(from, offset[j], to + j * 1024);
      else  // past the reduction: zeros
        load16_to_lds(c * kChunk + place[j] < g.reduce ? from + offset[j] : reinterpret_cast<const char*>(g_zero16),
                      to + j * 1024);
    }
  };
  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int n = 0; n < TN; ++n) acc[i][n] = i32x4{0, 0, 0, 0};
  // Chunks wave, wave + kWaves, ..: every slot of the ring is filled, and a slot is
  // filled again as soon as its chunk has been read.
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (wave + i * kWaves < chunks) load(wave + i * kWaves, i);
  const uint32_t in_row = m * 128 + ((q ^ ((m >> 1) & 7)) << 4);
  // Lane 16 q + m: 16 channels of row m of block n, of the chunk's half h.
  const auto fragment = [&](uint32_t base, int n, int h) {
    return *reinterpret_cast<const i32x4*>(lds + base + (in_row ^ (h * 64)) + n * 2048);
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
      i32x4 b[TN];
#pragma unroll
      for (int n = 0; n < TN; ++n) b[n] = fragment(now, n, h);
#pragma unroll
      for (int r = 0; r < TM; ++r) {
        const i32x4 a = fragment(now + TN * 2048, r, h);
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[r][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[n], a, acc[r][n], 0, 0, 0);
      }
    }
    // The slot's reads are back; it takes the chunk that comes a ring later.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (c + kSlots * kWaves < chunks) load(c + kSlots * kWaves, slot);
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  // Lane 16 q + m holds columns 4 q .. 4 q + 3 of row m of each block.
  int* const mine = reinterpret_cast<int*>(lds + wave * kRingBytes);
#pragma unroll
  for (int r = 0; r < TM; ++r)
#pragma unroll
    for (int k = 0; k < 4 * TN; ++k)
      mine[(r * 16 + m) * kPitch + k / 4 * 16 + q * 4 + k % 4] = acc[r][k / 4][k % 4];
  __syncthreads();
  const int32_t n = g.out_cols, width = kGlu ? 2 * n : n;
  uint16_t* const out = static_cast<uint16_t*>(g.out);
  uint16_t* const pre = static_cast<uint16_t*>(g.preact);
  const float* const row_scales = static_cast<const float*>(g.a_scales) + t.row0;
  const float* const col_scales = static_cast<const float*>(g.b_scales) + (int64_t)t.e * width;
  for (int i = threadIdx.x; i < 16 * TM * kOut; i += kWaves * 64) {
    const int r = i / kOut, c = i % kOut, col = first + c;
    if (r >= t.rows || col >= n) continue;
    const int64_t row = t.row0 + r;
    int sum = 0, sum_up = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int* const sums = reinterpret_cast<const int*>(lds + w * kRingBytes) + r * kPitch;
      sum += sums[c];
      if constexpr (kGlu) sum_up += sums[kOut + c];
    }
    float row_scale = row_scales[r];
    const float part = split_scale(row_scale) ? kLargePart : 1.0f;
    float z = (float)sum * row_scale * col_scales[col] * part, up = 0.0f;
    if constexpr (kGlu) up = (float)sum_up * row_scale * col_scales[n + col] * part;
    if (g.bias != nullptr) {
      z += elem_at<false>(g.bias, (int64_t)t.e * width + col);
      if constexpr (kGlu) up += elem_at<false>(g.bias, (int64_t)t.e * width + n + col);
    }
    if (pre != nullptr) {
      pre[row * width + col] = elem_rne<false>(z);
      if constexpr (kGlu) pre[row * width + n + col] = elem_rne<false>(up);
    }
    float v = kGlu ? silu(z) * up : act_value(g.act, z);
    if (g.residual != nullptr) v += elem_at<false>(g.residual, row * n + col);
    out[row * n + col] = elem_rne<false>(v);
  }
}

template <bool kGlu, int TM, int TN>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  constexpr int kOut = kGlu ? 8 * TN : 16 * TN;
  const int64_t ct = (g.out_cols + kOut - 1) / kOut;
  const int64_t blocks = (max_row_tiles(g.groups, 16 * TM) * ct + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, waves_of(TM, TN) * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_int8_few_kernel<kGlu, TM, TN><<<(uint32_t)blocks, waves_of(TM, TN) * 64, 0, stream>>>(g);
  return hipGetLastError();
}
template <bool kGlu, int TM>
hipError_t launch_width(const GemmArgs& g, int32_t width, hipStream_t stream) {
  if (width == 16) return launch<kGlu, TM, 1>(g, stream);
  if (width == 32) return launch<kGlu, TM, 2>(g, stream);
  return launch<kGlu, TM, 4>(g, stream);
}
template <bool kGlu>
hipError_t launch_height(const GemmArgs& g, int32_t height, int32_t width, hipStream_t stream) {
  if (height == 16) return launch_width<kGlu, 1>(g, width, stream);
  if (height == 32) return launch_width<kGlu, 2>(g, width, stream);
  return launch_width<kGlu, 4>(g, width, stream);
}

}  // namespace

hipError_t launch_gemm_int8_few(const GemmArgs& g, int32_t height, int32_t width, hipStream_t stream) {
  return g.act == EP_ACT_SWIGLU ? launch_height<true>(g, height, width, stream)
                                : launch_height<false>(g, height, width, stream);
}

}  // namespace ep
