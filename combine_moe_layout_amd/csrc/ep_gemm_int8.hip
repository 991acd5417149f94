// ep_gemm_int8.hip -- the products of 8-bit integers with a scale for each row and each column:
//
//   z[r, n] = row_scale[r] col_scale[e, n] sum_c x[r, c] w[e, n, c]
//
// The sum is exact: at most 65,536 products of magnitude at most 2^14 in 32 bits.  It is rounded
// to fp32 once, and the scales, bias, activation and residual follow in fp32.
//
// A workgroup of 8 waves makes a tile of 192 rows and 256 columns, 96 x 64 to a wave (64 x 128,
// 32 x 32 to a wave, where that is too much for the rows there are).  A stage is 128 channels.
// While the matrix instructions work on stage s, both operands of stage s + 2 come into LDS: it
// holds three stages of rows and two of the matrix operand, whose fragments of stage s have been
// in registers since stage s - 1 ended.
#include "ep_int8.h"

namespace ep {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

constexpr int kWaves = 8;
constexpr int kASlots = 3;   // stages of rows in LDS
constexpr int kBSlots = 2;   // stages of the matrix operand
constexpr int kStage = 128;  // channels, and bytes, per stage

// Lane 16 q + m holds channels 16 q .. 16 q + 15 (`lo`) and 64 + 16 q .. (`hi`) of row m.
struct Fragment {
  i32x4 lo, hi;
};

template <bool kGlu, int TM, int TN, int WM, int WN>
struct Int8Gemm {
  static_assert(WM * WN == kWaves, "eight waves");
  static constexpr int kRows = 16 * TM * WM, kCols = 16 * TN * WN, kWaveCols = 16 * TN;
  static constexpr int kABytes = kRows * kStage, kBBytes = kCols * kStage;
  static constexpr int kBAt = kASlots * kABytes;
  static constexpr int kLdsBytes = kBAt + kBSlots * kBBytes;
  static constexpr int kALoads = kABytes / 1024 / kWaves, kBLoads = kBBytes / 1024 / kWaves;
  static_assert(kBLoads * 8 == kWaveCols / 2, "a wave loads half of a wave's columns");
  static constexpr int kWaveBytes = kLdsBytes / kWaves / 1024 * 1024;
  typedef TileStore<kForward, false, kGlu, TM, TN, WM, WN, kWaveBytes> Store;
  static constexpr int kOutCols = Store::kOutCols;
  static constexpr int kRing = 4;  // row fragments in registers: two in use, two read ahead
  static_assert(TM % kRing == 2, "two stages leave the ring where it was");
  static constexpr int kTurn = TM - 2;  // the row of blocks before which stage s + 1 has landed
  static constexpr int kLoads = kALoads + kBLoads;

  const GemmArgs& g;
  char* const lds;
  uint32_t lds0;
  Tile t;
  int32_t stages, whole, blocks;
  const char *a0, *b0;
  uint32_t a_off[kALoads], b_off[kBLoads];
  uint32_t a_read, b_read;
  int wm, wn, lane, wave, turn;
  i32x4 acc[TM][TN];
  Fragment af[kRing], bf[2][TN];

  __device__ __forceinline__ Int8Gemm(const GemmArgs& args, char* smem) : g(args), lds(smem) {}

  __device__ __forceinline__ int row_at(int p) const {
    return matrix_row(kGlu, p, kWaveCols, t.col * kOutCols, g.out_cols);
  }

  __device__ __forceinline__ void setup() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    turn = kTurns == 2 ? wave / 4 : 0;
    lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
    stages = tiles_of(g.reduce, kStage);
    whole = g.reduce / kStage;
    blocks = __builtin_amdgcn_readfirstlane(((t.rows + 15) / 16 - wm + WM - 1) / WM);
    a0 = static_cast<const char*>(g.a) + t.row0 * g.lda;
    // A load brings 8 rows of 128 bytes; 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7), so
    // that 16 rows read at one chunk touch every bank once.
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int row = (wave * kALoads + i) * 8 + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
      a_off[i] = (uint32_t)min(row, t.rows - 1) * (uint32_t)g.lda + chunk * 16;
    }
    // A wave loads half of some wave's columns, all gates or all ups: they are neighbours, up to
    // the last column.
    const int base = row_at(wave * kBLoads * 8);
    b0 = static_cast<const char*>(g.b) + t.e * g.b_stride + (int64_t)base * g.ldb;
#pragma unroll
    for (int i = 0; i < kBLoads; ++i) {
      const int row = (wave * kBLoads + i) * 8 + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
      b_off[i] = (uint32_t)(row_at(row) - base) * (uint32_t)g.ldb + chunk * 16;
    }
    const int q = lane >> 4, m = lane & 15;
    const uint32_t in_row = m * kStage + ((q ^ ((m >> 1) & 7)) << 4);
    a_read = wm * 16 * kStage + in_row;
    b_read = kBAt + wn * kWaveCols * kStage + in_row;
  }

  // Load j of stage s: of the row operand (into slot `slot`), of the matrix operand.  Chunks past
  // the end of the reduction are zeros on both sides.
  __device__ __forceinline__ void load_piece(int s, uint32_t slot, int j) const {
    const bool of_a = j < kALoads;
    const int i = of_a ? j : j - kALoads;
    const char* const from = (of_a ? a0 : b0) + s * kStage;
    const uint32_t off = of_a ? a_off[of_a ? i : 0] : b_off[of_a ? 0 : i];
    const uint32_t to = of_a ? lds0 + slot * kABytes + (wave * kALoads + i) * 1024
                             : lds0 + kBAt + (s & 1) * kBBytes + (wave * kBLoads + i) * 1024;
    if (s < whole) {
      load16_to_lds(from, off, to);
    } else {
      const int row = (wave * (of_a ? kALoads : kBLoads) + i) * 8 + (lane >> 3);
      const int channel = s * kStage + (((lane & 7) ^ ((row >> 1) & 7)) * 16);
      load16_to_lds(channel < g.reduce ? from + off : reinterpret_cast<const char*>(g_zero16), to);
    }
  }

  __device__ __forceinline__ Fragment read_fragment(uint32_t offset) const {
    return Fragment{*reinterpret_cast<const i32x4*>(lds + offset), *reinterpret_cast<const i32x4*>(lds + (offset ^ 64))};
  }
  __device__ __forceinline__ Fragment row_fragment(uint32_t slot, int i) const {
    return read_fragment(slot * kABytes + a_read + i * (WM * 16 * kStage));
  }
  template <int kSet>
  __device__ __forceinline__ void read_matrix(uint32_t b_slot, int j) {
    bf[kSet][j] = read_fragment(b_slot * kBBytes + b_read + j * (16 * kStage));
  }

  // Stage s, kSet = s & 1, its rows in slot `now`, those of the next two stages in `next` and
  // `after`.  Its matrix fragments are in the registers of kSet, its first two row fragments in
  // af (row block i's in af[(2 kSet + i) % kRing]); the next stage's are read as soon as it has
  // landed, in the last two row blocks.
  template <int kSet>
  __device__ __forceinline__ void step(int s, uint32_t now, uint32_t next, uint32_t after) {
    // Every wave is done with the rows of stage s - 1, and has the matrix operand of stage s in
    // registers (the youngest two reads are of this stage's second row fragment).
    lds_barrier<2>();
    const bool more2 = s + 2 < stages;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      load_in_row(i, more2, s, after);
      if (i == kTurn) {
        // Stage s + 1 has landed, for every wave: only the loads of stage s + 2 may be on their way.
        if (!more2) wait_loads<0>();
        else if (turn == 0) wait_loads<issued(kTurn, 0)>();
        else wait_loads<issued(kTurn, 1)>();
        lds_barrier<15>();
      }
      const int f = i + 2;
      af[(2 * kSet + f) % kRing] = f < TM ? row_fragment(now, f) : row_fragment(next, f - TM);
      if (i == kTurn) {
#pragma unroll
        for (int j = 0; j < TN; ++j) read_matrix<1 - kSet>((s + 1) & 1, j);
      }
      if (i < blocks) {
        const Fragment& a = af[(2 * kSet + i) % kRing];
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[kSet][j].lo, a.lo, acc[i][j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[kSet][j].hi, a.hi, acc[i][j], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Each SIMD has one of the first four waves and one of the others; the former load in the first
  // half of the rows, the latter in the second.  A load holds its wave until the address unit has
  // taken it, and only the other wave keeps the matrix unit busy then.  (Tiles of two row blocks
  // a wave are for streaming the matrix: all load at once.)
  static constexpr int kTurns = TM > 2 ? 2 : 1;
  static constexpr int kHalf = TM / 2, kPieces = (kLoads + kHalf - 1) / kHalf;
  static constexpr int issued(int row, int turn) {  // loads of a wave when it has been through `row`
    const int n = (row + 1 - turn * kHalf) * kPieces;
    return n < 0 ? 0 : n < kLoads ? n : kLoads;
  }
  __device__ __forceinline__ void load_in_row(int i, bool more2, int s, uint32_t slot) const {
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      const int j = i % kHalf * kPieces + n;
      if (more2 && turn == i / kHalf && j < kLoads) load_piece(s + 2, slot, j);
    }
  }

  __device__ __forceinline__ void accumulate() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load_piece(0, 0, j);
    if (stages > 1) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) load_piece(1, 1, j);
    }
    if (stages > 1) wait_loads<kLoads>();
    else wait_loads<0>();
    lds_barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j) read_matrix<0>(0, j);
    af[0] = row_fragment(0, 0);
    af[1] = row_fragment(0, 1);
    // (past the last stage, fragments are read from a slot that nobody uses)
    uint32_t slot = 0;
    for (int s = 0; s < stages; s += 2) {
      const uint32_t one = slot == 2 ? 0 : slot + 1, two = one == 2 ? 0 : one + 1;
      step<0>(s, slot, one, two);
      if (s + 1 < stages) step<1>(s + 1, one, two, slot);
      slot = two;
    }
  }

  __device__ __forceinline__ void run() {
    const int32_t ct = (g.out_cols + kOutCols - 1) / kOutCols;
    if (!find_tile<4>(g.groups, kRows, ct, blockIdx.x, t)) return;
    setup();
    accumulate();
    lds_barrier();
    // Lane 16 q + m: row m of each block, columns 4 q .. 4 q + 3.
    const float* const row_scales = static_cast<const float*>(g.a_scales) + t.row0;
    const float* const col_scales = static_cast<const float*>(g.b_scales) + t.e * (g.b_stride / g.ldb);
    float scale[TM];
    f32x4 sums[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) scale[i] = row_scales[min((i * WM + wm) * 16 + (lane & 15), t.rows - 1)];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float col = col_scales[row_at(wn * kWaveCols + j * 16 + (lane >> 4) * 4 + c)];
#pragma unroll
        for (int i = 0; i < TM; ++i) sums[i][j][c] = (float)acc[i][j][c] * scale[i] * col;
      }
    Store::store_tile(g, t, lds + wave * kWaveBytes, wm, wn, sums);
  }
};

template <bool kGlu, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(kWaves * 64, TM > 2 ? 2 : 4) void gemm_int8_kernel(GemmArgs g) {
  typedef Int8Gemm<kGlu, TM, TN, WM, WN> G;
  __shared__ __align__(1024) char lds[G::kLdsBytes];
  G gemm(g, lds);
  gemm.run();
}

template <bool kGlu, int TM, int TN, int WM, int WN>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  typedef Int8Gemm<kGlu, TM, TN, WM, WN> G;
  const int64_t ct = (g.out_cols + G::kOutCols - 1) / G::kOutCols;
  const int64_t blocks = (max_row_tiles(g.groups, G::kRows) * ct + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, kWaves * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_int8_kernel<kGlu, TM, TN, WM, WN><<<(uint32_t)blocks, kWaves * 64, 0, stream>>>(g);
  return hipGetLastError();
}

// Tiles of 64 x 128, two workgroups to a CU, where the big ones would leave the GPU waiting:
// experts of few rows, whose products read the matrix and little else, and products with so few
// tiles that all of the small ones run at once.
template <bool kGlu>
hipError_t launch_size(const GemmArgs& g, hipStream_t stream) {
  const RowGroups& r = g.groups;
  const int64_t groups = r.wanted > r.E ? r.E : r.wanted, rows = (r.wanted + r.E - 1) / r.E;
  const int64_t columns = (int64_t)g.out_cols * (kGlu ? 2 : 1);
  const bool small = rows <= 32 || groups * ((rows + 63) / 64) * ((columns + 127) / 128) <= 2 * kChipCUs;
  return small ? launch<kGlu, 2, 2, 2, 4>(g, stream) : launch<kGlu, 6, 4, 2, 4>(g, stream);
}

}  // namespace

hipError_t launch_gemm_int8(const GemmArgs& g, hipStream_t stream) {
  return g.act == EP_ACT_SWIGLU ? launch_size<true>(g, stream) : launch_size<false>(g, stream);
}

}  // namespace ep
