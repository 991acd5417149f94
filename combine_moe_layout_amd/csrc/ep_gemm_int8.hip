// ep_gemm_int8.hip -- the products of 8-bit integers with a scale for each row and each column:
//
//   z[r, n] = row_scale[r] col_scale[e, n] sum_c x[r, c] w[e, n, c]
//
// The sum is exact: at most 65,536 products of magnitude at most 2^14 in 32 bits.  It is rounded
// to fp32 once, and the scales, bias, activation and residual follow in fp32.
//
// A workgroup of 8 waves makes a tile of up to 128, 192 or 256 rows and 256 columns, 128 x 64 to a
// wave (128 x 128 or 64 x 128, 64 x 32 or 32 x 32 to a wave, where there are few).  A stage is 128
// channels, walked as two halves of 64 (the matrix instruction's reduction): a wave holds its
// columns' fragments of one half, and goes through its row blocks with three of theirs read ahead,
// so that 128 sums and all fragments fit 241 registers.  (Fragments of whole stages, twice, spilled;
// a spilled register's reload waits for the loads to LDS as well.)
//
// What bounds a stage of a short tile is LDS: of 128 bytes a cycle, a stage's fragments take 128 RB +
// 512 cycles and its loads 32 RB + 256, the matrix instructions 256 RB (RB row blocks to a wave), so
// that short tiles cost what RB + 2 row blocks would.  Four waves of 128 x 128 read a third less, but
// with one wave to a SIMD nothing hides its waits: 8192^3 in 440 us.
//
// LDS holds two stages of rows and three of the matrix operand, all 160 KiB of it.  There is one
// barrier to a stage, three slots before its end, where its last rows have been read and the next
// stage has landed: after it the rows of stage s + 2 take the place of those of stage s, and the
// matrix operand of stage s + 3 that of stage s.  So the matrix, which may come from HBM, is on
// its way for two stages.
//
// The stages of a tile are code without a branch, made for each number of row blocks from 2 to 8:
// two waves share a matrix unit, and one hides what the other does besides only as long as that is
// shorter than four matrix instructions.  Branches around the row blocks and loads made the
// product of 8192^3 470 us; without them it takes 384 (2.9 POP/s; the same matrix instructions
// alone, without loads and LDS reads, 300).  65,536 rows of 7168 channels to 4096 columns: 1470 us
// (2.6 POP/s) for 16 matrices, 1830 for 256 of 256 rows each (7.5 GB of matrices, 4.1 TB/s), 2130
// where experts have 256 rows on average (1.8 POP/s): those with more make two tiles.
#include "ep_int8.h"
#include "ep_int8_tiles.h"

namespace ep {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

constexpr int kWaves = 8;
constexpr int kASlots = 2;   // stages of rows in LDS
constexpr int kBSlots = 3;   // stages of the matrix operand
constexpr int kStage = 128;  // channels, and bytes, per stage
constexpr int kAhead = 3;    // row fragments read ahead
constexpr int kRing = 4;     // row fragments in registers

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
  static_assert(2 * TM % kRing == 0, "a stage leaves the ring where it was");

  const GemmArgs& g;
  char* const lds;
  uint32_t lds0;
  Tile t;
  int32_t stages, whole;  // stages, and those of 128 channels
  int32_t blocks;         // row blocks of a wave that any wave has
  int32_t a_loads;        // loads of rows of a wave and stage
  const char *a0, *b0;
  uint32_t a_off[kALoads], b_off[kBLoads];
  uint32_t a_read, b_read;
  int wm, wn, lane, wave;
  i32x4 acc[TM][TN];
  // Lane 16 q + m holds channels 16 q .. 16 q + 15 of a half of row m.
  i32x4 af[kRing], bf[2][TN];

  __device__ __forceinline__ Int8Gemm(const GemmArgs& args, char* smem) : g(args), lds(smem) {}

  __device__ __forceinline__ int row_at(int p) const {
    return matrix_row(kGlu, p, kWaveCols, t.col * kOutCols, g.out_cols);
  }

  __device__ __forceinline__ void setup() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
    stages = tiles_of(g.reduce, kStage);
    whole = g.reduce / kStage;
    blocks = __builtin_amdgcn_readfirstlane((t.rows + 16 * WM - 1) / (16 * WM));
    a_loads = (blocks * 2 * WM + kWaves - 1) / kWaves;
    a0 = static_cast<const char*>(g.a) + t.row0 * g.lda;
    // A load brings 8 rows of 128 bytes; 16-byte chunk c of row r lies at c ^ ((r >> 1) & 7), so
    // that 16 rows read at one chunk touch every bank once.  Rows past the last are the last.
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int row = a_group(i) * 8 + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
      a_off[i] = (uint32_t)min(row, t.rows - 1) * (uint32_t)g.lda + chunk * 16;
    }
    // A wave loads half of some wave's columns, all gates or all ups: they are neighbours, up to
    // the last column.
    const int base = row_at(wave * kBLoads * 8);
    b0 = static_cast<const char*>(g.b) + t.e * g.b_stride + (int64_t)base * g.ldb;
#pragma unroll
    for (int i = 0; i < kBLoads; ++i) {
      const int row = b_group(i) * 8 + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
      b_off[i] = (uint32_t)(row_at(row) - base) * (uint32_t)g.ldb + chunk * 16;
    }
    const int q = lane >> 4, m = lane & 15;
    const uint32_t in_row = m * kStage + ((q ^ ((m >> 1) & 7)) << 4);
    a_read = wm * 16 * kStage + in_row;
    b_read = kBAt + wn * kWaveCols * kStage + in_row;
  }

  // Load i of a wave brings rows 8 group .. 8 group + 7 of the operand's part of a stage.
  __device__ __forceinline__ int a_group(int i) const { return wave + i * kWaves; }
  __device__ __forceinline__ int b_group(int i) const { return wave * kBLoads + i; }
  // kWhole: stage s has all its 128 channels; otherwise those past the last are zeros.
  template <bool kWhole>
  __device__ __forceinline__ void load(const char* from, uint32_t off, uint32_t to, int s, int group) const {
    if (kWhole || s < whole) {
      load16_to_lds(from + s * kStage, off, to);
    } else {
      const int row = group * 8 + (lane >> 3);
      const int channel = s * kStage + (((lane & 7) ^ ((row >> 1) & 7)) * 16);
      load16_to_lds(channel < g.reduce ? from + s * kStage + off : reinterpret_cast<const char*>(g_zero16), to);
    }
  }
  template <bool kWhole>
  __device__ __forceinline__ void load_rows(int s, int i) const {
    load<kWhole>(a0, a_off[i], lds0 + (s & 1) * kABytes + a_group(i) * 1024, s, a_group(i));
  }
  template <bool kWhole>
  __device__ __forceinline__ void load_matrix(int s, uint32_t slot, int i) const {
    load<kWhole>(b0, b_off[i], lds0 + kBAt + slot * kBBytes + b_group(i) * 1024, s, b_group(i));
  }

  // Slot u of a stage of RB row blocks: half u / RB, row block u % RB; rows at `at`.
  template <int RB>
  __device__ __forceinline__ i32x4 row_fragment(uint32_t at, int u) const {
    return *reinterpret_cast<const i32x4*>(lds + ((at + a_read) ^ (u / RB * 64)) + u % RB * (WM * 16 * kStage));
  }
  __device__ __forceinline__ void read_matrix(uint32_t slot, int h, int j) {
    bf[h][j] = *reinterpret_cast<const i32x4*>(lds + ((slot * kBBytes + b_read) ^ (h * 64)) + j * (16 * kStage));
  }

  // An epoch, from one barrier to the next, issues the loads of the rows of stage `s` and of the
  // matrix of stage s + 1: the first three loads of rows in the three slots after the barrier, the
  // others over the next stage's 2 RB - 3 slots before its barrier.  Place of load j of those.
  template <int RB>
  static constexpr int late_slot(int j, int n) { return j * (2 * RB - kAhead) / n; }

  // Stage s; its matrix in slot `now`, those of the next two in `next` and `last`; kPar: which half
  // of the ring holds its first row fragments.  kFast: all row blocks in use, and every load of a
  // whole stage.
  template <int RB, bool kFast, int kPar>
  __device__ __forceinline__ void stage(int s, uint32_t now, uint32_t next, uint32_t last) {
    constexpr int kSlots = 2 * RB, kTurn = kSlots - kAhead, kFrom = kPar * kSlots % kRing;
    constexpr int kRowLoads = (RB * 2 * WM + kWaves - 1) / kWaves;
    constexpr int kLate = (kRowLoads > kAhead ? kRowLoads - kAhead : 0) + kBLoads;
    const uint32_t at = (s & 1) * kABytes, at_next = kABytes - at;
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      if (u == kTurn) {
        // The rows of stage s + 1 have landed (the youngest loads are of the matrix of stage s + 2,
        // all others older), and this wave has read all it needs of stage s.
        if (kFast || s + 2 < stages) wait_loads<kBLoads>();
        else wait_loads<0>();
        lds_barrier();
      }
      if (u >= kTurn) {
        const int i = u - kTurn;
        if (i < kRowLoads && (kFast || (i < a_loads && s + 2 < stages))) load_rows<kFast>(s + 2, i);
      } else {
#pragma unroll
        for (int j = 0; j < kLate; ++j) {
          if (late_slot<RB>(j, kLate) != u) continue;
          const int i = j - (kLate - kBLoads);  // of the matrix, or of the rows from the fourth on
          if (i >= 0) {
            if (kFast || s + 2 < stages) load_matrix<kFast>(s + 2, last, i);
          } else if (kFast || (kAhead + j < a_loads && s + 1 < stages)) {
            load_rows<kFast>(s + 1, kAhead + j);
          }
        }
      }
      const int v = u + kAhead;
      i32x4& ahead = af[(kFrom + v) % kRing];
      if (v >= kSlots) ahead = row_fragment<RB>(at_next, v - kSlots);
      else if (kFast || v % RB < blocks) ahead = row_fragment<RB>(at, v);
      // The second half's columns, before they are used and before the barrier; the next stage's,
      // after it and in the second half.
      constexpr int kHalfFrom = RB > TN + 2 ? RB - TN - 2 : 0, kHalfTo = RB < kTurn ? RB - 1 : kTurn - 1;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (u == (kHalfFrom + j < kHalfTo ? kHalfFrom + j : kHalfTo)) read_matrix(now, 1, j);
        if (u == (kTurn > RB ? kTurn : RB) + j / 2) read_matrix(next, 0, j);
      }
      if (kFast || u % RB < blocks) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[u % RB][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[u / RB][j], af[(kFrom + u) % kRing],
                                                                 acc[u % RB][j], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  static __device__ __forceinline__ uint32_t after(uint32_t slot) { return slot == kBSlots - 1 ? 0 : slot + 1; }
  // Two stages at a time while all their loads are of whole stages.
  template <int RB>
  __device__ __forceinline__ void fast_stages(int& s, uint32_t& slot) {
    if constexpr (RB > TM) return;
    else for (; s + 3 < whole; s += 2) {
      const uint32_t one = after(slot), two = after(one);
      stage<RB, true, 0>(s, slot, one, two);
      stage<RB, true, 1>(s + 1, one, two, slot);
      slot = two;
    }
  }

  __device__ __forceinline__ void accumulate() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kBLoads; ++i) load_matrix<false>(0, 0, i);
#pragma unroll
    for (int i = 0; i < kALoads; ++i)
      if (i < a_loads) load_rows<false>(0, i);
    if (stages > 1) {
#pragma unroll
      for (int i = 0; i < kBLoads; ++i) load_matrix<false>(1, 1, i);
      wait_loads<kBLoads>();
    } else {
      wait_loads<0>();
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kAhead && i < kALoads; ++i)
      if (i < a_loads && stages > 1) load_rows<false>(1, i);
#pragma unroll
    for (int j = 0; j < TN; ++j) read_matrix(0, 0, j);
    int s = 0;
    uint32_t slot = 0;  // of the matrix of stage s
    if (TM == 2 || blocks <= 2) {
      first_rows<2>();
      fast_stages<2>(s, slot);
      last_stages<2>(s, slot);
    } else {
      first_rows<TM>();
      if (blocks == 8) fast_stages<8>(s, slot);
      else if (blocks == 7) fast_stages<7>(s, slot);
      else if (blocks == 6) fast_stages<6>(s, slot);
      else if (blocks == 5) fast_stages<5>(s, slot);
      else if (blocks == 4) fast_stages<4>(s, slot);
      else fast_stages<3>(s, slot);
      last_stages<TM>(s, slot);
    }
  }
  template <int RB>
  __device__ __forceinline__ void first_rows() {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) af[u] = row_fragment<RB>(0, u);
  }
  // The last three or four.  (Past the last stage, fragments are read from a slot that nobody uses.)
  template <int RB>
  __device__ __forceinline__ void last_stages(int s, uint32_t slot) {
    s = __builtin_amdgcn_readfirstlane(s);  // (uniform, which the compiler loses sight of)
    slot = __builtin_amdgcn_readfirstlane(slot);
#pragma unroll 1
    for (; s < stages; ++s) {
      const uint32_t one = after(slot);
      stage<RB, false, 0>(s, slot, one, after(one));
      slot = one;
    }
  }

  __device__ __forceinline__ void run(int32_t height) {
    const int32_t ct = (g.out_cols + kOutCols - 1) / kOutCols;
    // Bands of up to eight row tiles of one group: what runs at one time on an XCD then shares rows and
    // matrix panels in its L2.  7168 x 4096, us, so / in fours of any groups: 256 experts of about 256
    // rows 2130 / 2400 (8.5 and 10.3 GB from beyond L2), of about 512 rows 3540 / 3850, 16 experts of
    // about 4096 rows 1537 / 1573; without a bound on the band, 8 experts of 8192 rows 1814 / 1458.
    if (!find_tile<8, true>(g.groups, height, ct, blockIdx.x, t)) return;
    setup();
    accumulate();
    lds_barrier();
    // Lane 16 q + m: row m of each block, columns 4 q .. 4 q + 3.
    const float* const row_scales = static_cast<const float*>(g.a_scales) + t.row0;
    const float* const col_scales = static_cast<const float*>(g.b_scales) + t.e * (g.b_stride / g.ldb);
    float scale[TM];
    f32x4 sums[TM][TN];
    uint32_t large = 0;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      scale[i] = row_scales[min((i * WM + wm) * 16 + (lane & 15), t.rows - 1)];
      large |= (uint32_t)split_scale(scale[i]) << i;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float col = col_scales[row_at(wn * kWaveCols + j * 16 + (lane >> 4) * 4 + c)];
#pragma unroll
        for (int i = 0; i < TM; ++i) sums[i][j][c] = (float)acc[i][j][c] * scale[i] * col;
      }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(large != 0) != 0, 0)) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) sums[i][j] *= large >> i & 1 ? kLargePart : 1.0f;
    }
    Store::store_tile(g, t, lds + wave * kWaveBytes, wm, wn, sums);
  }
};

// height: rows of a tile, at most kRows.
template <bool kGlu, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(kWaves * 64, TM > 4 ? 2 : 4) void gemm_int8_kernel(GemmArgs g, int32_t height) {
  typedef Int8Gemm<kGlu, TM, TN, WM, WN> G;
  __shared__ __align__(1024) char lds[G::kLdsBytes];
  G gemm(g, lds);
  gemm.run(height);
}

template <bool kGlu, int TM, int TN, int WM, int WN>
hipError_t launch(const GemmArgs& g, int32_t height, hipStream_t stream) {
  typedef Int8Gemm<kGlu, TM, TN, WM, WN> G;
  const int64_t ct = (g.out_cols + G::kOutCols - 1) / G::kOutCols;
  const int64_t blocks = (max_row_tiles(g.groups, height) * ct + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(blocks, kWaves * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_int8_kernel<kGlu, TM, TN, WM, WN><<<(uint32_t)blocks, kWaves * 64, 0, stream>>>(g, height);
  return hipGetLastError();
}

template <bool kGlu>
hipError_t launch_size(const GemmArgs& g, hipStream_t stream) {
  const Int8Tiles t = int8_tiles(g.groups, g.out_cols, kGlu, kChipCUs);
  if (t.few) return launch_gemm_int8_few(g, t.height, t.width, stream);
  if (t.height == 64) return launch<kGlu, 2, 2, 2, 4>(g, 64, stream);
  if (t.width == 128) return launch<kGlu, 4, 2, 2, 4>(g, 128, stream);
  return launch<kGlu, 8, 4, 2, 4>(g, t.height, stream);
}

}  // namespace

hipError_t launch_gemm_int8(const GemmArgs& g, hipStream_t stream) {
  return g.act == EP_ACT_SWIGLU ? launch_size<true>(g, stream) : launch_size<false>(g, stream);
}

}  // namespace ep
