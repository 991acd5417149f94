// ep_gemm_tile.hip -- bf16 and fp16 matrix products over ragged groups of rows,
// for groups of many rows: the experts' products, a dense layer's, and both
// kinds of gradients.
//
//   forward        out[r, n] = act(sum_k a[r, k] b[e, n, k] + bias[e, n]) + residual[r, n]
//   rows' gradient out[r, k] = (sum_n a[r, n] b[e, n, k]) act'(preact[r, k])
//   weights'       out[e, n, k] (+)= sum_{r in e} a[r, n] b[r, k]
//
// e is the group (expert) that row r belongs to.  The products are summed in
// fp32 by the matrix instructions and rounded once, after the epilogue.
//
// A workgroup of WM x WN waves makes one tile; each wave owns TM x TN blocks of
// 16 x 16 results.  The reduction is cut into units of 64, so that a load to LDS
// (which needs no registers) covers rows of 128 bytes: rows of 64 bytes, in units
// of 32, come in at 14.5 TB/s from L2 where these reach 31, and 256 x 256 tiles
// need 19.  LDS holds three units of the row operand and two of the matrix
// operand.  A step is half a unit, 32 deep: while the matrix instructions work on
// step s, the matrix fragments of step s + 1 and the next row fragments are read
// into registers, so a matrix unit is free a step earlier than a row unit, and
// the even steps bring in the row unit two units ahead, the odd steps the matrix
// unit.  One barrier a step is the only time that a wave stands still.
//
// The matrix operand takes the instruction's row side and the row operand its
// column side, so that a lane ends up with 4 neighbouring columns of one result
// row.  Where an operand has its reduction as the slow dimension, the
// transposing LDS read makes the fragments.
#include <type_traits>

#include "ep_gemm.h"

namespace ep {

namespace {

constexpr int kStep = 32;   // reduction elements per step: one matrix instruction's
constexpr int kUnit = 64;   // and per unit in LDS
constexpr int kASlots = 3;  // units of the row operand in LDS
constexpr int kBSlots = 2;  // and of the matrix operand

template <bool kF16>
struct Frag;
template <>
struct Frag<false> {
  typedef bf16x8 type;
  static __device__ __forceinline__ f32x4 mfma(type a, type b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<true> {
  typedef f16x8 type;
  static __device__ __forceinline__ f32x4 mfma(type a, type b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// How `kSpan` rows (or columns) of an operand sit in a unit of LDS, and how they
// get there.
//  Reduction contiguous in memory: kSpan rows of 128 bytes, 16-byte chunk c of
//  row r at place c ^ ((r >> 1) & 7).  A 16-byte read goes in four phases of 16
//  lanes, 0-3, 12-15, 20-23, 24-27 and so on; with this order the lanes of a
//  phase touch every bank once.
//  Reduction slow in memory: 64 rows of kSpan elements, pair p of 16-byte chunks
//  of row k at place p ^ f(k), f(k) = 4 * bit 3 of k + (k & 3): the eight rows
//  that one half wave of a transposing read touches lie in different banks.
template <bool kContiguous, int kSpan, int kWaves>
struct Operand {
  static constexpr int kBytes = kSpan * kUnit * 2;
  static constexpr int kLoads = kBytes / 1024 / kWaves;  // loads of a wave per unit
  static constexpr int kChunks = kContiguous ? 8 : kSpan / 8;  // chunks per LDS row
  static_assert(kContiguous || kSpan >= 128, "the bank pattern spans 16 chunks");

  static __device__ __forceinline__ int swizzle(int k) { return ((k >> 3) & 1) * 4 + (k & 3); }

  // The row (contiguous) or reduction row (slow) of this lane's i-th load, and its chunk.
  static __device__ __forceinline__ int load_row(int i) {
    return ((threadIdx.x >> 6) * kLoads + i) * (64 / kChunks) + (threadIdx.x & 63) / kChunks;
  }
  static __device__ __forceinline__ int load_chunk(int i) {
    const int place = (threadIdx.x & 63) % kChunks, row = load_row(i);
    return kContiguous ? (place ^ ((row >> 1) & 7)) : (place ^ (swizzle(row) << 1));
  }
};

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN>
struct TileGemm {
  static constexpr int kWaves = WM * WN;
  static constexpr int kRows = 16 * TM * WM;  // result rows of a tile
  static constexpr int kCols = 16 * TN * WN;  // product columns of a tile
  static constexpr bool kAContig = kMode != kWeightsGrad;
  static constexpr bool kBContig = kMode == kForward;
  typedef Operand<kAContig, kRows, kWaves> A;
  typedef Operand<kBContig, kCols, kWaves> B;
  typedef typename Frag<kF16>::type F;
  static constexpr int kLdsBytes = kASlots * A::kBytes + kBSlots * B::kBytes;
  static constexpr int kAhead = TM == 8 ? 4 : 2;  // row fragments read ahead
  static constexpr int kRing = TM == 8 ? 8 : 4;   // at least kAhead + 2: a pair is in use meanwhile
  static constexpr int kWaveCols = 16 * TN;
  static constexpr int kWaveBytes = kLdsBytes / kWaves / 1024 * 1024;
  typedef TileStore<kMode, kF16, kGlu, TM, TN, WM, WN, kWaveBytes> Store;
  static constexpr int kOutCols = Store::kOutCols;

  const GemmArgs& g;
  char* const lds;
  uint32_t lds0;
  Tile t;
  int32_t reduce, units, whole_units;
  int32_t a_limit, b_limit;  // valid rows (contiguous) or columns (slow) of each operand
  const char *a0, *b0;       // first element of the operand of this tile
  int64_t a_step, b_step;    // bytes from one unit to the next
  uint32_t a_off[A::kLoads], b_off[B::kLoads];
  uint32_t a_read, b_read;
  uint32_t a_place, b_place;  // where a wave's loads go in slot 0
  int wm, wn, lane;
  int blocks;  // blocks of 16 rows of this wave that the tile has
  f32x4 acc[TM][TN];
  float bias_sum[2];
  bool bias_tile;
  F af[kRing], bf[2][TN];

  __device__ __forceinline__ TileGemm(const GemmArgs& args, char* smem) : g(args), lds(smem) {}

  __device__ __forceinline__ int row_at(int p) const {
    return matrix_row(kGlu && kMode == kForward, p, kWaveCols, t.col * kOutCols, g.out_cols);
  }

  __device__ __forceinline__ void setup() {
    lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    lds0 = __builtin_amdgcn_readfirstlane(lds_address(lds));
    blocks = __builtin_amdgcn_readfirstlane(((t.rows + 15) / 16 - wm + WM - 1) / WM);
    a_place = lds0 + wave * A::kLoads * 1024;
    b_place = lds0 + kASlots * A::kBytes + wave * B::kLoads * 1024;
    whole_units = reduce / kUnit;
    units = tiles_of(reduce, kUnit);
#pragma unroll
    for (int i = 0; i < A::kLoads; ++i) {
      const int row = A::load_row(i), chunk = A::load_chunk(i);
      if constexpr (kAContig) a_off[i] = (uint32_t)min(row, a_limit - 1) * (uint32_t)g.lda * 2u + chunk * 16;
      else a_off[i] = (uint32_t)row * (uint32_t)g.lda * 2u + min(chunk * 8, a_limit - 8) * 2;
    }
    // A wave's rows of the matrix operand are neighbours in memory (all gates, or
    // all ups): offsets count from their first.
    static_assert(!kBContig || kWaveCols / 2 % (B::kLoads * 8) == 0, "a wave loads gates or ups");
    const int wave_row = kBContig ? row_at(wave * B::kLoads * 8) : 0;
    if constexpr (kBContig) b0 += (int64_t)wave_row * g.ldb * 2;
#pragma unroll
    for (int i = 0; i < B::kLoads; ++i) {
      const int row = B::load_row(i), chunk = B::load_chunk(i);
      if constexpr (kBContig) b_off[i] = (uint32_t)(row_at(row) - wave_row) * (uint32_t)g.ldb * 2u + chunk * 16;
      else b_off[i] = (uint32_t)row * (uint32_t)g.ldb * 2u + min(chunk * 8, b_limit - 8) * 2;
    }
    a_step = kAContig ? kUnit * 2 : (int64_t)kUnit * g.lda * 2;
    b_step = kBContig ? kUnit * 2 : (int64_t)kUnit * g.ldb * 2;
    a_read = read_offset<A, kAContig>(wm * 16);
    b_read = kASlots * A::kBytes + read_offset<B, kBContig>(wn * 16 * TN);
  }

  // LDS offset of this lane's part of the first fragment at row (column) w0.
  template <class Op, bool kContig>
  __device__ __forceinline__ uint32_t read_offset(int w0) const {
    const int q = lane >> 4, m = lane & 15;
    if constexpr (kContig) {
      return (w0 + m) * 128 + ((q ^ ((m >> 1) & 7)) << 4);
    } else {
      const int k = q * 8 + (m >> 2), gran = m & 3;
      return k * (Op::kChunks * 16) + (((w0 >> 3) ^ (Op::swizzle(k) << 1)) << 4) + ((gran >> 1) << 4) +
             ((gran & 1) << 3);
    }
  }

  // Fragment `tile` of half `kHalf` of the unit at LDS offset `unit`.  A wave's
  // blocks of the row operand are every WM-th one of the tile, so that a tile
  // with few rows is shared by all waves; those of the other operand are
  // neighbours.
  template <class Op, bool kContig, int kHalf>
  __device__ __forceinline__ F read_fragment(uint32_t offset, int tile) const {
    if constexpr (kContig) {
      return *reinterpret_cast<const F*>(lds + (offset ^ (kHalf * 64)) + tile * 2048);
    } else {
      // Two transposing reads: reduction rows q*8 .. q*8+3, and the four after them.
      const uint32_t at = (offset ^ (uint32_t)(tile << 5)) + kHalf * kStep * Op::kChunks * 16;
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)(lds0 + at));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds4*)(uintptr_t)(lds0 + at + 4 * Op::kChunks * 16));
      return __builtin_bit_cast(F, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  template <int kHalf>
  __device__ __forceinline__ F read_a(uint32_t unit, int i) const {
    return read_fragment<A, kAContig, kHalf>(unit + a_read, i * WM);
  }
  template <int kHalf>
  __device__ __forceinline__ F read_b(uint32_t unit, int j) const {
    return read_fragment<B, kBContig, kHalf>(unit + b_read, j);
  }

  // Load j of unit u of one operand, into the slot at LDS offset `slot` (of that
  // operand); whole: nothing of it lies past the reduction.
  template <bool kA>
  __device__ __forceinline__ void load_piece(const char* unit, uint32_t slot, int j) const {
    if constexpr (kA) load16_to_lds(unit, a_off[j], a_place + slot + j * 1024);
    else load16_to_lds(unit, b_off[j], b_place + slot + j * 1024);
  }
  // All loads of a unit; what lies past the reduction reads as zero.
  template <bool kA>
  __device__ __forceinline__ void load_unit(int u, uint32_t slot) const {
    typedef std::conditional_t<kA, A, B> Op;
    const int left = reduce - u * kUnit;
    const char* unit = kA ? a0 + u * a_step : b0 + u * b_step;
#pragma unroll
    for (int i = 0; i < Op::kLoads; ++i) {
      if (left >= kUnit) {
        load_piece<kA>(unit, slot, i);
      } else {
        const int r = (kA ? kAContig : kBContig) ? Op::load_chunk(i) * 8 : Op::load_row(i);
        const uint32_t off = kA ? a_off[kA ? i : 0] : b_off[kA ? 0 : i];
        load16_to_lds(r < left ? unit + off : reinterpret_cast<const char*>(g_zero16),
                      (kA ? a_place : b_place) + slot + i * 1024);
      }
    }
  }

  // Where things are in LDS while unit u is worked on: its row unit and the next
  // one, its matrix unit and the next one, and the row slot that is free.
  struct Slots {
    uint32_t a, a_next, a_free, b, b_next;
    __device__ __forceinline__ void turn() {
      const uint32_t free = a;
      a = a_next;
      a_next = a_free;
      a_free = free;
      const uint32_t last = b;
      b = b_next;
      b_next = last;
    }
  };

  // Step kHalf of unit u.  Its matrix fragments are in bf[kHalf] and its first
  // kAhead row fragments in af; the other row fragments are read while the
  // matrix instructions work, and so are the next step's first ones.
  template <int kHalf>
  __device__ __forceinline__ void step(int u, const Slots& at) {
    static_assert(TM % kRing == 0, "a step leaves the ring where it was");
    // Half 0: every wave is done with the row unit u - 1.  Half 1: unit u + 1 has
    // landed, for every wave (of later loads only the row unit u + 2 may be on
    // its way), and every wave is done with the matrix unit u.  All but the
    // youngest LDS reads, which are of units still in use, have returned.
    if constexpr (kHalf == 1) {
      if (u + 2 < units) wait_loads<A::kLoads>();
      else wait_loads<0>();
    }
    lds_barrier<kYoung>();
    const char* ahead = kHalf == 0 ? a0 + (u + 2) * a_step : b0 + (u + 2) * b_step;
    const uint32_t slot = kHalf == 0 ? at.a_free : at.b;
    const bool whole = u + 2 < whole_units;
    if (!whole && u + 2 < units) load_unit<kHalf == 0>(u + 2, slot);
    if constexpr (kMode == kWeightsGrad) {
      if (bias_tile) add_to_bias<kHalf>(at.a);
    }
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += 2) {
      if (i0 < blocks) {
        // Two matrix instructions, then one of the other operations, and so on.
#pragma unroll
        for (int n = 0; n < TN; ++n) {
#pragma unroll
          for (int m = 2 * n; m < 2 * n + 2; ++m)
            acc[i0 + m / TN][m % TN] =
                Frag<kF16>::mfma(bf[kHalf][m % TN], af[(i0 + m / TN) % kRing], acc[i0 + m / TN][m % TN]);
          for (int o = n; o < others<kHalf>(i0); o += TN) other_operation<kHalf>(i0, o, at, whole, ahead, slot);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int n = 0; n < others<kHalf>(i0); ++n) other_operation<kHalf>(i0, n, at, whole, ahead, slot);
      }
    }
  }
  // What goes with the rows i0 and i0 + 1: two reads of row fragments, kPieces
  // loads of a later unit, and in the first rows, before the reads of row
  // fragments turn to the next step's, kBReads reads of matrix fragments.
  static constexpr int kBReads = 2 * TN / (TM - kAhead);
  template <int kHalf>
  static constexpr int kLoadsOf = kHalf == 0 ? A::kLoads : B::kLoads;
  template <int kHalf>
  static constexpr int kPieces = (2 * kLoadsOf<kHalf> + TM - 1) / TM;
  template <int kHalf>
  static constexpr int others(int i0) {
    return 2 + kPieces<kHalf> + (i0 < TM - kAhead ? kBReads : 0);
  }
  template <int kHalf>
  __device__ __forceinline__ void other_operation(int i0, int n, const Slots& at, bool whole,
                                                  const char* ahead, uint32_t slot) {
    static_assert(kBReads * (TM - kAhead) == 2 * TN, "every matrix fragment has its turn");
    // (past the last unit these read a slot whose contents nobody uses)
    if (n < 2) {
      const int f = i0 + kAhead + n;
      af[f % kRing] = f < TM ? read_a<kHalf>(at.a, f)
                             : read_a<1 - kHalf>(kHalf == 0 ? at.a : at.a_next, f - TM);
    } else if (n < 2 + kPieces<kHalf>) {
      const int j = i0 / 2 * kPieces<kHalf> + n - 2;
      if (whole && j < kLoadsOf<kHalf>) load_piece<kHalf == 0>(ahead, slot, j);
    } else {
      const int j = i0 / 2 * kBReads + n - 2 - kPieces<kHalf>;
      bf[1 - kHalf][j] = read_b<1 - kHalf>(kHalf == 0 ? at.b : at.b_next, j);
    }
  }
  // The youngest LDS reads of a step, of the next step's row fragments: they come
  // after its last reads of its own row unit's half and of the matrix unit.
  static constexpr int kYoung = kAhead * (kAContig ? 1 : 2);
  static_assert(kYoung < 16, "lgkmcnt holds 4 bits");

  // Biases' gradient: the workgroups of the first column tile add up the rows of
  // dy that pass through their LDS, two columns and a part of the stage's rows
  // to a thread.
  static constexpr int kBiasParts = kWaves * 64 / (kRows / 2);
  template <int kHalf>
  __device__ __forceinline__ void add_to_bias(uint32_t unit) {
    const int pair = threadIdx.x % (kRows / 2), part = threadIdx.x / (kRows / 2);
#pragma unroll
    for (int j = 0; j < kStep / kBiasParts; ++j) {
      const int k = kHalf * kStep + part * (kStep / kBiasParts) + j;
      const uint32_t at = unit + k * (A::kChunks * 16) + (((pair >> 2) ^ (A::swizzle(k) << 1)) << 4) +
                          (pair & 3) * 4;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(lds + at);
      bias_sum[0] += elem_low<kF16>(w);
      bias_sum[1] += elem_high<kF16>(w);
    }
  }
  // Called by all threads once the operands' LDS is free; the parts meet there.
  __device__ __forceinline__ void store_bias() {
    float* sums = reinterpret_cast<float*>(lds);
    sums[threadIdx.x * 2] = bias_sum[0];
    sums[threadIdx.x * 2 + 1] = bias_sum[1];
    __syncthreads();
    for (int n = threadIdx.x; n < kRows && (int)t.row0 + n < g.out_rows; n += kWaves * 64) {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < kBiasParts; ++p) s += sums[p * kRows + n];
      const int64_t at = (int64_t)t.e * g.out_rows + t.row0 + n;
      if (g.grad_f32) {
        float* p = static_cast<float*>(g.bias_grad) + at;
        *p = g.accumulate ? *p + s : s;
      } else {
        if (g.accumulate) s += elem_at<kF16>(g.bias_grad, at);
        static_cast<uint16_t*>(g.bias_grad)[at] = elem_rne<kF16>(s);
      }
    }
    __syncthreads();
  }

  __device__ __forceinline__ void accumulate() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    bias_sum[0] = bias_sum[1] = 0.f;
    if (units == 0) return;
    load_unit<true>(0, 0);
    load_unit<false>(0, 0);
    if (units > 1) {
      load_unit<true>(1, A::kBytes);
      load_unit<false>(1, B::kBytes);
      wait_loads<A::kLoads + B::kLoads>();
    } else {
      wait_loads<0>();
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) af[i] = read_a<0>(0, i);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[0][j] = read_b<0>(0, j);
    Slots at = {0, A::kBytes, 2 * A::kBytes, 0, B::kBytes};
    for (int u = 0; u < units; ++u) {
      step<0>(u, at);
      step<1>(u, at);
      at.turn();
    }
  }

  // Where the tile's operands lie; false for a workgroup without a tile.
  __device__ __forceinline__ bool place() {
    if constexpr (kMode == kWeightsGrad) {
      const int32_t rt = (g.out_rows + kRows - 1) / kRows, ct = (g.out_cols + kCols - 1) / kCols;
      // Every group's tiles are shared out among the XCDs, since the groups'
      // reductions may differ much in length.
      const int32_t share = (rt * ct + kXcds - 1) / kXcds;
      const int32_t in_share = blockIdx.x / kXcds;
      t.e = in_share / share;
      const int32_t rem = (int32_t)(blockIdx.x % kXcds) * share + in_share % share;
      if (t.e >= g.groups.E || rem >= rt * ct) return false;
      constexpr int32_t kBand = 4;
      const int32_t band = rem / (kBand * ct), in = rem - band * kBand * ct;
      const int32_t high = min(kBand, rt - band * kBand);
      t.row0 = (int64_t)(band * kBand + in % high) * kRows;
      t.col = in / high;
      t.rows = (int32_t)min((int64_t)kRows, g.out_rows - t.row0);
      bias_tile = g.bias_grad != nullptr && t.col == 0;
      const int64_t first = group_first(g.groups, t.e);
      reduce = __builtin_amdgcn_readfirstlane(group_count(g.groups, t.e));
      a_limit = g.out_rows - (int32_t)t.row0;
      b_limit = g.out_cols - t.col * kCols;
      a0 = static_cast<const char*>(g.a) + (first * g.lda + t.row0) * 2;
      b0 = static_cast<const char*>(g.b) + (first * g.ldb + (int64_t)t.col * kCols) * 2;
    } else {
      const int32_t ct = (g.out_cols + kOutCols - 1) / kOutCols;
      if (!find_tile<4>(g.groups, kRows, ct, blockIdx.x, t)) return false;
      reduce = g.reduce;
      a_limit = t.rows;
      a0 = static_cast<const char*>(g.a) + t.row0 * g.lda * 2;
      b0 = static_cast<const char*>(g.b) + t.e * g.b_stride * 2;
      if constexpr (kMode == kRowsGrad) {
        b_limit = g.out_cols - t.col * kCols;
        b0 += (int64_t)t.col * kCols * 2;
      }
    }
    return true;
  }

  __device__ __forceinline__ void run() {
    if (!place()) return;
    setup();
    accumulate();
    lds_barrier();  // every wave is done with its operands
    if constexpr (kMode == kWeightsGrad) {
      if (bias_tile) store_bias();
    }
    Store::store_tile(g, t, lds + (wm * WN + wn) * kWaveBytes, wm, wn, acc);
  }
};

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 2) void gemm_tile_kernel(GemmArgs g) {
  typedef TileGemm<kMode, kF16, kGlu, TM, TN, WM, WN> G;
  __shared__ __align__(1024) char lds[G::kLdsBytes];
  G gemm(g, lds);
  gemm.run();
}

template <int kMode, bool kF16, bool kGlu, int TM, int TN, int WM, int WN>
hipError_t launch(const GemmArgs& g, hipStream_t stream) {
  typedef TileGemm<kMode, kF16, kGlu, TM, TN, WM, WN> G;
  const int64_t ct = (g.out_cols + G::kOutCols - 1) / G::kOutCols;
  const int64_t rt = kMode == kWeightsGrad
                         ? (int64_t)g.groups.E * ((g.out_rows + G::kRows - 1) / G::kRows)
                         : max_row_tiles(g.groups, G::kRows);
  const int64_t rounds = kMode == kWeightsGrad ? (rt / g.groups.E * ct + kXcds - 1) / kXcds * g.groups.E
                                               : (rt * ct + kXcds - 1) / kXcds;
  const int64_t blocks = rounds * kXcds;
  if (!grid_fits(blocks, WM * WN * 64)) return hipErrorInvalidValue;
  if (blocks == 0) return hipSuccess;
  gemm_tile_kernel<kMode, kF16, kGlu, TM, TN, WM, WN>
      <<<(uint32_t)blocks, WM * WN * 64, 0, stream>>>(g);
  return hipGetLastError();
}

// Eight waves for the small tile too: with four, one to a SIMD, nothing goes on
// while a wave waits (reduction 7168, 512 rows, 4096 columns: 65 us, four 72; rows'
// gradient of 512 x 4096 x 7168 44 us, four 49; 2048 x 16,384 x 4096 281, four 270).
template <int kMode, bool kF16, bool kGlu>
hipError_t launch_size(const GemmArgs& g, bool large, hipStream_t stream) {
  return large ? launch<kMode, kF16, kGlu, 8, 4, 2, 4>(g, stream)
               : launch<kMode, kF16, kGlu, 4, 2, 2, 4>(g, stream);
}

template <bool kF16>
hipError_t launch_mode(const GemmArgs& g, int mode, bool large, hipStream_t stream) {
  const bool glu = g.act == EP_ACT_SWIGLU;
  if (mode == kWeightsGrad)
    return launch_size<kWeightsGrad, kF16, false>(g, large, stream);
  if (mode == kRowsGrad)
    return glu ? launch_size<kRowsGrad, kF16, true>(g, large, stream)
               : launch_size<kRowsGrad, kF16, false>(g, large, stream);
  return glu ? launch_size<kForward, kF16, true>(g, large, stream)
             : launch_size<kForward, kF16, false>(g, large, stream);
}

}  // namespace

hipError_t launch_gemm_tile(const GemmArgs& g, int mode, bool f16, bool large, hipStream_t stream) {
  return f16 ? launch_mode<true>(g, mode, large, stream) : launch_mode<false>(g, mode, large, stream);
}

// Which kernel.  Tiles of 128 x 128 stream the matrix at 6.1 TB/s if there are
// enough of them, but one tile takes 0.6 us for every 64 of the reduction, however
// few there are.  So where there are few, the kernels whose waves share out the
// reduction are faster: 16 matrix rows to a workgroup fill the GPU from 4096
// columns on, but read a once for every 16 columns; 64 x 64 tiles are right up to
// one for every CU.  Measured, us, by 16 columns / 64 x 64 / 128 x 128:
//   reduction 7168: 16 rows, 4096 columns    13 /  31 /  89
//                   64 rows, 4096 columns    22 /  33 /  91
//                   256 rows, 4096 columns      /  40 /  72 (256 tiles of 64 x 64)
//                   512 rows, 4096 columns      /  77 /  65
//   reduction 4096: 16 rows, 16,384 columns  28 /  24 /
//                   64 rows, 16,384 columns  50 /  27 /  39
//   reduction 2048: 1024 rows, 1024 columns     /  15 /  25 (256)
//                   2048 rows, 1024 columns     /  28 /  24
//   reduction 2048, 32 experts of 1024 columns: 16 rows each (512) 41 / 29 / 24
//   reduction 256:  16 rows, 4096 columns   4.0 / 5.6 / 5.7
//                   64 rows, 2048 columns   4.3 / 7.1 / 6.3
//                   8 experts of 1024 columns, 32 rows each  8.8 / 5.8 / 6.6
//   reduction 2048, the same                                16.3 /12.7 /21.0
// (the last two are where counting 128 x 128 tiles errs: 512 or more workgroups of 16
// columns, one to a CU for their LDS, go in rounds).
// The gradients, 64 x 64 / 128 x 128:
//   rows', 16,384 x 4096, 16 rows            72 / 130 (64)
//          4096 x 7168, 128 rows             27 /  42 (224)
//          4096 x 7168, 256 rows             49 /  42 (448)
//          128 x 7168, 16 rows              5.7 / 5.1 (a reduction of 128)
//   weights', 9689 rows, 184 x 840           61 /  99 (42)
//             4096 rows, 1024 x 1024         31 /  46 (256)
//             8192 rows, 1024 x 2048        101 /  86 (512)
//             256 rows, 512 x 512           7.2 / 7.1 (64)
//             16 rows, 1024 x 1024          7.6 / 5.5 (256)
// so for them only from a reduction of 256 on.
// Otherwise 256 x 256 tiles where the groups have the rows for them and there
// are enough tiles for every CU.
hipError_t launch_gemm(const GemmArgs& g, int mode, bool f16, hipStream_t stream) {
  const RowGroups& r = g.groups;
  const int64_t rows = mode == kWeightsGrad ? g.out_rows : (r.wanted + r.E - 1) / r.E;
  const int64_t groups = mode == kWeightsGrad || r.wanted > r.E ? r.E : r.wanted;
  const int64_t columns = (int64_t)g.out_cols * (mode == kForward && g.act == EP_ACT_SWIGLU ? 2 : 1);
  if (mode == kForward && rows <= 64 && groups * ((columns + 127) / 128) * ((rows + 15) / 16) <= 128)
    return launch_gemm_few(g, mode, rows, false, f16, stream);
  const int64_t reduce = mode == kWeightsGrad ? (r.wanted + r.E - 1) / r.E : g.reduce;
  if (groups * ((rows + 63) / 64) * ((columns + 63) / 64) <= kChipCUs && (mode == kForward || reduce >= 256))
    return launch_gemm_few(g, mode, rows, true, f16, stream);
  const int64_t tiles = groups * ((rows + 255) / 256) * ((columns + 255) / 256);
  return launch_gemm_tile(g, mode, f16, rows >= 192 && tiles >= kChipCUs, stream);
}

}  // namespace ep
